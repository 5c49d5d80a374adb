// The grouped product for few rows an expert: each expert's weights are
// streamed once, and the streaming is all there is to it.
//
// One workgroup takes a run of up to 16 rows of one expert and `sweep` tiles
// of 32 output columns.  Its four waves share the contraction in consecutive
// quarters; a wave's loads go from memory straight into the operand registers
// of 16x16 MFMAs (16 bytes a lane: 64 bytes of each of 16 weight rows), the
// next four steps in flight while the present ones are multiplied, on across
// the tiles.  Lanes of rows that the run does not have read nothing.  The
// waves' sums meet in LDS, in wave order.  Workgroups find their run by
// themselves: one is launched for each row and column range, and the ones
// whose row does not begin a run end at once.
#include <algorithm>
#include <type_traits>

#include "grouped.hpp"

namespace qrmoe {

constexpr int kVecRun = 16, kVecWaves = 4;
constexpr int kVecTiles = 2, kVecCols = 16 * kVecTiles;  // columns of one pass
constexpr int kVecSteps = 4;                             // 64-byte steps loaded ahead

template <int NT, int U>
struct VecRegs {
    i32x4 x[U], y[NT][U];
    uint32_t sx[U], sy[NT][U];
};

// Scale words of steps s .. s+U-1 of one row (four blocks a step) with this
// lane's block in the low byte; zeros past the row's end and for no row.
template <int U>
__device__ __forceinline__ void vec_scales(uint32_t (&w)[U], const uint8_t *row, int s, int blocks, int q) {
    if (row && 4 * (s + U) <= blocks) {
        __builtin_memcpy(w, row + 4 * s, 4 * U);
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] >>= 8 * q;
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = row && 4 * (s + u) + q < blocks ? row[4 * (s + u) + q] : 0;
    }
}

template <Elt ELT, bool F32>
__global__ __launch_bounds__(kVecWaves * 64) void grouped_vec_kernel(GroupedArgs a) {
    constexpr bool FP4 = ELT == Elt::Fp4;
    constexpr int NT = kVecTiles, U = kVecSteps;
    typedef VecRegs<NT, U> Regs;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p = blockIdx.x / a.n_tiles, nb = (blockIdx.x - p * a.n_tiles) * (16 * NT * a.sweep);

    // ---- the group of row p: the first offset past p ends it, the largest of those before that one begins it (an
    // offset less than one before it counts as that one)
    int start = 0, next = a.E + 1, row1 = a.P;  // next: the offset that ends the group; E + 1: none, past the last group
    bool found = false;
    constexpr int kAhead = 5;  // 320 offsets in flight
    for (int i0 = 0; i0 <= a.E && !found; i0 += 64 * kAhead) {
        int o[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) o[j] = a.offsets[min(i0 + 64 * j + lane, a.E)];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int v = i0 + 64 * j + lane > a.E ? a.P : min(max(o[j], 0), a.P);
            const uint64_t past = __ballot(v > p);
            if (found) continue;
            const int at = past ? __ffsll((long long)past) - 1 : 64;
            start = lane < at ? max(start, v) : start;
            if (past) {
                found = true;
                next = min(i0 + 64 * j + at, a.E + 1);
                row1 = __builtin_amdgcn_readlane(v, at);
            }
        }
    }
    const int row0 = __builtin_amdgcn_readfirstlane(
        (int)group_reduce<64>((uint32_t)start, [](uint32_t x, uint32_t y) { return max(x, y); }));
    const bool none = next == 0 || next > a.E;  // before the first group or past the last
    const int e = none ? 0 : next - 1;
    if ((p - row0) % kVecRun != 0) return;
    const int rows = min(row1 - p, kVecRun);

    // ---- this lane's weight row (column n0 + l16) and activation row (p + l16)
    const int KB = FP4 ? a.depth / 2 : a.depth * 2;  // bytes of a row
    const int blocks = a.depth / 32;
    const uint8_t *xrow = nullptr, *xsrow = nullptr;
    if (!none && l16 < rows) {
        int src = p + l16;
        bool ok = true;
        if (a.rows) {
            src = a.rows[src];
            ok = (uint32_t)src < (uint32_t)a.src_rows;
        }
        if (ok) {
            xrow = a.x + src * a.x_ld;
            if constexpr (FP4) xsrow = a.xs + (int64_t)src * blocks;
        }
    }

    // ---- this wave's quarter of the contraction, in steps of 64 bytes
    const int steps = none ? 0 : (KB + 63) / 64;
    const int per = ((steps + kVecWaves - 1) / kVecWaves + U - 1) / U * U;
    const int s0 = wave * per;
    // iteration i: steps s0 + U c .. of column tile i / chunks, c = i % chunks
    const int chunks = per / U, n_end = min(a.N, nb + 16 * NT * a.sweep);
    const int iters = none ? 0 : chunks * ((n_end - nb + 16 * NT - 1) / (16 * NT));
    auto load = [&](Regs &r, int tile, int c) {
        const int s = s0 + c * U;
        const uint8_t *yrow[NT], *ysrow[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int n = nb + (tile * NT + t) * 16 + l16;
            yrow[t] = n < n_end ? a.y + e * a.y_mat + (int64_t)n * a.y_ld : nullptr;
            ysrow[t] = FP4 && n < n_end ? a.ys + ((int64_t)e * a.N + n) * blocks : nullptr;
        }
        if constexpr (FP4) {
            vec_scales<U>(r.sx, xsrow, s, blocks, q);
#pragma unroll
            for (int t = 0; t < NT; ++t) vec_scales<U>(r.sy[t], ysrow[t], s, blocks, q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = (s + u) * 64 + 16 * q;
            r.x[u] = i32x4{};
            if (at < KB && xrow) r.x[u] = *reinterpret_cast<const i32x4 *>(xrow + at);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                r.y[t][u] = i32x4{};
                if (at < KB && yrow[t])
                    r.y[t][u] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(yrow[t] + at));
            }
        }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{};
    auto multiply = [&](const Regs &r) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[t] = mfma16<ELT>(r.y[t][u], r.x[u], acc[t], FP4 ? (int)r.sy[t][u] : 0, FP4 ? (int)r.sx[u] : 0);
    };
    // ---- a tile's end: the quarters' sums, in wave order; register i: column 4 q + i of row l16
    __shared__ f32x4 part[2][kVecWaves][NT][64];
    typedef typename Out<ELT, F32>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    auto finish = [&](int tile) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            part[tile & 1][wave][t][lane] = acc[t];
            acc[t] = f32x4{};
        }
        lds_barrier();  // the other half of `part` is free again: every wave has passed its reads of tile - 1 before
        for (int t = wave; t < NT; t += kVecWaves) {
            const int n = nb + (tile * NT + t) * 16 + 4 * q;
            if (l16 >= rows || n >= n_end) continue;
            f32x4 v = part[tile & 1][0][t][lane];
#pragma unroll
            for (int w = 1; w < kVecWaves; ++w) v += part[tile & 1][w][t][lane];
            T4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = Out<ELT, F32>::cvt(v[i]);
            *reinterpret_cast<T4 *>((T *)a.out + (int64_t)(p + l16) * a.out_ld + n) = o;
        }
    };
    if (iters == 0) {
        for (int n = nb + 4 * tid; n < n_end; n += 4 * kVecWaves * 64)
            for (int r = 0; r < rows; ++r)
                *reinterpret_cast<T4 *>((T *)a.out + (int64_t)(p + r) * a.out_ld + n) = T4{};
        return;
    }
    Regs ra, rb;
    int tile = 0, c = 0, lt = 0, lc = 0;  // being multiplied; being loaded
    auto advance = [&](int &tl, int &ch) {
        if (++ch == chunks) ch = 0, ++tl;
    };
    load(ra, 0, 0);
    advance(lt, lc);
    auto turn = [&](Regs &now, Regs &next, int i) {
        if (i + 1 < iters) {
            load(next, lt, lc);
            advance(lt, lc);
        }
        multiply(now);
        if (c == chunks - 1) finish(tile);
        advance(tile, c);
    };
    for (int i = 0; i < iters; i += 2) {
        turn(ra, rb, i);
        if (i + 1 < iters) turn(rb, ra, i + 1);
    }
}

hipError_t launch_grouped_vec(GroupedArgs a, Elt elt, bool f32, hipStream_t s) {
    constexpr int64_t kBytes = 256 << 10, kWorkgroups = 1024;
    const int64_t tile = (int64_t)kVecCols * a.y_ld, tiles = (a.N + kVecCols - 1) / kVecCols;
    // Column tiles of one workgroup: enough that it streams 256 KB of weights,
    // while four workgroups a CU are left.  4096 x 4096 four-bit weights (64 KB
    // a tile), 32 / 128 tokens top-6 of 256: 165 / 579 us with one tile a
    // workgroup, 136 / 471 with four; one token 15.0 us with one, 22.1 with four.
    a.sweep = (int32_t)std::max<int64_t>(1, std::min(kBytes / tile, tiles * a.P / kWorkgroups));
    a.n_tiles = (int32_t)((tiles + a.sweep - 1) / a.sweep);
    const dim3 grid((unsigned)((int64_t)a.n_tiles * a.P)), block(kVecWaves * 64);
    auto go = [&](auto e) {
        constexpr Elt E = decltype(e)::value;
        if (f32) klaunch(grouped_vec_kernel<E, true>, grid, block, s, a);
        else klaunch(grouped_vec_kernel<E, false>, grid, block, s, a);
    };
    if (elt == Elt::Bf16) go(std::integral_constant<Elt, Elt::Bf16>{});
    else if (elt == Elt::F16) go(std::integral_constant<Elt, Elt::F16>{});
    else go(std::integral_constant<Elt, Elt::Fp4>{});
    return hipGetLastError();
}

}  // namespace qrmoe
