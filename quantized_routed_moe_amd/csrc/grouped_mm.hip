// Products grouped by expert, and their gradients.
//
//   forward  c[p][n]  = sum_k a[r(p)][k] b[e(p)][n][k]     b: [E][N][K]
//   grad_a   da[p][k] = sum_n dc[p][n] b[e(p)][n][k]
//   grad_b   db[e][n][k] = sum over the group's rows p of dc[p][n] a[r(p)][k]
//
// All three are out[m][n] = sum over d of x(m, d) y(n, d).  An operand is
// stored either along d ("row" operand: x and y of forward, x of grad_a) or
// across it ("column" operand: y of grad_a, both of grad_b).
#include <type_traits>

#include "grouped.hpp"

namespace qrmoe {

constexpr int kSlab = 128;  // bytes of one row operand's row, per K step: 64 elements of 16 bits, 256 of four
constexpr int kStep = 64;   // rows of a column operand per K step

// ---------------------------------------------------------------- tiles
// LDS image of one K step of an operand, R rows (columns) wide, 128 R bytes.
//  Row operand: [R][128 B], the 16-byte piece c of row r in slot
//  c ^ ((r >> 1) & 7).  An MFMA operand read takes one piece of 32
//  consecutive rows; any 16 of them then cover all 64 banks once.
//  Column operand: [64][2 R B], piece c of row d in slot c ^ ((d & 3) << 2):
//  a transposing read takes 32 bytes of four consecutive rows, which the
//  exchange puts into four different 64-byte groups of banks.
template <int R, int NW, bool COL>
struct Stager {
    static constexpr int kLoads = R / 8 / NW;  // 1 KB copies of each wave and step
    static_assert(kLoads >= 1, "every wave copies");
    uint32_t off[kLoads];  // byte offset of this lane's piece, or kOob
    uint32_t rem[kLoads];  // row operand: byte position of the piece inside the K step; column: its row of the step

    // row operand
    __device__ __forceinline__ int row(int i) const {
        return ((threadIdx.x >> 6) * kLoads + i) * 8 + ((threadIdx.x & 63) >> 3);
    }
    static __device__ __forceinline__ int piece(int r) { return (threadIdx.x & 7) ^ ((r >> 1) & 7); }
    // column operand
    static constexpr int kPer = R / 8;  // pieces of one row
    __device__ __forceinline__ int col_row(int i) const {
        return ((threadIdx.x >> 6) * kLoads + i) * (64 / kPer) + (threadIdx.x & 63) / kPer;
    }
    static __device__ __forceinline__ int col_piece(int d) { return ((threadIdx.x & 63) % kPer) ^ ((d & 3) << 2); }
};

struct Frag {
    i32x4 v;
};

typedef __attribute__((address_space(3))) i16x4 *lds_i16x4;

// Where workgroup b's tile lies: tiles are dealt in contiguous runs to the
// eight XCDs (workgroups go round them in turn), so that the tiles that share
// an operand run behind the same L2; inside a run kGroupM row tiles advance
// together through the columns.
constexpr int kXcds = 8, kGroupM = 4;
__device__ __forceinline__ bool xcd_tile(int b, int total, int &t) {
    const int per = (total + kXcds - 1) / kXcds;
    t = (b % kXcds) * per + b / kXcds;
    return b / kXcds < per && t < total;
}
__device__ __forceinline__ void tile_mn(int t, int m_tiles, int n_tiles, int &m, int &n) {
    const int g = t / (kGroupM * n_tiles), first = g * kGroupM, gm = min(kGroupM, m_tiles - first);
    const int r = t - g * kGroupM * n_tiles;
    m = first + r % gm;
    n = r / gm;
}

template <Elt ELT, bool XCOL, bool YCOL, int BM, int BN, int WM, int WN, bool F32>
__global__ __launch_bounds__(WM *WN * 64) void grouped_gemm_kernel(GroupedArgs a) {
    constexpr int NW = WM * WN, MI = BM / WM / 32, NI = BN / WN / 32;
    constexpr bool FP4 = ELT == Elt::Fp4;
    constexpr int kStages = 2;
    constexpr int XB = BM * kSlab, YB = BN * kSlab;
    typedef Stager<BM, NW, XCOL> SX;
    typedef Stager<BN, NW, YCOL> SY;
    __shared__ __align__(1024) uint8_t smem[kStages * (XB + YB)];
    __shared__ __align__(16) uint8_t sscale[FP4 ? kStages * (BM + BN) * 8 : 16];

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // ---- this workgroup's tile
    int e, row0, rows, m0, n0, depth;
    bool none = false;  // rows of no group
    if constexpr (XCOL) {
        int t, mt, nt;
        if (!xcd_tile(blockIdx.x, a.E * a.m_tiles * a.n_tiles, t)) return;
        e = t / (a.m_tiles * a.n_tiles);
        tile_mn(t - e * a.m_tiles * a.n_tiles, a.m_tiles, a.n_tiles, mt, nt);
        m0 = mt * BM;
        n0 = nt * BN;
        row0 = min(max(a.offsets[e], 0), a.P);
        rows = max(min(max(a.offsets[e + 1], 0), a.P) - row0, 0);
        depth = rows;
    } else {
        const TileList<BM> list(a.offsets, a.E, a.P);
        int t, mt, nt;
        if (!xcd_tile(blockIdx.x, list.total * a.n_tiles, t)) return;
        tile_mn(t, list.total, a.n_tiles, mt, nt);
        const RowTile r = list.find(mt);
        none = r.expert < 0 || r.expert >= a.E;
        e = none ? 0 : r.expert;
        row0 = m0 = r.row0;
        rows = r.rows;
        n0 = nt * BN;
        depth = none ? 0 : a.depth;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    depth = __builtin_amdgcn_readfirstlane(depth);
    n0 = __builtin_amdgcn_readfirstlane(n0);
    m0 = __builtin_amdgcn_readfirstlane(m0);
    constexpr int kElems = FP4 ? 256 : kStep;  // contraction elements of one K step
    const int steps = (depth + kElems - 1) / kElems;

    // ---- copies of one K step
    SX sx;
    SY sy;
    const uint8_t *xb, *yb;  // bases, advanced by one step at a time
    int64_t x_step, y_step;
    if constexpr (XCOL) {
        xb = a.x + (int64_t)row0 * a.x_ld + (int64_t)m0 * 2;
        x_step = kStep * a.x_ld;
#pragma unroll
        for (int i = 0; i < SX::kLoads; ++i) {
            const int d = sx.col_row(i), c = SX::col_piece(d);
            sx.rem[i] = d;
            sx.off[i] = m0 + 8 * c < a.M ? (uint32_t)(d * a.x_ld + 16 * c) : kOob;
        }
    } else {
        x_step = kSlab;
        xb = a.rows ? a.x : a.x + (int64_t)row0 * a.x_ld;
#pragma unroll
        for (int i = 0; i < SX::kLoads; ++i) {
            const int r = sx.row(i), c = SX::piece(r);
            int src = r;
            bool ok = r < rows && !none;
            if (a.rows && ok) {
                src = a.rows[row0 + r];
                ok = (uint32_t)src < (uint32_t)a.src_rows;
            }
            sx.rem[i] = 16 * c;
            sx.off[i] = ok ? (uint32_t)(src * a.x_ld + 16 * c) : kOob;
        }
    }
    if constexpr (YCOL) {
        const bool rows_y = XCOL;  // grad_b: y is a, whose rows are the contraction
        yb = rows_y ? (a.rows ? a.y : a.y + (int64_t)row0 * a.y_ld) + (int64_t)n0 * 2
                    : a.y + e * a.y_mat + (int64_t)n0 * 2;
        y_step = rows_y && a.rows ? 0 : kStep * a.y_ld;
#pragma unroll
        for (int i = 0; i < SY::kLoads; ++i) {
            const int d = sy.col_row(i), c = SY::col_piece(d);
            sy.rem[i] = d;
            sy.off[i] = n0 + 8 * c < a.N ? (uint32_t)((rows_y && a.rows ? 0 : d * a.y_ld) + 16 * c) : kOob;
        }
    } else {
        yb = a.y + e * a.y_mat + (int64_t)n0 * a.y_ld;
        y_step = kSlab;
#pragma unroll
        for (int i = 0; i < SY::kLoads; ++i) {
            const int r = sy.row(i), c = SY::piece(r);
            sy.rem[i] = 16 * c;
            sy.off[i] = n0 + r < a.N ? (uint32_t)(r * a.y_ld + 16 * c) : kOob;
        }
    }
    // grad_b with gathered rows: the source row of each copy, one step ahead
    int src[SY::kLoads];
    auto load_src = [&](int k) {
        if constexpr (XCOL && YCOL) {
            if (a.rows) {
#pragma unroll
                for (int i = 0; i < SY::kLoads; ++i) {
                    const int d = k * kStep + (int)sy.rem[i];
                    src[i] = d < depth ? a.rows[row0 + d] : -1;
                }
            }
        }
    };
    // four-bit operands: block scales of a step, 8 bytes a row; thread t holds the word t % 2 of row t / 2
    constexpr int kSX = FP4 ? (BM * 2 + NW * 64 - 1) / (NW * 64) : 1, kSY = FP4 ? (BN * 2 + NW * 64 - 1) / (NW * 64) : 1;
    uint32_t wsx[kSX], wsy[kSY];
    const uint8_t *px[kSX], *py[kSY];
    const int blocks = depth / 32;
    if constexpr (FP4) {
#pragma unroll
        for (int i = 0; i < kSX; ++i) {
            const int r = (i * NW * 64 + tid) >> 1;
            int s = -1;
            if (r < rows && !none) s = a.rows ? a.rows[row0 + r] : row0 + r;
            if (a.rows && (uint32_t)s >= (uint32_t)a.src_rows) s = -1;
            px[i] = s < 0 ? nullptr : a.xs + (int64_t)s * blocks;
        }
#pragma unroll
        for (int i = 0; i < kSY; ++i) {
            const int r = (i * NW * 64 + tid) >> 1;
            py[i] = r < BN && n0 + r < a.N ? a.ys + ((int64_t)e * a.N + n0 + r) * blocks : nullptr;
        }
    }
    auto load_word = [&](const uint8_t *p, int b) -> uint32_t {  // scales b .. b+3 of a row, zeros past its end
        uint32_t w = 0;
        if (p && b < blocks) {
            if (b + 4 <= blocks)
                __builtin_memcpy(&w, p + b, 4);
            else
                for (int j = 0; j < blocks - b; ++j) w |= (uint32_t)p[b + j] << (8 * j);
        }
        return w;
    };
    auto load_scales = [&](int k) {
        if constexpr (FP4) {
#pragma unroll
            for (int i = 0; i < kSX; ++i) wsx[i] = load_word(px[i], 8 * k + 4 * (tid & 1));
#pragma unroll
            for (int i = 0; i < kSY; ++i) wsy[i] = load_word(py[i], 8 * k + 4 * (tid & 1));
        }
    };
    auto store_scales = [&](int stg) {
        if constexpr (FP4) {
            uint32_t *d = reinterpret_cast<uint32_t *>(sscale + stg * (BM + BN) * 8);
#pragma unroll
            for (int i = 0; i < kSX; ++i) {
                const int w = i * NW * 64 + tid;
                if (w < BM * 2) d[w] = wsx[i];
            }
#pragma unroll
            for (int i = 0; i < kSY; ++i) {
                const int w = i * NW * 64 + tid;
                if (w < BN * 2) d[BM * 2 + w] = wsy[i];
            }
        }
    };
    const int row_bytes = FP4 ? depth / 2 : depth * 2;
    const uint32_t lds0 = lds_addr(smem);
    auto issue = [&](int k, int stg) {
        const i32x4 rx = dma_rsrc(xb + k * x_step), ry = dma_rsrc(yb + k * y_step);
        const uint32_t lx = lds0 + stg * (XB + YB) + wave * (SX::kLoads * 1024);
        const uint32_t ly = lds0 + stg * (XB + YB) + XB + wave * (SY::kLoads * 1024);
        const uint32_t left_x = XCOL ? depth - k * kStep : row_bytes - k * kSlab;
        const uint32_t left_y = YCOL ? depth - k * kStep : row_bytes - k * kSlab;
#pragma unroll
        for (int i = 0; i < SX::kLoads; ++i) dma16_async(rx, lx + i * 1024, sx.rem[i] < left_x ? sx.off[i] : kOob);
#pragma unroll
        for (int i = 0; i < SY::kLoads; ++i) {
            uint32_t o = sy.rem[i] < left_y ? sy.off[i] : kOob;
            if constexpr (XCOL && YCOL)
                if (a.rows)
                    o = sy.off[i] != kOob && (uint32_t)src[i] < (uint32_t)a.src_rows
                            ? (uint32_t)(src[i] * a.y_ld + sy.off[i]) : kOob;
            dma16_async(ry, ly + i * 1024, o);
        }
    };

    // ---- operand reads: 32 rows (columns) at w0 of the tile, 32 bytes (16 rows) kk of the step
    const int swz = (l32 >> 1) & 7;
    auto read_row = [&](const uint8_t *t, int w0, int kk) -> i32x4 {
        return *reinterpret_cast<const i32x4 *>(t + (w0 + l32) * kSlab + 16 * ((2 * kk + half) ^ swz));
    };
    // lane l gets elements d = 16 kk + 8 half .. +7 of column w0 + l32: two
    // transposing reads of four rows each; lanes 4 j .. 4 j + 3 of a group of
    // 16 read 32 bytes of row j, lane i receives column i of the four rows
    const int tr_d = 8 * half + ((lane & 15) >> 2), tr_c = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    auto read_col = [&](const uint8_t *t, int width, int w0, int kk) -> i32x4 {
        const int d = 16 * kk + tr_d, c = w0 + tr_c;
        const uint8_t *p = t + d * width * 2 + (((c >> 3) ^ ((d & 3) << 2)) << 4) + (c & 7) * 2;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)p);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)(p + 4 * width * 2));
        struct { i16x4 a, b; } both{lo, hi};
        return __builtin_bit_cast(i32x4, both);
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};

    auto compute = [&](int stg) {
        const uint8_t *tx = smem + stg * (XB + YB), *ty = tx + XB;
        uint64_t qx[MI], qy[NI];
        if constexpr (FP4) {
            const uint8_t *s = sscale + stg * (BM + BN) * 8;
#pragma unroll
            for (int i = 0; i < MI; ++i)
                qx[i] = *reinterpret_cast<const uint64_t *>(s + (wm * MI * 32 + i * 32 + l32) * 8) >> (8 * half);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                qy[j] = *reinterpret_cast<const uint64_t *>(s + (BM + wn * NI * 32 + j * 32 + l32) * 8) >> (8 * half);
        }
        auto step = [&](auto kk_c) {
            constexpr int kk = decltype(kk_c)::value, S = (kk & 1) * 2;
            i32x4 xf[MI], yf[NI];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                xf[i] = XCOL ? read_col(tx, BM, wm * MI * 32 + i * 32, kk) : read_row(tx, wm * MI * 32 + i * 32, kk);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                yf[j] = YCOL ? read_col(ty, BN, wn * NI * 32 + j * 32, kk) : read_row(ty, wn * NI * 32 + j * 32, kk);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = mfma32<ELT, S>(yf[j], xf[i], acc[i][j], FP4 ? (int)(qy[j] >> (kk >> 1) * 32) : 0,
                                               FP4 ? (int)(qx[i] >> (kk >> 1) * 32) : 0);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
    };

    // ---- K steps: while step k is multiplied, step k + 1 arrives in the other half
    if (steps > 0) {
        load_src(0);
        load_scales(0);
        issue(0, 0);
        load_src(1);
        store_scales(0);
    }
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        const int stg = k & 1;
        wait_vm<0>();
        lds_barrier();
        if (k + 1 < steps) {
            load_scales(k + 1);
            issue(k + 1, stg ^ 1);
            load_src(k + 2);
        }
        compute(stg);
        if (k + 1 < steps) store_scales(stg ^ 1);
    }

    // ---- out: register 4 q + i of a tile holds column 8 q + 4 half + i of row l32
    typedef typename Out<ELT, F32>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T *out = (T *)a.out;
    if constexpr (XCOL) out += (int64_t)e * a.M * a.out_ld;
    const int m_end = XCOL ? a.M : m0 + rows;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = m0 + (wm * MI + i) * 32 + l32;
        if (m >= m_end) continue;
        T *o = out + (int64_t)m * a.out_ld;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int n = n0 + (wn * NI + j) * 32 + 4 * half;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (n + 8 * q >= a.N) continue;
                T4 v;
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = Out<ELT, F32>::cvt(acc[i][j][4 * q + u]);
                *reinterpret_cast<T4 *>(o + n + 8 * q) = v;
            }
        }
    }
}

// --------------------------------------------------------------- launches
namespace {

constexpr int kVecRowsPerGroup = 4;

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <Elt ELT, bool XCOL, bool YCOL, int BM, int BN, int WM, int WN>
hipError_t launch_tiles(GroupedArgs a, bool f32, hipStream_t s) {
    a.n_tiles = ceil_div(a.N, BN);
    a.m_tiles = ceil_div(a.M, BM);
    // row tiles of the ragged groups: at most one part tile for each group and for the rows before and past them
    const int64_t tiles = XCOL ? (int64_t)a.E * a.m_tiles * a.n_tiles : ((int64_t)a.P / BM + a.E + 2) * a.n_tiles;
    const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (f32)
        klaunch(grouped_gemm_kernel<ELT, XCOL, YCOL, BM, BN, WM, WN, true>, dim3((unsigned)grid), dim3(WM * WN * 64), s,
                a);
    else
        klaunch(grouped_gemm_kernel<ELT, XCOL, YCOL, BM, BN, WM, WN, false>, dim3((unsigned)grid), dim3(WM * WN * 64),
                s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_mm(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    if (a.P <= kVecRowsPerGroup * a.E) return launch_grouped_vec(a, elt, f32, s);
    switch (elt) {
        case Elt::Bf16: return launch_tiles<Elt::Bf16, false, false, 128, 128, 2, 2>(a, f32, s);
        case Elt::F16: return launch_tiles<Elt::F16, false, false, 128, 128, 2, 2>(a, f32, s);
        default: return launch_tiles<Elt::Fp4, false, false, 128, 128, 2, 2>(a, f32, s);
    }
}

hipError_t launch_grouped_grad_a(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    if (elt == Elt::Bf16) return launch_tiles<Elt::Bf16, false, true, 128, 128, 2, 2>(a, f32, s);
    return launch_tiles<Elt::F16, false, true, 128, 128, 2, 2>(a, f32, s);
}

hipError_t launch_grouped_grad_b(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    if (elt == Elt::Bf16) return launch_tiles<Elt::Bf16, true, true, 128, 128, 2, 2>(a, f32, s);
    return launch_tiles<Elt::F16, true, true, 128, 128, 2, 2>(a, f32, s);
}

}  // namespace qrmoe
