// The orthogonalised update: a matrix with the row and column space of g and
// singular values near 1, by Newton-Schulz products.
//
//   X = g / (|g| + eps), transposed where g is tall;  steps times
//     A = X X^T,   P = a I + b A + c A A,   X <- P X
//
// Small singular values grow by `a` a step, and so does whatever a rounding
// put beside them: 16 bits would show in the result (a step of 2^-12 can come
// out 500 times as large).  Everything between the products is therefore kept
// as two fp16 numbers, hi + lo, 22 bits, scaled by a power of two so that both
// stay clear of fp16's ends, and a product is three: hi hi + hi lo + lo hi,
// summed in fp32 by the matrix units.  What is left out, lo lo, is 2^-22.
//
// Layout of a split matrix: rows of 128-byte chunks, 32 hi and the same 32 lo
// elements each, rows padded with zeros to whole chunks.  One K step of an
// operand is a chunk of every row of the tile (or 32 rows of its columns), so
// hi and lo arrive together and each is multiplied from registers by both
// parts of the other operand: 48 matrix instructions a wave for the copies
// that 32 of a plain 16-bit product need.
//
// A and P are symmetric: the tiles on and below the diagonal are computed, a
// tile below is stored a second time, transposed on the way by LDS reads.
// The norm is taken out as a power of two when X is made, which is exact; what
// is left of it, a factor in (1, 2], goes into the first step's products.
//
// What bounds it: the matrix units.  16 x 4096 x 2048 bf16, five steps: 9.7 ms,
// of which the products 9.3 at up to 1310 TFLOP/s (P X: 2048 tiles of 256 x 256
// and 64 steps in 1255 us, the matrix units busy 74% at the clock that power
// allows; a library product of random 16-bit matrices reaches 1110 to 1310).
// The symmetric ones take 413 to 440 us for 288 steps of a CU, as 576 tiles
// are 2.25 rounds.  Norm, split and join move 1.6 GB at 3.8 to 5.5 TB/s in 330
// us.  The first step's products of 16-bit input have one part of X: 490 us
// instead of 750 for X X^T, where the copies then set the pace.
#include <algorithm>
#include <type_traits>

#include "mxfp4.hpp"
#include "ops.hpp"

namespace qrmoe {

namespace {

constexpr int kCus = 256, kXcds = 8;
constexpr int kChunk = 128;  // bytes of 32 split elements
enum : int { kSym = 0, kPoly = 1, kApply = 2 };  // x y^T, symmetric; P of A = x = y; x y

template <int N, int I = 0, class F>
__device__ __forceinline__ void unroll(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

typedef __attribute__((address_space(3))) i16x4 *lds_i16x4;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight values as two fp16 numbers each, v = hi + lo, both rounded to nearest: v is off by 2^-22 of itself at most, or by
// 2^-25 where that is more (the values are scaled to at most 2^15).  lo has to be taken from the hi that is stored: of
// the two conversions that the compiler may use for it (v_cvt_f16_f32 and v_cvt_pk_f16_f32) one rounds some values the
// other way, and a hi that is computed twice can come out a whole place apart.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void split8(const float (&v)[8], f16x8 &hi, f16x8 &lo) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t h = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[i], (_Float16)v[i + 1]});
        asm("" : "+v"(h));  // this value and no other
        const f16x2 p = __builtin_bit_cast(f16x2, h);
        hi[i] = p.x;
        hi[i + 1] = p.y;
        lo[i] = (_Float16)(v[i] - (float)p.x);
        lo[i + 1] = (_Float16)(v[i + 1] - (float)p.y);
    }
}

struct GemmArgs {
    const uint8_t *x, *y, *add;  // add: kPoly, A
    uint8_t *out;
    int64_t x_ld, y_ld, out_ld;     // row strides, bytes (add: as out)
    int64_t x_mat, y_mat, out_mat;  // a matrix of the batch, bytes (add: as out)
    int32_t rows, cols;             // of the output; cols padded to whole chunks
    int32_t y_rows;                 // kApply: contraction rows that y has
    int32_t steps;                  // chunks of the contraction
    int32_t batch, m_tiles, n_tiles;
    int32_t rounds, tail, parts;    // whole tiles of each workgroup; tiles behind them, the parts each is cut into
    float scale;                    // of the sum (not kPoly)
    float c0, c1, c2;               // kPoly: identity, A, A A
    const float *rest;              // what is left of each matrix's norm, or null
    int32_t rest_power;             // how often it goes into the sum
    float *partial;                 // [tail][parts] tiles of sums
    int32_t *arrived;               // [tail], zeros between launches
};

// Place in the list of tiles of turn b: runs of `run` consecutive tiles go to one XCD.
__device__ __forceinline__ int xcd_tile(int b, int run) {
    const int i = b / kXcds;
    return (i / run * kXcds + b % kXcds) * run + i % run;
}

// A tile, or part `part` of one of the tail: matrix, tile row and column, its steps k .. k + n - 1.
struct Tile {
    int b, m, n, k, steps, part, slot;  // slot: of the tail, or -1
};

// XL, YL: whether the operand has a lo part.  A workgroup a CU, eight waves of 128 x 64 (four of 64 x 64 in the small
// tile), walks its tiles; copies run RING - 1 steps ahead of the arithmetic, across tiles: what LDS holds beside the
// block that results leave through.  The small tile has four stages; with two 4 x 1024 x 1024 takes 514 us instead of
// 502, but 13 x 1000 x 519 483 instead of 487 and 64 x 128 x 128 175 instead of 191: in short products filling them costs
// what they hide.
template <int MODE, bool XL, bool YL, int BM, int BN, int WM, int WN, int RING>  // RING: stages of the LDS ring
__global__ __launch_bounds__(WM *WN * 64, WM *WN / 4) void split_gemm_kernel(GemmArgs a) {
    constexpr bool YCOL = MODE == kApply, TRI = !YCOL;
    constexpr int NW = WM * WN, MI = BM / WM / 32, NI = BN / WN / 32;
    constexpr int XB = BM * kChunk, YB = BN * kChunk, STAGE = XB + YB;
    constexpr int XC = BM / 8 / NW, YC = BN / 8 / NW;  // 1 KB copies of each wave and step
    constexpr int OUT_ROW = BN * 4;
    static_assert(!TRI || BM == BN, "tiles of a symmetric product are square");
    __shared__ __align__(1024) uint8_t smem[RING * STAGE + 32 * OUT_ROW];
    uint8_t *const sout = smem + RING * STAGE;

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // ---- the list of tiles: lower triangle row by row, or eight row tiles advancing through the columns together.
    // First whole tiles, as many for every workgroup; what is left over is cut along the contraction into as many
    // parts as there are workgroups for (each XCD takes the same part of neighbouring tiles).
    constexpr int kRun = kCus / kXcds;
    const int each = TRI ? a.m_tiles * (a.m_tiles + 1) / 2 : a.m_tiles * a.n_tiles;
    auto find = [&](int turn, Tile &t) -> bool {
        int at;
        t = Tile{0, 0, 0, 0, a.steps, 0, -1};
        if (turn < a.rounds) {
            at = xcd_tile(blockIdx.x + turn * kCus, kRun);
        } else {
            const int p = (blockIdx.x % kXcds) * kRun + blockIdx.x / kXcds;
            if (turn > a.rounds || p >= a.tail * a.parts) return false;
            at = a.rounds * kCus + p % a.tail;
            t.part = p / a.tail;
            t.slot = a.parts > 1 ? p % a.tail : -1;
            t.k = t.part * a.steps / a.parts;
            t.steps = (t.part + 1) * a.steps / a.parts - t.k;
        }
        t.b = at / each;
        const int r = at - t.b * each;
        if constexpr (TRI) {
            int m = (int)((__builtin_sqrtf(8.0f * r + 1.0f) - 1.0f) * 0.5f);
            while ((m + 1) * (m + 2) / 2 <= r) ++m;
            while (m * (m + 1) / 2 > r) --m;
            t.m = m;
            t.n = r - m * (m + 1) / 2;
        } else {
            const int g = r / (8 * a.n_tiles), gm = min(8, a.m_tiles - 8 * g), q = r - g * 8 * a.n_tiles;
            t.m = 8 * g + q % gm;
            t.n = q / gm;
        }
        t.b = __builtin_amdgcn_readfirstlane(t.b);
        t.m = __builtin_amdgcn_readfirstlane(t.m);
        t.n = __builtin_amdgcn_readfirstlane(t.n);
        return true;
    };

    // ---- the stream of copies.  Row operand: piece c (16 bytes) of row r in slot c ^ ((r >> 1) & 7); column operand:
    // [32][4 BN bytes], piece c of row d in slot c ^ ((d & 3) << 2).
    constexpr int kPer = BN * 4 / 16;  // pieces of a row of a column operand
    uint32_t xoff[XC], yoff[YC];
    const uint8_t *cx = nullptr, *cy = nullptr;
    int cturn = -1, cleft = 0, crows = 0;  // tile being sent for, its steps left, contraction rows left (kApply)
    auto x_row = [&](int i) { return (wave * XC + i) * 8 + (lane >> 3); };
    auto y_row = [&](int i) { return YCOL ? (wave * YC + i) * (64 / kPer) + lane / kPer : (wave * YC + i) * 8 + (lane >> 3); };
    auto next_tile = [&] {
        Tile t;
        const bool more = find(++cturn, t);
        cleft = more ? t.steps : 0x7fffffff;  // past the end: copies of nothing
        crows = a.y_rows - 32 * t.k;
        cx = a.x + t.b * a.x_mat + (int64_t)t.m * BM * a.x_ld + (int64_t)t.k * kChunk;
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const int r = x_row(i);
            xoff[i] = more && t.m * BM + r < a.rows ? (uint32_t)(r * a.x_ld + 16 * ((lane & 7) ^ ((r >> 1) & 7))) : kOob;
        }
        cy = a.y + t.b * a.y_mat + (YCOL ? (int64_t)t.n * BN * 4 + (int64_t)t.k * 32 * a.y_ld
                                         : (int64_t)t.n * BN * a.y_ld + (int64_t)t.k * kChunk);
#pragma unroll
        for (int i = 0; i < YC; ++i) {
            const int r = y_row(i);
            if constexpr (YCOL) {
                const int p = (lane % kPer) ^ ((r & 3) << 2);
                yoff[i] = more && t.n * BN + 4 * p < a.cols ? (uint32_t)(r * a.y_ld + 16 * p) : kOob;
            } else {
                yoff[i] = more && t.n * BN + r < a.rows ? (uint32_t)(r * a.y_ld + 16 * ((lane & 7) ^ ((r >> 1) & 7))) : kOob;
            }
        }
    };
    const uint32_t lds0 = lds_addr(smem);
    struct Copy {
        i32x4 rx, ry;
        uint32_t lx, ly;
    };
    auto begin_copy = [&](int stg) {
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + stg * STAGE);
        return Copy{dma_rsrc(cx), dma_rsrc(cy), base + wave * (XC * 1024), base + XB + wave * (YC * 1024)};
    };
    auto send = [&](const Copy &c, auto idx) {
        constexpr int I = decltype(idx)::value;
        if constexpr (I < XC) dma16_async(c.rx, c.lx + I * 1024, xoff[I]);
        else dma16_async(c.ry, c.ly + (I - XC) * 1024, !YCOL || y_row(I - XC) < crows ? yoff[I - XC] : kOob);
    };
    auto end_copy = [&] {
        if (--cleft == 0) {
            next_tile();
        } else {
            cx += kChunk;
            cy += YCOL ? 32 * a.y_ld : kChunk;
            crows -= 32;
        }
    };

    // ---- operand reads: 32 rows (columns) at w0, elements 16 s + 8 half .. +7 of the step, hi (L 0) or lo (1)
    const int swz = (l32 >> 1) & 7;
    auto read_row = [&](const uint8_t *t, int w0, int s, int L) -> i32x4 {
        return *reinterpret_cast<const i32x4 *>(t + (w0 + l32) * kChunk + 16 * ((4 * L + 2 * s + half) ^ swz));
    };
    const int tr_d = 8 * half + ((lane & 15) >> 2), tr_c = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    auto read_col = [&](const uint8_t *t, int w0, int s, int L) -> i32x4 {
        const int d = 16 * s + tr_d, at = (w0 >> 5) * kChunk + 64 * L + 2 * tr_c;
        const uint8_t *p = t + d * OUT_ROW + (((at >> 4) ^ ((d & 3) << 2)) << 4) + (at & 15);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)p);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)(p + 4 * OUT_ROW));
        struct { i16x4 a, b; } both{lo, hi};
        return __builtin_bit_cast(i32x4, both);
    };

    // ---- a tile's product.  A step is two halves s of 16 elements, each three groups of MFMAs: hi hi, hi lo, lo hi.
    // A group's operands are read during the group before.  A step's stage is free before its last group: there the
    // waves meet, the next step has arrived, and one more is sent for.
    constexpr int kCopies = XC + YC;
    const int wrow = wm * MI * 32, wcol = wn * NI * 32;
    int stg = 0;
    f32x16 acc[MI][NI];
    auto product = [&](int steps) {
        i32x4 xh[MI], xl[XL ? MI : 1], yh[2][NI], yl[YL ? NI : 1];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};
        auto read_x = [&](i32x4 &v, int st, int i, int s, int L) { v = read_row(smem + st * STAGE, wrow + i * 32, s, L); };
        auto read_y = [&](i32x4 &v, int st, int j, int s, int L) {
            const uint8_t *t = smem + st * STAGE + XB;
            v = YCOL ? read_col(t, wcol + j * 32, s, L) : read_row(t, wcol + j * 32, s, L);
        };
        auto mul = [&](const i32x4 &y, const i32x4 &x, f32x16 &c) { c = mfma32<Elt::F16, 0>(y, x, c, 0, 0); };
        constexpr int kMf = MI * NI;
        // what runs beside the MFMAs of a group: `reads` reads and `sends` copies, spread evenly
        auto group = [&](auto &&mm, auto reads_c, auto &&rd, auto sends_c, const Copy &c) {
            constexpr int R = decltype(reads_c)::value, S = decltype(sends_c)::value;
            unroll<kMf>([&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
                mm(std::integral_constant<int, m / NI>{}, std::integral_constant<int, m % NI>{});
                unroll<(m + 1) * R / kMf - m * R / kMf>([&](auto r_c) {
                    rd(std::integral_constant<int, m * R / kMf + decltype(r_c)::value>{});
                });
                unroll<(m + 1) * S / kMf - m * S / kMf>([&](auto s_c) {
                    send(c, std::integral_constant<int, m * S / kMf + decltype(s_c)::value>{});
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        constexpr std::integral_constant<int, 0> none{};
        auto nothing = [](auto) {};
#pragma unroll
        for (int j = 0; j < NI; ++j) read_y(yh[0][j], stg, j, 0, 0);
#pragma unroll
        for (int i = 0; i < MI; ++i) read_x(xh[i], stg, i, 0, 0);
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            // half 0
            group([&](auto i, auto j) { mul(yh[0][j], xh[i], acc[i][j]); },
                  std::integral_constant<int, (YL ? NI : 0) + (XL ? MI : 0)>{},
                  [&](auto r) {
                      constexpr int R = decltype(r)::value;
                      if constexpr (YL && R < NI) read_y(yl[R], stg, R, 0, 1);
                      else read_x(xl[R - (YL ? NI : 0)], stg, R - (YL ? NI : 0), 0, 1);
                  },
                  none, Copy{});
            if constexpr (YL)
                group([&](auto i, auto j) { mul(yl[j], xh[i], acc[i][j]); }, none, nothing, none, Copy{});
            if constexpr (XL) {
                group([&](auto i, auto j) { mul(yh[0][j], xl[i], acc[i][j]); }, std::integral_constant<int, NI + MI>{},
                      [&](auto r) {
                          constexpr int R = decltype(r)::value;
                          if constexpr (R < NI) read_y(yh[1][R], stg, R, 1, 0);
                          else read_x(xh[R - NI], stg, R - NI, 1, 0);
                      },
                      none, Copy{});
            } else {
#pragma unroll
                for (int j = 0; j < NI; ++j) read_y(yh[1][j], stg, j, 1, 0);
#pragma unroll
                for (int i = 0; i < MI; ++i) read_x(xh[i], stg, i, 1, 0);
            }
            // half 1; the last group runs on the other side of the barrier
            auto hand_over = [&] {
                wait_vm<(RING - 2) * kCopies>();
                lds_barrier();
            };
            auto ahead = [&](auto r) {  // the next step's first operands
                constexpr int R = decltype(r)::value;
                if constexpr (R < NI) read_y(yh[0][R], stg, R, 0, 0);
                else read_x(xh[R - NI], stg, R - NI, 0, 0);
            };
            constexpr std::integral_constant<int, NI + MI> all{};
            constexpr std::integral_constant<int, kCopies> copies{};
            if constexpr (XL) {
                group([&](auto i, auto j) { mul(yh[1][j], xh[i], acc[i][j]); },
                      std::integral_constant<int, (YL ? NI : 0) + MI>{},
                      [&](auto r) {
                          constexpr int R = decltype(r)::value;
                          if constexpr (YL && R < NI) read_y(yl[R], stg, R, 1, 1);
                          else read_x(xl[R - (YL ? NI : 0)], stg, R - (YL ? NI : 0), 1, 1);
                      },
                      none, Copy{});
                if constexpr (YL)
                    group([&](auto i, auto j) { mul(yl[j], xh[i], acc[i][j]); }, none, nothing, none, Copy{});
                hand_over();
                const Copy c = begin_copy(stg);
                stg = stg + 1 == RING ? 0 : stg + 1;
                group([&](auto i, auto j) { mul(yh[1][j], xl[i], acc[i][j]); }, all, ahead, copies, c);
            } else {
                // only hi hi: the operands are in registers, but xh is read for the next step while it is used
                i32x4 now[MI];
#pragma unroll
                for (int i = 0; i < MI; ++i) now[i] = xh[i];
                hand_over();
                const Copy c = begin_copy(stg);
                stg = stg + 1 == RING ? 0 : stg + 1;
                group([&](auto i, auto j) { mul(yh[1][j], now[i], acc[i][j]); }, all, ahead, copies, c);
            }
            end_copy();
        }
    };

    // ---- out, through LDS in blocks of 32 rows of fp32 sums; register 4 q + u of a 32x32 tile holds column
    // 8 q + 4 half + u of row l32.  16-byte slot c of row r is at c ^ (r & 63).  Eight columns (two slots) become
    // eight hi and eight lo elements of the same place, from which the transposed copy is read.
    auto slot_of = [&](int r, int c) { return sout + r * OUT_ROW + ((c ^ (r & (OUT_ROW / 16 - 1))) << 4); };
    auto finish = [&](const Tile &t) {
        const float rest = a.rest_power ? a.rest[t.b] : 1.0f;
        const float scale = a.scale * (a.rest_power == 2 ? rest * rest : a.rest_power == 1 ? rest : 1.0f);
        uint8_t *out = a.out + t.b * a.out_mat;
        const uint8_t *add = a.add + t.b * a.out_mat;
        const int m0 = t.m * BM, n0 = t.n * BN;
        const bool mirror = TRI && t.m != t.n;
        unroll<WM * MI>([&](auto part_c) {
            constexpr int part = decltype(part_c)::value, w0 = part / MI, i = part % MI;
            const int r0 = m0 + w0 * MI * 32 + i * 32;  // the block's first row
            if (r0 >= a.rows) return;
            if (wm == w0) {
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                        *reinterpret_cast<f32x4 *>(slot_of(l32, ((wn * NI + j) * 32 + 8 * q + 4 * half) >> 2)) = v;
                    }
            }
            lds_barrier();
            constexpr int kUnits = 32 * BN / 8;
#pragma unroll
            for (int s = 0; s < kUnits / (NW * 64); ++s) {
                const int p = s * NW * 64 + tid, r = p / (BN / 8), u = p % (BN / 8);  // row of the block, eight columns
                uint8_t *s0 = slot_of(r, 2 * u), *s1 = slot_of(r, 2 * u + 1);
                const f32x4 v0 = *reinterpret_cast<f32x4 *>(s0), v1 = *reinterpret_cast<f32x4 *>(s1);
                float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                const int row = r0 + r, col = n0 + 8 * u;
                const bool in = row < a.rows && col < a.cols;
                const int64_t at = row * a.out_ld + (col >> 5) * kChunk + (col & 31) * 2;
                if constexpr (MODE == kPoly) {
                    f16x8 h{}, l{};
                    if (in) {
                        h = *reinterpret_cast<const f16x8 *>(add + at);
                        l = *reinterpret_cast<const f16x8 *>(add + at + 64);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = __builtin_fmaf(a.c2, v[e], a.c1 * ((float)h[e] + (float)l[e])) + (row == col + e ? a.c0 : 0.0f);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= scale;
                }
                f16x8 h, l;
                split8(v, h, l);
                if (in) {
                    *reinterpret_cast<f16x8 *>(out + at) = h;
                    *reinterpret_cast<f16x8 *>(out + at + 64) = l;
                }
                if (mirror) {
                    *reinterpret_cast<f16x8 *>(s0) = h;
                    *reinterpret_cast<f16x8 *>(s1) = l;
                }
            }
            lds_barrier();
            if (mirror) {
                // rows of the transposed tile are columns here: 32 of them at a time, the chunk of the block's 32 rows;
                // a lane gets elements 8 half .. +7 (16 s further) of column w + l32, hi or lo
                for (int w = wave * 32; w < BN; w += NW * 32) {
                    const int row = n0 + w + l32;
#pragma unroll
                    for (int L = 0; L < 2; ++L)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int d = 16 * s + tr_d, c = w + tr_c;
                            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (lds_i16x4)(slot_of(d, 2 * (c >> 3) + L) + (c & 7) * 2));
                            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (lds_i16x4)(slot_of(d + 4, 2 * (c >> 3) + L) + (c & 7) * 2));
                            struct { i16x4 a, b; } both{lo, hi};
                            if (row < a.rows)
                                *reinterpret_cast<i32x4 *>(out + row * a.out_ld + (r0 >> 5) * kChunk + 64 * L + 32 * s +
                                                           16 * half) = __builtin_bit_cast(i32x4, both);
                        }
                }
                lds_barrier();
            }
        });
    };

    // ---- the parts of a tile of the tail: every part's sums go to memory, and the workgroup that comes last adds them
    // up, in the order of the parts whichever it is.  Nobody waits.  True for the last.  The sums are stored and loaded
    // past the XCD's own L2 (scope bit sc1), so that they need no fence, which would write back all of it: with fences
    // a product of 13 x 519 x 519 took 151 us.
    auto joined = [&](const Tile &t) -> bool {
        constexpr int kQuads = MI * NI * 4, kTile = BM * BN * 4, kAgent = 16;
        const auto sums = buf_rsrc((const uint8_t *)a.partial + (int64_t)t.slot * a.parts * kTile, a.parts * kTile);
        auto at = [&](int part, int quad) { return part * kTile + (quad * NW * 64 + tid) * 16; };
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), sums,
                                                           at(t.part, (i * NI + j) * 4 + q), 0, kAgent);
                }
        wait_vm<0>();  // this wave's sums are there
        lds_barrier();
        int *said = reinterpret_cast<int *>(sout);
        if (tid == 0) *said = atomicAdd(a.arrived + t.slot, 1);
        lds_barrier();
        const bool last = *said == a.parts - 1;
        lds_barrier();
        if (!last) return false;
        if (tid == 0) a.arrived[t.slot] = 0;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};
        constexpr int kAhead = 8;  // loads in flight
#pragma unroll 1
        for (int p = 0; p < a.parts; ++p)
            unroll<kQuads / kAhead>([&](auto g_c) {
                constexpr int g = decltype(g_c)::value * kAhead;
                u32x4 v[kAhead];
#pragma unroll
                for (int n = 0; n < kAhead; ++n) v[n] = __builtin_amdgcn_raw_buffer_load_b128(sums, at(p, g + n), 0, kAgent);
                __builtin_amdgcn_sched_barrier(0);
                unroll<kAhead>([&](auto n_c) {
                    constexpr int n = decltype(n_c)::value, quad = g + n, i = quad / 4 / NI, j = quad / 4 % NI, q = quad % 4;
                    const f32x4 f = __builtin_bit_cast(f32x4, v[n]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[i][j][4 * q + u] += f[u];
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        return true;
    };

    next_tile();
    auto copy_step = [&](int s) {
        const Copy c = begin_copy(s);
        unroll<kCopies>([&](auto i) { send(c, i); });
        end_copy();
    };
#pragma unroll
    for (int i = 0; i < RING; ++i) copy_step(i);
    wait_vm<(RING - 1) * kCopies>();
    lds_barrier();
    Tile t;
    for (int turn = 0; find(turn, t); ++turn) {
        product(t.steps);
        if (t.slot < 0 || joined(t)) finish(t);
    }
    wait_vm<0>();
}

// -------------------------------------------------------------- in and out
// The norm of each matrix: 64-bit sums of squares, `parts` of them a matrix.
template <int DT>
__device__ __forceinline__ float element(const void *p, int64_t at) {
    if constexpr (DT == kDtF32) return ((const float *)p)[at];
    else if constexpr (DT == kDtBf16) return (float)((const __bf16 *)p)[at];
    else return (float)((const _Float16 *)p)[at];
}

template <int DT>
__global__ __launch_bounds__(kThreads) void norm_kernel(const void *g, int64_t n, int parts, double *sums,
                                                        int32_t *arrived) {
    __shared__ double part[kThreads / 64];
    const int tid = threadIdx.x;
    if (blockIdx.x == 0)
        for (int i = tid; i < kCus; i += kThreads) arrived[i] = 0;
    const int64_t b = blockIdx.x / parts, p = blockIdx.x % parts;
    const int64_t per = ((n + parts - 1) / parts + 7) / 8 * 8, lo = p * per, hi = min(n, lo + per);
    const int64_t base = b * n;
    const bool wide = (uintptr_t)g % 16 == 0 && n % 8 == 0;
    double s = 0;
    if (wide) {
        for (int64_t i = lo + 8 * tid; i < hi; i += 8 * kThreads) {
            float v[8];
            load8<DT>(g, base + i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += (double)v[j] * v[j];
        }
    } else {
        for (int64_t i = lo + tid; i < hi; i += kThreads) {
            const double v = element<DT>(g, base + i);
            s += v * v;
        }
    }
    s = wave_sum_f64(s);
    if ((tid & 63) == 0) part[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) sums[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X split and scaled to 2^scale times g / 2^e, 2^e the power of two above the norm; rest: 2^e / norm.  A workgroup
// takes 64 rows by 64 columns of X; where g is tall they are read transposed, through LDS.  wide: rows of g are whole
// aligned runs of eight.  16-bit elements are fp16 numbers but for a power of two: they have no lo part, and what is
// in its place is never multiplied.
template <int DT>
__global__ __launch_bounds__(kThreads) void split_kernel(const void *g, int rows, int cols, bool tall, bool wide, int parts,
                                                         const double *sums, float eps, int scale, uint8_t *x,
                                                         int64_t x_ld, int64_t x_mat, float *rest) {
    __shared__ float tile[64][65];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t b = blockIdx.z;
    const double norm = sqrt(wave_sum_f64(lane < parts ? sums[b * parts + lane] : 0.0)) + eps;
    int e = 0;
    frexp(norm, &e);  // norm = f 2^e, f in [1/2, 1)
    const bool usual = norm > 0 && norm < INFINITY;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
        rest[b] = usual ? (float)(ldexp(1.0, e) / norm) : norm == 0 ? 1.0f : NAN;
    if (!usual) e = 0;
    const int m = tall ? cols : rows, n = tall ? rows : cols;  // of X
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int64_t base = b * rows * cols;
    constexpr int kEach = 64 * 8 / kThreads;  // runs of eight of a thread
    float v[kEach][8];
    if (wide) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r = (i * kThreads + tid) >> 3, u = tid & 7, gr = (tall ? n0 : m0) + r, gc = (tall ? m0 : n0) + 8 * u;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0;
            if (gr < rows && gc < cols) load8<DT>(g, base + (int64_t)gr * cols + gc, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = ldexpf(v[i][j], scale - e);
                if (tall) tile[8 * (tid & 7) + j][(i * kThreads + tid) >> 3] = v[i][j];
            }
    } else {
        for (int r = tid >> 6; r < 64; r += kThreads / 64) {
            // consecutive threads read consecutive elements of g
            const int gr = (tall ? n0 : m0) + r, gc = (tall ? m0 : n0) + lane;
            const float f = gr < rows && gc < cols ? ldexpf(element<DT>(g, base + (int64_t)gr * cols + gc), scale - e) : 0.0f;
            if (tall) tile[lane][r] = f;
            else tile[r][lane] = f;
        }
    }
    if (!wide || tall) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = tile[(i * kThreads + tid) >> 3][8 * (tid & 7) + j];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int row = m0 + ((i * kThreads + tid) >> 3), col = n0 + 8 * (tid & 7);
        if (row >= m || col >= (n + 31) / 32 * 32) continue;
        f16x8 h, l;
        split8(v[i], h, l);
        uint8_t *o = x + b * x_mat + row * x_ld + (col >> 5) * kChunk + (col & 31) * 2;
        *reinterpret_cast<f16x8 *>(o) = h;
        if constexpr (DT == kDtF32) *reinterpret_cast<f16x8 *>(o + 64) = l;
    }
}

template <int DT>
__device__ __forceinline__ void put(void *p, int64_t at, float v) {
    if constexpr (DT == kDtF32) ((float *)p)[at] = v;
    else if constexpr (DT == kDtBf16) ((__bf16 *)p)[at] = (__bf16)v;
    else ((_Float16 *)p)[at] = (_Float16)v;
}

// The way back.  wide: rows of out are whole aligned runs of eight.
template <int DT>
__global__ __launch_bounds__(kThreads) void join_kernel(const uint8_t *x, int64_t x_ld, int64_t x_mat, int scale,
                                                        int rows, int cols, bool tall, bool wide, void *out) {
    __shared__ float tile[64][65];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t b = blockIdx.z;
    const int m = tall ? cols : rows, n = tall ? rows : cols;
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const float back = ldexpf(1.0f, -scale);
    constexpr int kEach = 64 * 8 / kThreads;
    float v[kEach][8];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int row = m0 + ((i * kThreads + tid) >> 3), col = n0 + 8 * (tid & 7);
        f16x8 h{}, l{};
        if (row < m && col < (n + 31) / 32 * 32) {
            const uint8_t *o = x + b * x_mat + row * x_ld + (col >> 5) * kChunk + (col & 31) * 2;
            h = *reinterpret_cast<const f16x8 *>(o);
            l = *reinterpret_cast<const f16x8 *>(o + 64);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = ((float)h[j] + (float)l[j]) * back;
    }
    if (!wide || tall) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) tile[(i * kThreads + tid) >> 3][8 * (tid & 7) + j] = v[i][j];
        __syncthreads();
    }
    const int64_t base = b * rows * cols;
    if (wide) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r = (i * kThreads + tid) >> 3, u = tid & 7, gr = (tall ? n0 : m0) + r, gc = (tall ? m0 : n0) + 8 * u;
            if (tall) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = tile[8 * u + j][r];
            }
            if (gr < rows && gc < cols) store8<DT>(out, base + (int64_t)gr * cols + gc, v[i]);
        }
    } else {
        for (int r = tid >> 6; r < 64; r += kThreads / 64) {
            const int gr = (tall ? n0 : m0) + r, gc = (tall ? m0 : n0) + lane;
            if (gr < rows && gc < cols) put<DT>(out, base + (int64_t)gr * cols + gc, tall ? tile[lane][r] : tile[r][lane]);
        }
    }
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The tiles of a product: squares of `side`, which of them are whole and how the rest are cut.
struct Cut {
    int side, m_tiles, n_tiles, rounds, tail, parts;
    double cost;
    int64_t bytes() const { return parts > 1 ? (int64_t)tail * parts * side * side * 4 : 0; }
};
// The side and the number of parts that cost least by what was measured, in steps of a 128x128 tile (0.78 us): a step
// of a tile, its end (sums to hi and lo, stores, the mirrored tile), each part of one that is joined.  Of 256 x 256 a
// step costs 3.1, not 4: half the copies and LDS reads for an element.  But with few tiles CUs stay idle, and joining
// parts is slow, as one workgroup reads them all.  A symmetric product in tiles of 256 / 128: 1 x 2048 x 2048 95 / 56
// us, 8 x 1536 x 1536 130 / 109, 16 x 2048 x 2048 430 / 445; P X of 1 x 4096 x 4096 318 / 398.
Cut cut_of(int mode, int64_t batch, int rows, int cols, int steps) {
    auto of = [&](int side, double step, double end, double join) {
        Cut c;
        c.side = side;
        c.m_tiles = ceil_div(rows, side);
        c.n_tiles = ceil_div(cols, side);
        const int64_t tiles = batch * (mode == kApply ? (int64_t)c.m_tiles * c.n_tiles
                                                      : (int64_t)c.m_tiles * (c.m_tiles + 1) / 2);
        c.rounds = (int)(tiles / kCus);
        c.tail = (int)(tiles - (int64_t)c.rounds * kCus);
        c.parts = 1;
        c.cost = c.rounds * (steps * step + end);
        if (c.tail > 0) {
            auto cut = [&](int p) { return step * ceil_div(steps, p) + end + (p > 1 ? p * join : 0); };
            for (int p = 2; p <= std::min(kCus / c.tail, steps); ++p)
                if (cut(p) < cut(c.parts)) c.parts = p;
            c.cost += cut(c.parts);
        }
        return c;
    };
    const Cut big = of(256, 3.1, 12, 11), small = of(128, 1, 5, 2.7);
    return big.cost <= small.cost ? big : small;
}

template <int MODE, bool XL, bool YL>
hipError_t launch_product(GemmArgs a, hipStream_t s) {
    const Cut c = cut_of(MODE, a.batch, a.rows, a.cols, a.steps);
    a.m_tiles = c.m_tiles;
    a.n_tiles = c.n_tiles;
    a.rounds = c.rounds;
    a.tail = c.tail;
    a.parts = c.parts;
    if (c.side == 256) klaunch(split_gemm_kernel<MODE, XL, YL, 256, 256, 2, 4, 2>, dim3(kCus), dim3(512), s, a);
    else klaunch(split_gemm_kernel<MODE, XL, YL, 128, 128, 2, 2, 4>, dim3(kCus), dim3(256), s, a);
    return hipGetLastError();
}

// The buffers of a pass in the workspace.
struct Layout {
    uint8_t *x[2], *m[5];  // X and the X it becomes; A, P, Q and two more of their kind
    float *partial;
    double *sums;
    float *rest;
    int32_t *arrived;
    int64_t bytes;
    Layout(uint8_t *at, const OrthogonalSizes &z, int64_t batch) {
        const uint8_t *begin = at;
        auto take = [&](int64_t n) {
            uint8_t *p = at;
            at += (n + 255) / 256 * 256;
            return p;
        };
        for (auto &p : x) p = take(batch * z.x_mat);
        for (auto &p : m) p = take(z.gram ? batch * z.a_mat : &p < m + 2 ? batch * z.a_mat : 0);
        const int mp = ceil_div(z.m, 32), np = ceil_div(z.n, 32);
        const int64_t most = std::max({cut_of(kSym, batch, z.m, mp * 32, np).bytes(),
                                       cut_of(kSym, batch, z.m, mp * 32, mp).bytes(),
                                       cut_of(kApply, batch, z.m, np * 32, mp).bytes()});
        partial = (float *)take(most);
        sums = (double *)take(8 * batch * z.parts);
        rest = (float *)take(4 * batch);
        arrived = (int32_t *)take(4 * kCus);
        bytes = at - begin;
    }
};

}  // namespace

OrthogonalSizes orthogonal_sizes(int64_t rows, int64_t cols) {
    OrthogonalSizes z;
    z.m = (int32_t)(rows < cols ? rows : cols);
    z.n = (int32_t)(rows < cols ? cols : rows);
    z.x_ld = (int64_t)ceil_div(z.n, 32) * kChunk;
    z.a_ld = (int64_t)ceil_div(z.m, 32) * kChunk;
    z.x_mat = z.m * z.x_ld;
    z.a_mat = z.m * z.a_ld;
    // A step on A alone is three or four products of m x m x m in place of m x m x n and m x n x m.  16-bit, on X / on A:
    // 16 x 1024 x 1152 1492 / 1561 us, x 1280 1602 / 1582, x 1536 1746 / 1639, x 2048 1962 / 1710; 4 x 2048 x 2304 3008
    // / 3159, x 3584 3738 / 3428.
    z.gram = 4 * (int64_t)z.n >= 5 * (int64_t)z.m;
    const int64_t want = rows * cols / 32768;  // elements a workgroup sums
    z.parts = (int32_t)(want < 1 ? 1 : want > 64 ? 64 : want);
    return z;
}
int64_t orthogonal_bytes(const OrthogonalSizes &z, int64_t batch) { return Layout(nullptr, z, batch).bytes; }

hipError_t launch_orthogonal(int dt, const OrthogonalArgs &o, hipStream_t s) {
    const OrthogonalSizes z = orthogonal_sizes(o.rows, o.cols);
    const bool tall = o.rows > o.cols;
    const Layout w(o.work, z, o.batch);
    const dim3 block(kThreads), blocks64(ceil_div(z.n, 64), ceil_div(z.m, 64), o.batch);
    auto wide = [&](const void *p) { return o.cols % 8 == 0 && (uintptr_t)p % 16 == 0; };
    auto in = [&](auto d) {
        constexpr int DT = decltype(d)::value;
        klaunch(norm_kernel<DT>, dim3(o.batch * z.parts), block, s, o.g, (int64_t)o.rows * o.cols, (int)z.parts, w.sums,
                w.arrived);
        klaunch(split_kernel<DT>, blocks64, block, s, o.g, (int)o.rows, (int)o.cols, tall, wide(o.g), (int)z.parts,
                (const double *)w.sums, o.eps, (int)o.step[0].x, w.x[0], z.x_ld, z.x_mat, w.rest);
        return hipGetLastError();
    };
    hipError_t err = dt == kDtF32 ? in(std::integral_constant<int, kDtF32>{})
                                  : dt == kDtBf16 ? in(std::integral_constant<int, kDtBf16>{})
                                                  : in(std::integral_constant<int, kDtF16>{});
    // A split matrix and the power of two it is scaled by; of X also whether the norm's rest is still missing and
    // whether it has a lo part (16-bit input has none: it is as it was but for a power of two).
    struct Held {
        uint8_t *p;
        int scale;
    };
    bool fresh = true;
    auto args = [&](Held x, Held y, Held out) {
        GemmArgs a{};
        a.batch = o.batch;
        a.x = x.p;
        a.y = y.p;
        a.out = out.p;
        a.x_ld = a.y_ld = a.out_ld = z.a_ld;
        a.x_mat = a.y_mat = a.out_mat = z.a_mat;
        a.rows = z.m;
        a.cols = ceil_div(z.m, 32) * 32;
        a.steps = ceil_div(z.m, 32);
        a.scale = ldexpf(1.0f, out.scale - x.scale - y.scale);
        a.partial = w.partial;
        a.arrived = w.arrived;
        a.rest = w.rest;
        return a;
    };
    auto run = [&](hipError_t e) { err = err == hipSuccess ? e : err; };
    auto sym = [&](Held x, Held y, Held out) {  // out = x y of symmetric matrices that commute
        if (err == hipSuccess) run(launch_product<kSym, true, true>(args(x, y, out), s));
    };
    auto gram = [&](Held x, Held out) {  // out = x x^T
        if (err != hipSuccess) return;
        GemmArgs a = args(x, x, out);
        a.x_ld = a.y_ld = z.x_ld;
        a.x_mat = a.y_mat = z.x_mat;
        a.steps = ceil_div(z.n, 32);
        a.rest_power = fresh ? 2 : 0;
        run(fresh && dt != kDtF32 ? launch_product<kSym, false, false>(a, s) : launch_product<kSym, true, true>(a, s));
    };
    auto poly = [&](const OrthogonalStep &t, Held A, Held out) {
        if (err != hipSuccess) return;
        GemmArgs a = args(A, A, out);
        a.add = A.p;
        a.c0 = ldexpf(t.c0, out.scale);
        a.c1 = ldexpf(t.c1, out.scale - A.scale);
        a.c2 = ldexpf(t.c2, out.scale - 2 * A.scale);
        run(launch_product<kPoly, true, true>(a, s));
    };
    auto apply = [&](Held q, Held x, Held out) {  // out = q x
        if (err != hipSuccess) return;
        GemmArgs a = args(q, x, out);
        a.y_ld = a.out_ld = z.x_ld;
        a.y_mat = a.out_mat = z.x_mat;
        a.cols = ceil_div(z.n, 32) * 32;
        a.y_rows = z.m;
        a.rest_power = fresh ? 1 : 0;
        run(fresh && dt != kDtF32 ? launch_product<kApply, true, false>(a, s) : launch_product<kApply, true, true>(a, s));
        fresh = false;
    };
    int now = 0;  // which X
    for (int k = 0; k < o.steps;) {
        int end = k + 1;
        while (!o.step[end].anew) ++end;
        const Held X{w.x[now], o.step[k].x}, next{w.x[now ^ 1], o.step[end].x};
        uint8_t *A = w.m[0], *P = w.m[1], *Q = nullptr, *spare[3] = {w.m[2], w.m[3], w.m[4]};
        int q_scale = 0;
        gram(X, {A, o.step[k].a});
        for (int i = k; i < end; ++i) {
            const OrthogonalStep &t = o.step[i];
            poly(t, {A, t.a}, {P, t.p});
            if (i + 1 < end) {  // A <- P A P
                sym({P, t.p}, {A, t.a}, {spare[0], t.pa});
                sym({spare[0], t.pa}, {P, t.p}, {A, o.step[i + 1].a});
            }
            if (!Q) {  // the first P is what there is of Q
                Q = P;
                q_scale = t.p;
                P = spare[1];
            } else {
                sym({P, t.p}, {Q, q_scale}, {spare[2], t.q});
                std::swap(Q, spare[2]);
                q_scale = t.q;
            }
        }
        apply({Q, q_scale}, X, next);
        now ^= 1;
        k = end;
    }
    if (err != hipSuccess) return err;
    auto k = dt == kDtF32 ? join_kernel<kDtF32> : dt == kDtBf16 ? join_kernel<kDtBf16> : join_kernel<kDtF16>;
    klaunch(k, blocks64, block, s, (const uint8_t *)w.x[now], z.x_ld, z.x_mat, (int)o.step[o.steps].x, (int)o.rows,
            (int)o.cols, tall, wide(o.out), o.out);
    return hipGetLastError();
}

}  // namespace qrmoe
