// Products grouped by expert, and their gradients.
//
//   forward  c[p][n]  = sum_k a[r(p)][k] b[e(p)][n][k]     b: [E][N][K]
//   grad_a   da[p][k] = sum_n dc[p][n] b[e(p)][n][k]
//   grad_b   db[e][n][k] = sum over the group's rows p of dc[p][n] a[r(p)][k]
//
// All three are out[m][n] = sum over d of x(m, d) y(n, d).  An operand is
// stored either along d ("row" operand: x and y of forward, x of grad_a) or
// across it ("column" operand: y of grad_a, both of grad_b).
//
// One workgroup a CU (or two) stays for the whole call and takes tile after
// tile.  A stream of copies (global -> LDS, no registers) runs ahead of the
// arithmetic by the depth of an LDS ring, from one tile into the next: the
// first steps of a tile arrive while the tile before is stored.
//
// What bounds them on an MI355X.  Long groups: the matrix units at the clock
// the power limit leaves (8192^3 bf16: 1290 TFLOP/s, the library 1311 with the
// units 87% busy at 1.58 GHz), and how fast 64 KB a step come from the L2s
// (1.7 us a step of a 256x256 tile; 1.2 us with nothing to fetch).  Short
// groups: reading the weights (48 rows an expert, 4096 x 2048 of 256: 5.1 TB/s).
// grad_b of short groups: with three steps a tile, the copies' latency and the
// serial end of a tile (64 experts of 192 rows, 4096 x 4096, rows gathered: 865
// to 923 us by card; 772 where they are not; where it took 865, a copy of the
// kernel took 592 without fetching and 786 without storing).
//
// LDS: the operand reads meet no bank conflicts (none are counted in a kernel
// that writes fp32).  What is counted are two lanes a bank in the writes of
// 16-bit results (17 to 19% of the LDS cycles where a tile is three or four
// steps, 2% at 64) and in the reads of four-bit operands' scales (23%).
// Layouts without them made no difference in time.
#include <algorithm>
#include <type_traits>

#include "grouped.hpp"

namespace qrmoe {

constexpr int kSlab = 128;  // bytes of one row operand's row, per K step: 64 elements of 16 bits, 256 of four
constexpr int kStep = 64;   // rows of a column operand per K step
constexpr int kCus = 256, kXcds = 8;

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, class F>
__device__ __forceinline__ void unroll(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

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

    // row operand: row of copy i's piece, and the piece
    static __device__ __forceinline__ int row(int tid, int i) { return ((tid >> 6) * kLoads + i) * 8 + ((tid & 63) >> 3); }
    static __device__ __forceinline__ int piece(int tid, int r) { return (tid & 7) ^ ((r >> 1) & 7); }
    // column operand
    static constexpr int kPer = R / 8;  // pieces of one row
    static __device__ __forceinline__ int col_row(int tid, int i) {
        return ((tid >> 6) * kLoads + i) * (64 / kPer) + (tid & 63) / kPer;
    }
    static __device__ __forceinline__ int col_piece(int tid, int d) { return ((tid & 63) % kPer) ^ ((d & 3) << 2); }
    // where copy i's piece lies in the step: byte of the row, or row
    static __device__ __forceinline__ uint32_t pos(int tid, int i) {
        return COL ? col_row(tid, i) : 16 * piece(tid, row(tid, i));
    }
};

typedef __attribute__((address_space(3))) i16x4 *lds_i16x4;

// The same value, computed from anew by whoever uses it: keeps what is needed
// once a tile out of the registers that the multiplication lives on.
__device__ __forceinline__ int afresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Place in the list of tiles of turn b.  Workgroups go round the eight XCDs;
// runs of `run` consecutive tiles go to one XCD, in which group_m row tiles
// advance together through the columns.
__device__ __forceinline__ int xcd_tile(int b, int run) {
    const int i = b / kXcds;
    return (i / run * kXcds + b % kXcds) * run + i % run;
}
__device__ __forceinline__ void tile_mn(int t, int group_m, int m_tiles, int n_tiles, int &m, int &n) {
    const int g = t / (group_m * n_tiles), first = g * group_m, gm = min(group_m, m_tiles - first);
    const int r = t - g * group_m * n_tiles;
    m = first + r % gm;
    n = r / gm;
}

// A tile: its expert, first row and column, its rows (forward, grad_a: pairs;
// grad_b: of the output, row0 .. row0 + depth being its pairs) and its depth
// (0: zeros, rows of no group or an expert without pairs).
struct Tile {
    int e, row0, rows, m0, n0, depth;
};

template <Elt ELT, bool XCOL, bool YCOL, int BM, int BN, int WM, int WN, int PER_CU, bool F32>
__global__ __launch_bounds__(WM *WN * 64, (WM * WN * PER_CU + 3) / 4) void grouped_gemm_kernel(GroupedArgs a) {
    constexpr int NW = WM * WN, MI = BM / WM / 32, NI = BN / WN / 32;
    constexpr bool FP4 = ELT == Elt::Fp4;
    constexpr int XB = BM * kSlab, YB = BN * kSlab;
    // LDS ring of two steps.  (Three, which the 64x128 tile leaves room for: 48 rows an expert 966 us against 866, 161
    // rows of one expert 41 against 43.)  The scales of four-bit operands are read for the last step that the copies
    // have reached, which is the next one with two.
    constexpr int kStages = 2;
    typedef Stager<BM, NW, XCOL> SX;
    typedef Stager<BN, NW, YCOL> SY;
    typedef typename Out<ELT, F32>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    // out goes through LDS in blocks of 32 rows; of half a row each where space is short
    constexpr int kHalves = F32 && FP4 && NI > 1 ? 2 : 1;
    constexpr int kOutCols = BN / kHalves, kOutBytes = 32 * kOutCols * (int)sizeof(T);
    constexpr int kScaleBytes = FP4 ? 2 * (BM + BN) * 16 : 0;
    constexpr int kLds = 163840 / PER_CU;
    constexpr int kOutBlocks = kStages * (XB + YB) + WM * kOutBytes + kScaleBytes <= kLds ? WM : 1;  // at a time
    __shared__ __align__(1024) uint8_t smem[kStages * (XB + YB) + kOutBlocks * kOutBytes + kScaleBytes];
    uint8_t *const sout = smem + kStages * (XB + YB), *const sscale = sout + kOutBlocks * kOutBytes;

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // ---- the list of tiles
    const TileList<BM> list(a.offsets, a.E, a.P);
    const int total = XCOL ? a.E * a.m_tiles * a.n_tiles : list.total * a.n_tiles;
    const int run = a.run ? a.run : max((total + kXcds - 1) / kXcds, 1);
    auto find = [&](int turn, Tile &t) -> bool {
        const int at = xcd_tile(blockIdx.x + turn * gridDim.x, run);
        if (at >= total) {
            t = Tile{0, 0, 0, 0, 0, 0};
            return false;
        }
        int mt, nt;
        if constexpr (XCOL) {
            const int each = a.m_tiles * a.n_tiles;
            t.e = at / each;
            tile_mn(at - t.e * each, a.group_m, a.m_tiles, a.n_tiles, mt, nt);
            t.row0 = list.bound_of(t.e + 1);
            t.depth = max(list.bound_of(t.e + 2) - t.row0, 0);
            t.m0 = mt * BM;
            t.rows = min(a.M - t.m0, BM);
        } else {
            tile_mn(at, a.group_m, list.total, a.n_tiles, mt, nt);
            const RowTile r = list.find(mt);
            const bool none = r.expert < 0 || r.expert >= a.E;
            t.e = none ? 0 : r.expert;
            t.row0 = t.m0 = r.row0;
            t.rows = r.rows;
            t.depth = none ? 0 : a.depth;
        }
        t.n0 = nt * BN;
        t.e = __builtin_amdgcn_readfirstlane(t.e);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
        t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
        t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
        t.depth = __builtin_amdgcn_readfirstlane(t.depth);
        return true;
    };
    constexpr int kElems = FP4 ? 256 : kStep;  // contraction elements of one K step
    auto steps_of = [&](const Tile &t) { return (t.depth + kElems - 1) / kElems; };

    // ---- the stream of copies: tile `ct`, of which `cleft` bytes of a row (with a column operand: rows) are still to
    // be sent for, cstep steps having been; `nt` (this workgroup's turn `cturn`) is the tile after it
    SX sx;
    SY sy;
    Tile ct, nt;
    int cturn = 0, cleft = 0, cstep = 0;
    bool more = false;           // nt is a tile
    const uint8_t *cx, *cy;      // bases, advanced by one step at a time
    int64_t cx_step, cy_step;
    constexpr int kScaleRows = FP4 ? ((BM + BN) * 4 + NW * 64 - 1) / (NW * 64) : 1;  // rows this thread loads scales of
    const uint8_t *ps[kScaleRows];                                                 // null: no row
    i32x4 ws[kScaleRows];
    int nsrc[SX::kLoads], nsrc_scale[kScaleRows];  // gathered: the next tile's source rows, -1 for none
    int src[SY::kLoads];                           // grad_b, gathered: the next step's source rows

    // The tile after ct and, where rows are gathered, what its copies will read from.
    auto look_ahead = [&] {
        const int tid = afresh(threadIdx.x);
        more = false;
        while (true) {  // tiles without depth need no copies
            if (!find(++cturn, nt)) break;
            if (nt.depth > 0) {
                more = true;
                break;
            }
        }
        if constexpr (!XCOL) {
            if (a.rows && more) {
#pragma unroll
                for (int i = 0; i < SX::kLoads; ++i) {
                    const int r = SX::row(tid, i);
                    nsrc[i] = r < nt.rows ? a.rows[nt.row0 + r] : -1;
                }
                if constexpr (FP4) {
#pragma unroll
                    for (int i = 0; i < kScaleRows; ++i) {
                        const int r = (i * NW * 64 + tid) >> 2;
                        nsrc_scale[i] = r < BM && r < nt.rows ? a.rows[nt.row0 + r] : -1;
                    }
                }
            }
        }
    };
    auto load_src = [&] {  // source rows of the step at cstep of ct
        if constexpr (XCOL && YCOL) {
            if (a.rows) {
#pragma unroll
                for (int i = 0; i < SY::kLoads; ++i) {
                    const int d = SY::col_row(tid, i);
                    src[i] = d < cleft ? a.rows[ct.row0 + cstep * kStep + d] : -1;
                }
            }
        }
    };
    // The stream goes on to nt (nothing to copy if there is none).
    auto next_tile = [&] {
        const int tid = afresh(threadIdx.x);
        ct = nt;
        cstep = 0;
        cleft = !more ? 0 : XCOL || YCOL ? ct.depth : FP4 ? ct.depth / 2 : ct.depth * 2;
        if constexpr (XCOL) {
            cx = a.x + (int64_t)ct.row0 * a.x_ld + (int64_t)ct.m0 * 2;
            cx_step = kStep * a.x_ld;
#pragma unroll
            for (int i = 0; i < SX::kLoads; ++i) {
                const int d = SX::col_row(tid, i), c = SX::col_piece(tid, d);
                sx.off[i] = ct.m0 + 8 * c < a.M ? (uint32_t)(d * a.x_ld + 16 * c) : kOob;
            }
        } else {
            cx_step = kSlab;
            cx = a.rows ? a.x : a.x + (int64_t)ct.row0 * a.x_ld;
#pragma unroll
            for (int i = 0; i < SX::kLoads; ++i) {
                const int r = SX::row(tid, i);
                const int s = !a.rows ? r : nsrc[i];
                const bool ok = r < ct.rows && (!a.rows || (uint32_t)s < (uint32_t)a.src_rows);
                sx.off[i] = ok ? (uint32_t)(s * a.x_ld + SX::pos(tid, i)) : kOob;
            }
        }
        if constexpr (YCOL) {
            const bool gathered = XCOL && a.rows;  // grad_b: y is a, whose rows are the contraction
            cy = XCOL ? (gathered ? a.y : a.y + (int64_t)ct.row0 * a.y_ld) + (int64_t)ct.n0 * 2
                      : a.y + ct.e * a.y_mat + (int64_t)ct.n0 * 2;
            cy_step = gathered ? 0 : kStep * a.y_ld;
#pragma unroll
            for (int i = 0; i < SY::kLoads; ++i) {
                const int d = SY::col_row(tid, i), c = SY::col_piece(tid, d);
                sy.off[i] = ct.n0 + 8 * c < a.N ? (uint32_t)((gathered ? 0 : d * a.y_ld) + 16 * c) : kOob;
            }
        } else {
            cy = a.y + ct.e * a.y_mat + (int64_t)ct.n0 * a.y_ld;
            cy_step = kSlab;
#pragma unroll
            for (int i = 0; i < SY::kLoads; ++i) {
                const int r = SY::row(tid, i);
                sy.off[i] = ct.n0 + r < a.N ? (uint32_t)(r * a.y_ld + SY::pos(tid, i)) : kOob;
            }
        }
        if constexpr (FP4) {
            const int blocks = a.depth / 32;
#pragma unroll
            for (int i = 0; i < kScaleRows; ++i) {
                const int r = (i * NW * 64 + tid) >> 2;
                ps[i] = nullptr;
                if (r < BM) {
                    const int s = !a.rows ? (r < ct.rows ? ct.row0 + r : -1) : nsrc_scale[i];
                    if (more && s >= 0 && (!a.rows || (uint32_t)s < (uint32_t)a.src_rows))
                        ps[i] = a.xs + (int64_t)s * blocks;
                } else if (more && r < BM + BN && ct.n0 + r - BM < a.N) {
                    ps[i] = a.ys + ((int64_t)ct.e * a.N + ct.n0 + r - BM) * blocks;
                }
            }
        }
        look_ahead();
    };

    // One step's copies into ring stage stg: begin, kCopies times send, end.  The stream goes on to the next tile when a
    // tile's last step has been sent for; with four-bit operands only when the next step is, because that last step's
    // scales are still to be read.
    constexpr int kCopies = SX::kLoads + SY::kLoads;
    struct Copy {
        i32x4 rx, ry;
        uint32_t lx, ly;
    };
    const uint32_t lds0 = lds_addr(smem);
    auto begin_copy = [&](int stg) {
        if (FP4 && cleft == 0 && more) next_tile();
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + stg * (XB + YB));
        return Copy{dma_rsrc(cx), dma_rsrc(cy), base + wave * (SX::kLoads * 1024),
                    base + XB + wave * (SY::kLoads * 1024)};
    };
    auto send = [&](const Copy &c, auto idx) {
        constexpr int I = decltype(idx)::value;
        const uint32_t left = (uint32_t)cleft;
        if constexpr (I < SX::kLoads) {
            const uint32_t left_x = !XCOL && YCOL ? 2 * left : left;
            dma16_async(c.rx, c.lx + I * 1024, SX::pos(tid, I) < left_x ? sx.off[I] : kOob);
        } else {
            constexpr int i = I - SX::kLoads;
            uint32_t o = SY::pos(tid, i) < left ? sy.off[i] : kOob;
            if constexpr (XCOL && YCOL)
                if (a.rows)
                    o = o != kOob && (uint32_t)src[i] < (uint32_t)a.src_rows ? (uint32_t)(src[i] * a.y_ld + o) : kOob;
            dma16_async(c.ry, c.ly + i * 1024, o);
        }
    };
    auto end_copy = [&] {
        cx += cx_step;
        cy += cy_step;
        ++cstep;
        cleft = max(cleft - (XCOL || YCOL ? kStep : kSlab), 0);
        if (!FP4 && cleft == 0 && more) next_tile();
        load_src();
    };

    // four-bit operands: block scales.  64 bytes of each row (eight steps) are loaded at a time, 16 by each of four
    // lanes, and go to LDS a pair of steps at a time, by the lane that has it, as words [step][half]: the blocks half,
    // 2 + half, 4 + half, 6 + half that a lane's four MFMAs of a step need.  (A read
    // takes words 16 bytes apart of 32 rows: two lanes a bank.)
    auto load_scales = [&](int pair) {  // four pairs from `pair` on; zeros past the row's end and for no row
        if constexpr (FP4) {
            const int blocks = a.depth / 32, at = 16 * (pair + (tid & 3));
#pragma unroll
            for (int i = 0; i < kScaleRows; ++i) {
                ws[i] = i32x4{};
                if (!ps[i]) continue;
                if (at + 16 <= blocks) {
                    __builtin_memcpy(&ws[i], ps[i] + at, 16);
                } else {
#pragma unroll 1
                    for (int j = blocks - 1; j >= at; --j)  // shift in from the last to the first
                        ws[i] = i32x4{ws[i].x << 8 | ps[i][j], (int)__builtin_amdgcn_alignbyte(ws[i].y, ws[i].x, 3),
                                      (int)__builtin_amdgcn_alignbyte(ws[i].z, ws[i].y, 3),
                                      (int)__builtin_amdgcn_alignbyte(ws[i].w, ws[i].z, 3)};
                }
            }
        }
    };
    auto store_scales = [&](int buf, int pair) {
        if constexpr (FP4) {
            if (((tid ^ pair) & 3) != 0) return;
            i32x4 *d = reinterpret_cast<i32x4 *>(sscale + buf * (BM + BN) * 16);
#pragma unroll
            for (int i = 0; i < kScaleRows; ++i) {
                const i32x4 w = ws[i];
                const int r = (i * NW * 64 + tid) >> 2;
                if (r < BM + BN)
                    d[r] = i32x4{(int)__builtin_amdgcn_perm(w.y, w.x, 0x06040200),
                                 (int)__builtin_amdgcn_perm(w.y, w.x, 0x07050301),
                                 (int)__builtin_amdgcn_perm(w.w, w.z, 0x06040200),
                                 (int)__builtin_amdgcn_perm(w.w, w.z, 0x07050301)};
            }
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

    // ---- a tile's product
    // K steps in four groups of MFMAs (32 bytes of every row each), the operands
    // of a group being read while the group before is multiplied.  The stage of
    // a step is free once every wave has read its last group, which is before
    // the last quarter of the step's arithmetic: there the waves meet, the next
    // step (of this tile or the next) has arrived, and one more is sent for.
    // Reads and copies are spread between the MFMAs (an MFMA keeps its unit
    // busy for 32 cycles and the wave goes on issuing).
    //
    // LIVE: row blocks of 32 that a wave covers; a short tile takes fewer.
    int stg = 0, sbuf = 0;  // ring stage of the step being multiplied; scale buffer of its pair of steps
    auto product = [&](const Tile &t, auto live_c) {
        constexpr int LIVE = decltype(live_c)::value;
        constexpr int kReads = LIVE + NI, kMf = LIVE * NI;
        const int wrow = wm * LIVE * 32, wcol = wn * NI * 32;
        const int steps = steps_of(t);
        i32x4 xf[2][LIVE], yf[2][NI];
        int qx[LIVE], qy[NI];  // block scales of this step, read for the next as soon as they have served
        f32x16 acc[LIVE][NI];
#pragma unroll
        for (int i = 0; i < LIVE; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};
        auto read_one = [&](auto buf, auto idx, int s, int kk) {
            constexpr int B = decltype(buf)::value, I = decltype(idx)::value;
            const uint8_t *tx = smem + s * (XB + YB), *ty = tx + XB;
            if constexpr (I < NI)
                yf[B][I] = YCOL ? read_col(ty, BN, wcol + I * 32, kk) : read_row(ty, wcol + I * 32, kk);
            else
                xf[B][I - NI] = XCOL ? read_col(tx, BM, wrow + (I - NI) * 32, kk) : read_row(tx, wrow + (I - NI) * 32, kk);
        };
        auto read_scale = [&](auto idx, int sb, int odd) {
            constexpr int I = decltype(idx)::value;
            const uint8_t *s = sscale + sb * (BM + BN) * 16 + odd * 8 + half * 4;
            const int r = I < NI ? BM + wcol + I * 32 + l32 : wrow + (I - NI) * 32 + l32;
            const int v = *reinterpret_cast<const int *>(s + r * 16);
            if constexpr (I < NI) qy[I] = v;
            else qx[I - NI] = v;
        };
        // group kk out of buffer kk & 1; meanwhile group `next` of stage s into the other, in the step's last group the
        // next step's scales, and this wave's copies
        auto group = [&](auto kk_c, int s, int next, int sb, int odd, const Copy &c) {
            constexpr int kk = decltype(kk_c)::value, B = kk & 1;
            constexpr bool kLast = kk == 3;
            constexpr int kSend = kLast ? kCopies : 0;
            unroll<kMf>([&](auto m_c) {
                constexpr int m = decltype(m_c)::value, i = m / NI, j = m % NI;
                acc[i][j] = mfma32<ELT, kk>(yf[B][j], xf[B][i], acc[i][j], FP4 ? qy[j] : 0, FP4 ? qx[i] : 0);
                unroll<(m + 1) * kReads / kMf - m * kReads / kMf>([&](auto r_c) {
                    constexpr std::integral_constant<int, m * kReads / kMf + decltype(r_c)::value> idx{};
                    read_one(std::integral_constant<int, B ^ 1>{}, idx, s, next);
                });
                if constexpr (FP4 && kLast) {
                    if constexpr (j == NI - 1) read_scale(std::integral_constant<int, NI + i>{}, sb, odd);
                    if constexpr (i == LIVE - 1) read_scale(std::integral_constant<int, j>{}, sb, odd);
                }
                unroll<(m + 1) * kSend / kMf - m * kSend / kMf>([&](auto c_c) {
                    send(c, std::integral_constant<int, m * kSend / kMf + decltype(c_c)::value>{});
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        constexpr std::integral_constant<int, 0> c0{};
        constexpr std::integral_constant<int, 1> c1{};
        constexpr std::integral_constant<int, 2> c2{};
        constexpr std::integral_constant<int, 3> c3{};
        if (steps > 0)
            unroll<kReads>([&](auto i) {
                read_one(c0, i, stg, 0);
                if constexpr (FP4) read_scale(i, sbuf, 0);
            });
        // (after the tile's last step the operands read ahead are not used: the next tile reads its own)
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            // the copies of the step after this one are under way: ct is its tile, cstep - 1 its place there
            const bool fresh = FP4 && ((cstep - 1) & 1) == 0;  // it begins a pair
            const int pair = (cstep - 1) >> 1;
            if (fresh && (pair & 3) == 0) load_scales(pair);
            group(c0, stg, 1, 0, 0, Copy{});
            group(c1, stg, 2, 0, 0, Copy{});
            group(c2, stg, 3, 0, 0, Copy{});
            if constexpr (FP4) {
                // keeps the compiler from moving the three groups' MFMAs past the branch, behind all their reads
#pragma unroll
                for (int i = 0; i < LIVE; ++i)
#pragma unroll
                    for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
            }
            if (fresh) store_scales(sbuf ^= 1, pair);
            wait_vm<(kStages - 2) * kCopies>();
            lds_barrier();
            const Copy c = begin_copy(stg);
            stg = stg + 1 == kStages ? 0 : stg + 1;
            group(c3, stg, 0, sbuf, (k + 1) & 1, c);
            end_copy();
        }

        // ---- out, through LDS in blocks of 32 rows, so that a wave stores
        // whole stretches of them.  Register 4 q + i of a 32x32 tile holds
        // column 8 q + 4 half + i of row l32.  Piece c (16 bytes) of row r lies
        // in slot c ^ (r & (kPieces - 1)): the pieces of a read and the 32
        // rows of an fp32 write fall on different banks; a write of 16-bit
        // results is half a piece, which puts rows 16 apart on the same ones.
        constexpr int kPer = 16 / (int)sizeof(T), kPieces = kOutCols / kPer;  // elements of a piece, pieces of a row
        constexpr int kNh = NI / kHalves;
        const int tid = afresh(threadIdx.x), lane = tid & 63, l32 = lane & 31, half = lane >> 5;
        T *out = (T *)a.out + (XCOL ? ((int64_t)t.e * a.M + t.m0) * a.out_ld : (int64_t)t.m0 * a.out_ld) + t.n0;
        unroll<LIVE * (WM / kOutBlocks) * kHalves>([&](auto part_c) {
            constexpr int part = decltype(part_c)::value, h = part % kHalves, i = part / kHalves % LIVE,
                          w0 = part / kHalves / LIVE * kOutBlocks;  // blocks i of the wave rows w0 .. w0 + kOutBlocks - 1
            if ((w0 * LIVE + i) * 32 >= t.rows) return;
            if (wm >= w0 && wm < w0 + kOutBlocks) {
#pragma unroll
                for (int j = 0; j < kNh; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = (wn * kNh + j) * 32 + 8 * q + 4 * half;
                        T4 v;
#pragma unroll
                        for (int u = 0; u < 4; ++u) v[u] = Out<ELT, F32>::cvt(acc[i][h * kNh + j][4 * q + u]);
                        const int slot = (n / kPer) ^ (l32 & (kPieces - 1));
                        *reinterpret_cast<T4 *>(sout + (((wm - w0) * 32 + l32) * kPieces + slot) * 16 +
                                                (n % kPer) * (int)sizeof(T)) = v;
                    }
            }
            lds_barrier();
#pragma unroll
            for (int s = 0; s < kOutBlocks * 32 * kPieces / (NW * 64); ++s) {
                const int p = s * NW * 64 + tid, r = p / kPieces, c = p % kPieces;
                const int m = ((w0 + r / 32) * LIVE + i) * 32 + r % 32;
                // column of piece c: pieces of a wave column's half stand together
                const int n = kHalves == 1 ? c * kPer
                                           : (c * kPer / (kNh * 32) * NI + h * kNh) * 32 + c * kPer % (kNh * 32);
                // not kept in the caches, which hold the operands
                if (m < t.rows && t.n0 + n < a.N)
                    __builtin_nontemporal_store(
                        *reinterpret_cast<const i32x4 *>(sout + (r * kPieces + (c ^ (r & (kPieces - 1)))) * 16),
                        reinterpret_cast<i32x4 *>(out + (int64_t)m * a.out_ld + n));
            }
            lds_barrier();
        });
    };

    // ---- first copies, then tile after tile
    cturn = -1;
    look_ahead();
    next_tile();
    load_src();
    auto copy_step = [&](int s) {
        const Copy c = begin_copy(s);
        unroll<kCopies>([&](auto i) { send(c, i); });
        end_copy();
    };
    if (FP4) {
        load_scales(0);
        store_scales(0, 0);
    }
    copy_step(0);
    wait_vm<0>();
    for (int s = 1; s < kStages; ++s) copy_step(s);
    lds_barrier();
    Tile t;
    for (int turn = 0; find(turn, t); ++turn) {
        const int need = XCOL ? BM : t.rows;
        if (need <= BM / MI)
            product(t, std::integral_constant<int, 1>{});
        else if (MI > 2 && need <= BM / MI * 2)
            product(t, std::integral_constant<int, MI < 2 ? MI : 2>{});
        else if (MI > 3 && need <= BM / MI * 3)
            product(t, std::integral_constant<int, MI < 3 ? MI : 3>{});
        else
            product(t, std::integral_constant<int, MI>{});
    }
    wait_vm<0>();
}

// --------------------------------------------------------------- launches
namespace {

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Row tiles of the ragged groups, at most: one part tile for each group and for the rows before and past them, and no
// more than there are rows.
inline int64_t row_tiles(const GroupedArgs &a, int bm) { return std::min<int64_t>(a.P, (int64_t)a.P / bm + a.E + 2); }

template <Elt ELT, bool XCOL, bool YCOL, int BM, int BN, int WM, int WN, int PER_CU>
hipError_t launch_tiles(GroupedArgs a, bool streaming, bool f32, hipStream_t s) {
    a.n_tiles = ceil_div(a.N, BN);
    a.m_tiles = ceil_div(a.M, BM);
    const int64_t tiles = XCOL ? (int64_t)a.E * a.m_tiles * a.n_tiles : row_tiles(a, BM) * a.n_tiles;
    if (tiles > 0x3fffffff) return hipErrorInvalidValue;
    a.group_m = streaming ? 1 : 8;
    a.run = streaming ? 0 : kCus / kXcds * PER_CU;
    const dim3 grid(kCus * PER_CU), block(WM * WN * 64);
    if (f32)
        klaunch(grouped_gemm_kernel<ELT, XCOL, YCOL, BM, BN, WM, WN, PER_CU, true>, grid, block, s, a);
    else
        klaunch(grouped_gemm_kernel<ELT, XCOL, YCOL, BM, BN, WM, WN, PER_CU, false>, grid, block, s, a);
    return hipGetLastError();
}

// Mean rows of a group up to which the weights, read for each group anew, are
// what a call waits for: tiles then follow the weights through memory, one row
// tile at a time, an eighth of the list to each XCD.  Above, the XCDs share
// the list in runs of one tile a CU, eight row tiles by a few columns, which
// share operands behind one L2 whatever the groups' sizes.  Measured, bf16,
// the first way / the second: 48 rows of 4096 x 2048 of 256 experts by 64x128
// tiles 882 / 943 us, by 256x256 862 / 956; 192 rows of 4096 x 4096 of 64 by
// 64x128 1018 / 843, by 256x256 594 / 599; eight experts of 2048 rows by
// 256x256 538 / 503.  (Whole experts to each XCD: the gradient of eight experts of
// 710 .. 4702 rows took 794 us, the XCDs being done after 215 .. 1034.)
constexpr int kStreamRows = 96, kFewRows = 16;

template <Elt ELT, bool YCOL>
hipError_t launch_ragged(const GroupedArgs &a, bool f32, hipStream_t s) {
    const bool streaming = a.P < (int64_t)kStreamRows * a.E;
    // The largest tile moves the least between L2 and LDS for its arithmetic,
    // the smallest wastes the least on short groups and fills the chip with
    // few tiles.  By 64x128 / 128x128 / 256x256 tiles, bf16, 256 experts of
    // 4096 x 2048: 16 rows 765 / 765 / 826 us, 32 rows 816 / 790 / 844, 48 rows
    // 885 / 823 / 864, 90 rows 1128 / 941 / 941; 64 experts of 4096 x 4096: 192
    // rows 843 / 681 / 596.  Between 40 rows and kStreamRows the order depends on
    // how the last round of tiles fills the chip: 24 experts of 2816 x 2048, 48
    // rows 86 / 93 / 108, 90 rows 83 / 91 / 109.  The smallest is taken there.
    // Four-bit operands stop at 128x256: with 256x256 the scales on their way
    // do not fit the registers (192 rows of 4096 x 4096 by 64x128 / 128x256 /
    // 256x256: 1144 / 874 / 1251 us; 48 rows 531 / 500 / 623), and take the
    // smallest tile for a few rows (8 / 32 tokens top-6 of 256 experts: 81 / 210
    // us against 88 / 236).
    constexpr int BM = ELT == Elt::Fp4 ? 128 : 256;
    const bool fills = row_tiles(a, BM) * ceil_div(a.N, 256) >= kCus;
    const bool few = a.P < (int64_t)kFewRows * a.E;
    if (fills && (ELT == Elt::Fp4 ? !few : !streaming))
        return launch_tiles<ELT, false, YCOL, BM, 256, 2, 4, 1>(a, streaming, f32, s);
    return launch_tiles<ELT, false, YCOL, 64, 128, 1, 4, 2>(a, streaming, f32, s);
}

}  // namespace

hipError_t launch_grouped_mm(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    // Few tiles leave CUs idle; the streaming kernel spreads a few rows' weights
    // over all of them, but reads them again for every 16 rows.  Tiles of 64x128
    // against it, 4096 x 4096 of 256 experts top-6, bf16: one token 64 / 41 us,
    // four 149 / 145, eight 249 / 259, 32 730 / 789; four-bit: one token 21 /
    // 16, two 29 / 28, 32 210 / 254.  One expert, bf16: 16 rows 39 / 19, 64 rows
    // 39 / 54.
    const int64_t tiles = row_tiles(a, 64) * ceil_div(a.N, 128);
    if (tiles <= kCus * (elt == Elt::Fp4 ? 1 : 3) && a.P <= 16 * (int64_t)a.E) return launch_grouped_vec(a, elt, f32, s);
    if (elt == Elt::Bf16) return launch_ragged<Elt::Bf16, false>(a, f32, s);
    if (elt == Elt::F16) return launch_ragged<Elt::F16, false>(a, f32, s);
    return launch_ragged<Elt::Fp4, false>(a, f32, s);
}

hipError_t launch_grouped_grad_a(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    if (elt == Elt::Bf16) return launch_ragged<Elt::Bf16, true>(a, f32, s);
    return launch_ragged<Elt::F16, true>(a, f32, s);
}

hipError_t launch_grouped_grad_b(const GroupedArgs &a, Elt elt, bool f32, hipStream_t s) {
    // 64 experts of 192 rows, 4096 x 4096, rows gathered, by 128x128 / 256x256 tiles: 1223 / 922 us.
    const bool fills = (int64_t)a.E * ceil_div(a.M, 256) * ceil_div(a.N, 256) >= kCus;
    auto go = [&](auto e) {
        constexpr Elt E = decltype(e)::value;
        return fills ? launch_tiles<E, true, true, 256, 256, 2, 4, 1>(a, false, f32, s)
                     : launch_tiles<E, true, true, 128, 128, 2, 2, 2>(a, false, f32, s);
    };
    return elt == Elt::Bf16 ? go(std::integral_constant<Elt, Elt::Bf16>{}) : go(std::integral_constant<Elt, Elt::F16>{});
}

}  // namespace qrmoe
