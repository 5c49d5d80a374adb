// Shared by the expert operators on 16-bit and four-bit data (grouped
// products, their gradients, the four-bit format): element types, the search
// of a group's row tile, global -> LDS copies and launchers.
//
// Rows (pairs) are grouped by expert: group e holds rows offsets[e] ..
// offsets[e+1].  The offsets live on the device, so a grid is sized by a
// bound the host knows and every workgroup finds its tile itself.  Whatever
// the offsets hold, they are clamped to [0, P] where they are read and taken
// no lower than the ones before them, so that no kernel leaves its buffers,
// no two groups share a row and the host's bound holds; rows of no group come
// out as zeros.
#pragma once

#include "common.hpp"

namespace qrmoe {

constexpr int kDtF32 = 1, kDtBf16 = 2, kDtF16 = 3;
inline int dt_bytes(int dt) { return dt == kDtF32 ? 4 : 2; }

enum class Elt { Bf16, F16, Fp4 };

struct GroupedArgs {
    const uint8_t *x, *y;      // operands; rows of x are pairs (or gathered rows)
    const uint8_t *xs, *ys;    // four-bit operands: block scales [row][depth/32]
    int64_t x_ld, y_ld;        // row strides, bytes
    int64_t y_mat;             // bytes of one expert's matrix of y
    const int32_t *offsets, *rows;
    int32_t E, P;
    int32_t src_rows;          // rows of the gathered operand
    int32_t M, N;              // output rows (per expert, grad_b only) and columns
    int32_t depth;             // contraction length, elements (not grad_b)
    void *out;
    int64_t out_ld;            // elements
    int32_t sweep;             // column tiles of one workgroup (few rows an expert)
    int32_t group_m, run;      // order of the tiles (grouped_mm.hip)
    int32_t n_tiles, m_tiles;  // column tiles; row tiles per expert (grad_b only)
};

// moe_status of a HIP result (recorded for moe_last_hip_error; api.cpp)
int status_of(hipError_t e);

hipError_t launch_grouped_vec(GroupedArgs a, Elt elt, bool f32_out, hipStream_t s);
hipError_t launch_grouped_mm(const GroupedArgs &a, Elt elt, bool f32_out, hipStream_t s);
hipError_t launch_grouped_grad_a(const GroupedArgs &a, Elt elt, bool f32_out, hipStream_t s);
hipError_t launch_grouped_grad_b(const GroupedArgs &a, Elt elt, bool f32_out, hipStream_t s);
hipError_t launch_mxfp4_quantize(int dt, const void *x, int64_t ld, int64_t rows, int64_t cols, uint8_t *codes,
                                 uint8_t *scales, hipStream_t s);
hipError_t launch_mxfp4_dequantize(int dt, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                                   void *x, int64_t ld, hipStream_t s);
hipError_t launch_swiglu(int dt, const void *gu, int64_t gu_ld, int64_t rows, int64_t ffn, void *h, int64_t h_ld,
                         hipStream_t s);
hipError_t launch_swiglu_mxfp4(int dt, const void *gu, int64_t gu_ld, int64_t rows, int64_t ffn, uint8_t *codes,
                               uint8_t *scales, hipStream_t s);
hipError_t launch_swiglu_grad(int dt, const void *dh, int64_t dh_ld, const void *gu, int64_t gu_ld, int64_t rows,
                              int64_t ffn, void *dgu, int64_t dgu_ld, hipStream_t s);

// --------------------------------------------------------- group search
// Groups are counted with the rows before the first one and past the last one
// as groups of their own: index 0 .. E + 1, expert index - 1.
__device__ __forceinline__ int wave_incl_scan(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(v, o);
        if (lane >= o) v += t;
    }
    return v;
}

struct RowTile {
    int expert;  // -1 or E: rows of no group
    int row0, rows;
};

// The row tiles of all groups in order, kept by one wave in registers (every
// wave of a workgroup keeps the same): lane l holds the bounds of (E + 2) / 64
// consecutive groups, a wave scan orders the lanes' tiles.  Up to 318 experts
// the bounds stay in registers; beyond, find() reads them again.
template <int BM>
struct TileList {
    static constexpr int kHeld = 5;
    const int32_t *off;
    int E, P, per, inc, total;
    int before;  // the largest bound of the lanes below, where some bound is less than one before it; else 0
    int held[kHeld + 1];

    static __device__ __forceinline__ int tiles(int rows) { return (rows + BM - 1) / BM; }
    __device__ __forceinline__ int read(int i) const {  // bound of group i of this lane's, 0 .. per, as it stands
        const int g = min((int)(threadIdx.x & 63) * per + i, E + 2);
        const int v = min(max(off[min(max(g - 1, 0), E)], 0), P);
        return g == 0 ? 0 : g > E + 1 ? P : v;
    }
    __device__ __forceinline__ int bound(int i) const {
        int v = before;
        for (int j = 0; j <= i; ++j) v = max(v, read(j));
        return v;
    }
    // The largest of v over the lanes below this one.
    static __device__ __forceinline__ int most_below(int v) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int t = __shfl_up(v, o);
            if (lane >= o) v = max(v, t);
        }
        const int t = __shfl_up(v, 1);
        return lane > 0 ? t : 0;
    }
    __device__ __forceinline__ TileList(const int32_t *o, int e, int p) : off(o), E(e), P(p), before(0) {
        per = (E + 2 + 63) / 64;
        int c = 0;
        bool falls = false;  // offsets that run backwards: then, and only then, the running maximum is formed
        if (per <= kHeld) {
#pragma unroll
            for (int i = 0; i <= kHeld; ++i) held[i] = read(min(i, per));
#pragma unroll
            for (int i = 0; i < kHeld; ++i) falls |= held[i + 1] < held[i];
            if (__ballot(falls)) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) held[i + 1] = max(held[i + 1], held[i]);
                before = most_below(held[kHeld]);
#pragma unroll
                for (int i = 0; i <= kHeld; ++i) held[i] = max(held[i], before);
            }
#pragma unroll
            for (int i = 0; i < kHeld; ++i) c += tiles(held[i + 1] - held[i]);
        } else {
#pragma unroll
            for (int i = 0; i <= kHeld; ++i) held[i] = 0;
            int lo = read(0);
            for (int i = 1; i <= per; ++i) {
                const int hi = read(i);
                falls |= hi < lo;
                c += tiles(max(hi - lo, 0));
                lo = max(lo, hi);
            }
            if (__ballot(falls)) {
                before = most_below(lo);
                c = 0;
                lo = bound(0);
                for (int i = 1; i <= per; ++i) {
                    const int hi = max(lo, read(i));
                    c += tiles(hi - lo);
                    lo = hi;
                }
            }
        }
        inc = wave_incl_scan(c);
        total = __builtin_amdgcn_readlane(inc, 63);
    }
    // Where group g (of 0 .. E + 2) begins.
    __device__ __forceinline__ int bound_of(int g) const {
        const int l = g / per, i = g - l * per;
        if (per > kHeld) return __builtin_amdgcn_readlane(bound(i), l);
        int v = 0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j == i) v = __builtin_amdgcn_readlane(held[j], l);
        return v;
    }
    // t < total
    __device__ __forceinline__ RowTile find(int t) const {
        const int l = __ffsll((long long)__ballot(inc > t)) - 1;
        int skip = t - (l > 0 ? __builtin_amdgcn_readlane(inc, l - 1) : 0);  // tiles of the lane's groups before it
        RowTile r{-1, 0, 0};
        bool found = false;
        auto look = [&](int i, int lo, int n) {
            const int c = tiles(n);
            if (!found && skip < c) {
                found = true;
                r = RowTile{l * per + i - 1, lo + skip * BM, min(n - skip * BM, BM)};
            }
            skip -= c;
        };
        if (per <= kHeld) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int lo = __builtin_amdgcn_readlane(held[i], l);
                look(i, lo, __builtin_amdgcn_readlane(held[i + 1], l) - lo);
            }
        } else {
            int lo = bound(0);
            for (int i = 0; i < per && !found; ++i) {
                const int hi = max(lo, read(i + 1)), first = __builtin_amdgcn_readlane(lo, l);
                look(i, first, __builtin_amdgcn_readlane(hi, l) - first);
                lo = hi;
            }
        }
        return r;
    }
};

// ------------------------------------------------ global -> LDS copies
// One buffer_load_dwordx4 ... lds: lane l's 16 bytes go to LDS byte lds + 16 l.
// Written as assembly without outputs: the compiler then adds no waits of its
// own before unrelated LDS reads, and the copies are awaited with wait_vm.
// A lane whose offset is kOob reads zeros.  (m0 holds the LDS address; the
// s_nop covers the wait states an SGPR written just before needs.)
constexpr uint32_t kOob = 0x80000000u;
constexpr int32_t kRecords = 0x7fffffff;

__device__ __forceinline__ i32x4 dma_rsrc(const uint8_t *base) {
    const uint64_t b = (uint64_t)base;
    i32x4 r;
    r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32) & 0xffff);
    r.z = kRecords;
    r.w = 0x00020000;
    return r;
}
__device__ __forceinline__ void dma16_async(i32x4 rsrc, uint32_t lds, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_ptr)p);
}

// ------------------------------------------------------------ matrix ops
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

// Four-bit operands fill the first half of the instruction's register tuple; the rest is not looked at.
__device__ __forceinline__ i32x8 fp4_operand(i32x4 v) {
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// 32x32 outer tile; 32 bytes of each row: 16 elements of 16 bits or 64 of four.
// S: which byte of the scale words holds this step's block scale.
template <Elt ELT, int S>
__device__ __forceinline__ f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
    if constexpr (ELT == Elt::Bf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else if constexpr (ELT == Elt::F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, S, sa, S, sb);
}
// 16x16 outer tile; 64 bytes of each row: 32 elements of 16 bits or 128 of four.
template <Elt ELT>
__device__ __forceinline__ f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
    if constexpr (ELT == Elt::Bf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else if constexpr (ELT == Elt::F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, 0, sa, 0, sb);
}

// Sums are held in fp32; the one rounding (to nearest even) is to the output type.
template <Elt ELT, bool F32>
struct Out;
template <Elt ELT>
struct Out<ELT, true> {
    typedef float T;
    static __device__ __forceinline__ T cvt(float v) { return v; }
};
template <Elt ELT>
struct Out<ELT, false> {
    typedef __bf16 T;
    static __device__ __forceinline__ T cvt(float v) { return (__bf16)v; }
};
template <>
struct Out<Elt::F16, false> {
    typedef _Float16 T;
    static __device__ __forceinline__ T cvt(float v) { return (_Float16)v; }
};

}  // namespace qrmoe
