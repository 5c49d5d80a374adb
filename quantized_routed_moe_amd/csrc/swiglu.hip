// SwiGLU of the stacked gate/up product and its gradient.
//
//   h  = g s(g) u,             s(g) = 1 / (1 + e^-g)
//   du = dh g s(g),            dg = dh u s(g) (1 + g (1 - s(g)))
//
// gu holds [gate | up] in each row (2 F elements), h and dh F, dgu [dg | du].
// All arithmetic is fp32, rounded once on the way out.  Memory-bound: one
// pass, eight elements a lane of each half.
#include "mxfp4.hpp"

namespace qrmoe {

// s(g) and 1 - s(g), each with a relative error of a few units of 2^-24
// whatever g is: with e = e^-|g| in [0, 1] they are 1 / (1 + e) and e / (1 + e).
//
// e = 2^n 2^f: n is the integer nearest to -|g| log2(e), f what is left, which
// fused multiply-adds form without the rounding of the product (its error
// would grow as |g| 2^-24) and with the part of log2(e) that fp32 lacks.  The
// power of n is put on last, so subnormal results come out too.  The
// reciprocal gets one Newton step.  49152 x 2048 bf16, gradient: 175 us, as
// with the bare exponential.
//
// g = -inf makes g s(g) NaN (-inf * 0), as the formula's product is.
struct Sigmoid {
    float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid_f(float g) {
    constexpr double kLog2e = 1.4426950408889634;
    constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
    const float x = fmaxf(-fabsf(g), -256.0f);  // e^-256 is 0; keeps the infinities out of what follows
    const float n = rintf(x * kHi), f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    const float e = ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    const float q = 1.0f + e, r0 = __builtin_amdgcn_rcpf(q);
    const float r = __builtin_fmaf(__builtin_fmaf(-q, r0, 1.0f), r0, r0), er = e * r;
    return g < 0 ? Sigmoid{er, r} : Sigmoid{r, er};
}

template <int DT>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const void *gu, int64_t gu_ld, int64_t rows, int64_t ffn,
                                                          void *h, int64_t h_ld) {
    const int64_t per = ffn / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per;
        const int c = 8 * (int)(i - r * per);
        float g[8], u[8], o[8];
        load8<DT>(gu, r * gu_ld + c, g);
        load8<DT>(gu, r * gu_ld + ffn + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid_f(g[j]).s * u[j];
        store8<DT>(h, r * h_ld + c, o);
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void swiglu_mxfp4_kernel(const void *gu, int64_t gu_ld, int64_t rows,
                                                                int64_t ffn, uint8_t *codes, uint8_t *scales) {
    const int64_t per = ffn / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per;
        const int c = 8 * (int)(i - r * per);
        float g[8], u[8], o[8];
        load8<DT>(gu, r * gu_ld + c, g);
        load8<DT>(gu, r * gu_ld + ffn + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid_f(g[j]).s * u[j];
        uint32_t s;
        const uint32_t q = mxfp4_quad(o, s);
        *reinterpret_cast<uint32_t *>(codes + 4 * i) = q;
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(const void *dh, int64_t dh_ld, const void *gu,
                                                               int64_t gu_ld, int64_t rows, int64_t ffn, void *dgu,
                                                               int64_t dgu_ld) {
    const int64_t per = ffn / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per;
        const int c = 8 * (int)(i - r * per);
        float d[8], g[8], u[8], dg[8], du[8];
        load8<DT>(dh, r * dh_ld + c, d);
        load8<DT>(gu, r * gu_ld + c, g);
        load8<DT>(gu, r * gu_ld + ffn + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Sigmoid s = sigmoid_f(g[j]);
            dg[j] = d[j] * u[j] * s.s * (1.0f + g[j] * s.rest);
            du[j] = d[j] * g[j] * s.s;
        }
        store8<DT>(dgu, r * dgu_ld + c, dg);
        store8<DT>(dgu, r * dgu_ld + ffn + c, du);
    }
}

namespace {
inline unsigned grid_for(int64_t n) {
    const int64_t b = (n + kThreads - 1) / kThreads;
    return (unsigned)(b < 1 ? 1 : b > (1 << 20) ? (1 << 20) : b);
}
}  // namespace

hipError_t launch_swiglu(int dt, const void *gu, int64_t gu_ld, int64_t rows, int64_t ffn, void *h, int64_t h_ld,
                         hipStream_t s) {
    auto k = dt == kDtF32 ? swiglu_kernel<kDtF32> : dt == kDtBf16 ? swiglu_kernel<kDtBf16> : swiglu_kernel<kDtF16>;
    klaunch(k, dim3(grid_for(rows * (ffn / 8))), dim3(kThreads), s, gu, gu_ld, rows, ffn, h, h_ld);
    return hipGetLastError();
}

hipError_t launch_swiglu_mxfp4(int dt, const void *gu, int64_t gu_ld, int64_t rows, int64_t ffn, uint8_t *codes,
                               uint8_t *scales, hipStream_t s) {
    auto k = dt == kDtF32 ? swiglu_mxfp4_kernel<kDtF32>
                          : dt == kDtBf16 ? swiglu_mxfp4_kernel<kDtBf16> : swiglu_mxfp4_kernel<kDtF16>;
    klaunch(k, dim3(grid_for(rows * (ffn / 8))), dim3(kThreads), s, gu, gu_ld, rows, ffn, codes, scales);
    return hipGetLastError();
}

hipError_t launch_swiglu_grad(int dt, const void *dh, int64_t dh_ld, const void *gu, int64_t gu_ld, int64_t rows,
                              int64_t ffn, void *dgu, int64_t dgu_ld, hipStream_t s) {
    auto k = dt == kDtF32 ? swiglu_grad_kernel<kDtF32>
                          : dt == kDtBf16 ? swiglu_grad_kernel<kDtBf16> : swiglu_grad_kernel<kDtF16>;
    klaunch(k, dim3(grid_for(rows * (ffn / 8))), dim3(kThreads), s, dh, dh_ld, gu, gu_ld, rows, ffn, dgu, dgu_ld);
    return hipGetLastError();
}

}  // namespace qrmoe
