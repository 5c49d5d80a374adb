// Device helpers of the four-bit format and of eight-element vector access.
#pragma once

#include <type_traits>

#include "grouped.hpp"

namespace qrmoe {

// Eight consecutive elements as fp32 (16-byte aligned; offsets in elements).
template <int DT>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&v)[8]) {
    if constexpr (DT == kDtF32) {
        const f32x4 *s = reinterpret_cast<const f32x4 *>((const float *)p + at);
        const f32x4 a = s[0], b = s[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else if constexpr (DT == kDtBf16) {
        const bf16x8 a = *reinterpret_cast<const bf16x8 *>((const __bf16 *)p + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    } else {
        const f16x8 a = *reinterpret_cast<const f16x8 *>((const _Float16 *)p + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    }
}
template <int DT>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&v)[8]) {
    if constexpr (DT == kDtF32) {
        f32x4 *d = reinterpret_cast<f32x4 *>((float *)p + at);
        d[0] = f32x4{v[0], v[1], v[2], v[3]};
        d[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else if constexpr (DT == kDtBf16) {
        bf16x8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = (__bf16)v[i];
        *reinterpret_cast<bf16x8 *>((__bf16 *)p + at) = a;
    } else {
        f16x8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = (_Float16)v[i];
        *reinterpret_cast<f16x8 *>((_Float16 *)p + at) = a;
    }
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign clear, NaN above all): its biased exponent less 2.  fp32 subnormals
// (exponent 0) and everything below 2^-125 take scale 0 = 2^-127.
__device__ __forceinline__ uint32_t mxfp4_scale(uint32_t amax) {
    const int e = (int)(amax >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 2^(s - 127) as fp32 bits; s = 0 is the subnormal 2^-127
__device__ __forceinline__ float mxfp4_scale_value(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}

// Quantises this lane's eight elements of a 32-element block that four
// neighbouring lanes (aligned) share: returns the eight codes, and the
// block's scale byte.  The conversion rounds to nearest even and saturates.
__device__ __forceinline__ uint32_t mxfp4_quad(const float (&v)[8], uint32_t &scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = group_reduce<4>(m, [](uint32_t a, uint32_t b) { return max(a, b); });
    scale = mxfp4_scale(m);
    const float d = mxfp4_scale_value(scale == 255 ? 127 : scale);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], d, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], d, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], d, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], d, 3);
    return q;
}

__device__ __forceinline__ void mxfp4_values(uint32_t q, uint32_t scale, float (&v)[8]) {
    const float d = mxfp4_scale_value(scale);
    auto two = [&](auto p, float &a, float &b) {
        const auto r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, decltype(p)::value);
        a = r[0] * d;
        b = r[1] * d;
    };
    two(std::integral_constant<int, 0>{}, v[0], v[1]);
    two(std::integral_constant<int, 1>{}, v[2], v[3]);
    two(std::integral_constant<int, 2>{}, v[4], v[5]);
    two(std::integral_constant<int, 3>{}, v[6], v[7]);
}

}  // namespace qrmoe
