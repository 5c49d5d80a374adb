// Microscaled four-bit floating point: blocks of 32 consecutive elements of a
// row, each element a sign, two exponent bits and one mantissa bit (values 0,
// .5, 1, 1.5, 2, 3, 4, 6), the block a power-of-two scale in one byte (2^(s -
// 127); 255: not a number).  Element 2 i of a row is the low nibble of byte i.
//
// Quantisation of a block: s = floor(log2(max |x|)) - 2, which puts the
// largest magnitude into [4, 8); elements are rounded to the nearest
// representable multiple of the scale, ties to the even mantissa, past 6 to
// 6.  A block that holds a NaN or an infinity gets scale 255: no finite scale
// stands for it, and its products then come out as NaN.
//
// Both directions are bound by memory: one pass, 16 bytes a lane on the wide
// side, the block maximum in registers across the lanes that share a block.
#include "grouped.hpp"
#include "mxfp4.hpp"

namespace qrmoe {

template <int DT>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const void *x, int64_t ld, int64_t rows,
                                                                  int64_t cols, uint8_t *codes, uint8_t *scales) {
    const int64_t per = cols / 8, n = rows * per;  // groups of eight elements
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per);
        float v[8];
        load8<DT>(x, r * ld + 8 * c, v);
        uint32_t s;
        const uint32_t q = mxfp4_quad(v, s);
        *reinterpret_cast<uint32_t *>(codes + 4 * i) = q;
        if ((c & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_kernel(const uint8_t *codes, const uint8_t *scales,
                                                                    int64_t rows, int64_t cols, void *x, int64_t ld) {
    const int64_t per = cols / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per);
        float v[8];
        mxfp4_values(*reinterpret_cast<const uint32_t *>(codes + 4 * i), scales[i >> 2], v);
        store8<DT>(x, r * ld + 8 * c, v);
    }
}

namespace {
inline unsigned grid_for(int64_t n) {
    const int64_t b = (n + kThreads - 1) / kThreads;
    return (unsigned)(b < 1 ? 1 : b > (1 << 20) ? (1 << 20) : b);
}
}  // namespace

hipError_t launch_mxfp4_quantize(int dt, const void *x, int64_t ld, int64_t rows, int64_t cols, uint8_t *codes,
                                 uint8_t *scales, hipStream_t s) {
    auto k = dt == kDtF32 ? mxfp4_quantize_kernel<kDtF32>
                          : dt == kDtBf16 ? mxfp4_quantize_kernel<kDtBf16> : mxfp4_quantize_kernel<kDtF16>;
    klaunch(k, dim3(grid_for(rows * (cols / 8))), dim3(kThreads), s, x, ld, rows, cols, codes, scales);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(int dt, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                                   void *x, int64_t ld, hipStream_t s) {
    auto k = dt == kDtF32 ? mxfp4_dequantize_kernel<kDtF32>
                          : dt == kDtBf16 ? mxfp4_dequantize_kernel<kDtBf16> : mxfp4_dequantize_kernel<kDtF16>;
    klaunch(k, dim3(grid_for(rows * (cols / 8))), dim3(kThreads), s, codes, scales, rows, cols, x, ld);
    return hipGetLastError();
}

}  // namespace qrmoe
