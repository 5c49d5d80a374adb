// Host side of the expert operators declared in include/moe.h (grouped
// products and gradients, the four-bit format, SwiGLU): argument checks and
// dispatch.  Nothing is allocated and nothing synchronises.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "checks.hpp"

using namespace qrmoe;

namespace {

static_assert(MOE_DT_F32 == kDtF32 && MOE_DT_BF16 == kDtBf16 && MOE_DT_F16 == kDtF16, "element types");

// The part of the checks the grouped calls share.
int check_group(const moe_grouped *g, int feature_step) {
    if (!g) return MOE_ERR_INVALID_ARG;
    if (g->n_experts < 1 || g->pairs < 0 || g->out_features < 1 || g->in_features < 1) return MOE_ERR_INVALID_ARG;
    if (g->n_experts > 1024) return MOE_ERR_UNSUPPORTED;
    if (g->out_features > kMaxFeatures || g->in_features > kMaxFeatures || g->out_features % 8 != 0 ||
        g->in_features % feature_step != 0)
        return MOE_ERR_UNSUPPORTED;
    if (g->pairs > MOE_MAX_PAIRS) return MOE_ERR_TOO_MANY_TOKENS;
    if (!g->offsets || ((uintptr_t)g->offsets & 3)) return MOE_ERR_INVALID_ARG;
    if (g->rows && (((uintptr_t)g->rows & 3) || g->src_rows < 0)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Rows of the operand that `rows` gathers (a): as many as it has, or one for each pair.
int64_t a_rows(const moe_grouped *g) { return g->rows ? g->src_rows : g->pairs; }

// The kernels address a gathered operand with 31-bit offsets.
bool gather_too_long(const moe_grouped *g, int64_t stride_bytes) {
    return g->rows && g->src_rows >= ((int64_t)0x7fffffff + stride_bytes - 1) / stride_bytes;
}

GroupedArgs base_args(const moe_grouped *g) {
    GroupedArgs a{};
    a.offsets = g->offsets;
    a.rows = g->rows;
    a.E = g->n_experts;
    a.P = (int32_t)g->pairs;
    a.src_rows = g->rows ? (int32_t)(g->src_rows > 0x7fffffff ? 0x7fffffff : g->src_rows) : 0;
    return a;
}

Elt elt_of(int dt) { return dt == MOE_DT_BF16 ? Elt::Bf16 : Elt::F16; }

// out_dtype: the operands' type or fp32
bool bad_types(int dt, int out_dt) {
    return (dt != MOE_DT_BF16 && dt != MOE_DT_F16) || (out_dt != dt && out_dt != MOE_DT_F32);
}

int check_elementwise(int dt, int64_t rows, int64_t cols, int step) {
    if (!known_dtype(dt) || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
    if (cols % step != 0 || cols > kMaxStride) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_mm(const moe_grouped *g, int32_t dtype, const void *a, int64_t a_stride, const void *b, void *c,
                   int32_t c_dtype, int64_t c_stride, void *stream) {
    MOE_TRY(check_group(g, 8));
    if (bad_types(dtype, c_dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t N = g->out_features, K = g->in_features;
    const Mat ma{a, a_rows(g), K, a_stride, 2}, mb{b, g->n_experts * N, K, K, 2},
        mc{c, g->pairs, N, c_stride, dt_bytes(c_dtype)};
    MOE_TRY(check_mat(ma));
    MOE_TRY(check_mat(mb));
    MOE_TRY(check_mat(mc));
    if (gather_too_long(g, a_stride * 2)) return MOE_ERR_UNSUPPORTED;
    if (overlap(mc, ma) || overlap(mc, mb)) return MOE_ERR_INVALID_ARG;
    if (g->pairs == 0) return MOE_OK;
    GroupedArgs k = base_args(g);
    k.x = (const uint8_t *)a;
    k.x_ld = a_stride * 2;
    k.y = (const uint8_t *)b;
    k.y_ld = K * 2;
    k.y_mat = N * K * 2;
    k.N = (int32_t)N;
    k.depth = (int32_t)K;
    k.out = c;
    k.out_ld = c_stride;
    return status_of(launch_grouped_mm(k, elt_of(dtype), c_dtype == MOE_DT_F32, (hipStream_t)stream));
}

int moe_grouped_mm_grad_a(const moe_grouped *g, int32_t dtype, const void *dc, int64_t dc_stride, const void *b,
                          void *da, int32_t da_dtype, int64_t da_stride, void *stream) {
    MOE_TRY(check_group(g, 8));
    if (bad_types(dtype, da_dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t N = g->out_features, K = g->in_features;
    const Mat md{dc, g->pairs, N, dc_stride, 2}, mb{b, g->n_experts * N, K, K, 2},
        ma{da, g->pairs, K, da_stride, dt_bytes(da_dtype)};
    MOE_TRY(check_mat(md));
    MOE_TRY(check_mat(mb));
    MOE_TRY(check_mat(ma));
    if (overlap(ma, md) || overlap(ma, mb)) return MOE_ERR_INVALID_ARG;
    if (g->pairs == 0) return MOE_OK;
    GroupedArgs k = base_args(g);
    k.rows = nullptr;  // one gradient row for each pair: a caller adds the pairs of a gathered row
    k.x = (const uint8_t *)dc;
    k.x_ld = dc_stride * 2;
    k.y = (const uint8_t *)b;
    k.y_ld = K * 2;
    k.y_mat = N * K * 2;
    k.N = (int32_t)K;
    k.depth = (int32_t)N;
    k.out = da;
    k.out_ld = da_stride;
    return status_of(launch_grouped_grad_a(k, elt_of(dtype), da_dtype == MOE_DT_F32, (hipStream_t)stream));
}

int moe_grouped_mm_grad_b(const moe_grouped *g, int32_t dtype, const void *dc, int64_t dc_stride, const void *a,
                          int64_t a_stride, void *db, int32_t db_dtype, void *stream) {
    MOE_TRY(check_group(g, 8));
    if (bad_types(dtype, db_dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t N = g->out_features, K = g->in_features;
    const Mat md{dc, g->pairs, N, dc_stride, 2}, ma{a, a_rows(g), K, a_stride, 2},
        mb{db, g->n_experts * N, K, K, dt_bytes(db_dtype)};
    MOE_TRY(check_mat(md));
    MOE_TRY(check_mat(ma));
    MOE_TRY(check_mat(mb));
    if (gather_too_long(g, a_stride * 2)) return MOE_ERR_UNSUPPORTED;
    if (overlap(mb, md) || overlap(mb, ma)) return MOE_ERR_INVALID_ARG;
    GroupedArgs k = base_args(g);
    k.x = (const uint8_t *)dc;
    k.x_ld = dc_stride * 2;
    k.y = (const uint8_t *)a;
    k.y_ld = a_stride * 2;
    k.M = (int32_t)N;
    k.N = (int32_t)K;
    k.out = db;
    k.out_ld = K;
    return status_of(launch_grouped_grad_b(k, elt_of(dtype), db_dtype == MOE_DT_F32, (hipStream_t)stream));
}

int moe_mxfp4_quantize(int32_t dtype, const void *x, int64_t x_stride, int64_t rows, int64_t cols, uint8_t *codes,
                       uint8_t *scales, void *stream) {
    MOE_TRY(check_elementwise(dtype, rows, cols, 32));
    const Mat mx{x, rows, cols, x_stride, dt_bytes(dtype)}, mq{codes, rows, cols / 2, cols / 2, 1},
        ms{scales, rows, cols / 32, cols / 32, 1};
    MOE_TRY(check_mat(mx));
    MOE_TRY(check_mat(mq));
    if (rows > 0 && !scales) return MOE_ERR_INVALID_ARG;
    if (overlap(mq, mx) || overlap(ms, mx) || overlap(ms, mq)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    return status_of(launch_mxfp4_quantize(dtype, x, x_stride, rows, cols, codes, scales, (hipStream_t)stream));
}

int moe_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int32_t dtype,
                         void *x, int64_t x_stride, void *stream) {
    MOE_TRY(check_elementwise(dtype, rows, cols, 32));
    const Mat mx{x, rows, cols, x_stride, dt_bytes(dtype)}, mq{codes, rows, cols / 2, cols / 2, 1},
        ms{scales, rows, cols / 32, cols / 32, 1};
    MOE_TRY(check_mat(mx));
    MOE_TRY(check_mat(mq));
    if (rows > 0 && !scales) return MOE_ERR_INVALID_ARG;
    if (overlap(mx, mq) || overlap(mx, ms)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    return status_of(launch_mxfp4_dequantize(dtype, codes, scales, rows, cols, x, x_stride, (hipStream_t)stream));
}

int moe_mxfp4_grouped_mm(const moe_grouped *g, const uint8_t *a_codes, const uint8_t *a_scales,
                         const uint8_t *b_codes, const uint8_t *b_scales, void *c, int32_t c_dtype, int64_t c_stride,
                         void *stream) {
    MOE_TRY(check_group(g, 32));
    if (c_dtype != MOE_DT_BF16 && c_dtype != MOE_DT_F32) return MOE_ERR_INVALID_ARG;
    const int64_t N = g->out_features, K = g->in_features, R = a_rows(g), B = g->n_experts * N;
    const Mat ma{a_codes, R, K / 2, K / 2, 1}, mas{a_scales, R, K / 32, K / 32, 1}, mb{b_codes, B, K / 2, K / 2, 1},
        mbs{b_scales, B, K / 32, K / 32, 1}, mc{c, g->pairs, N, c_stride, dt_bytes(c_dtype)};
    MOE_TRY(check_mat(ma));
    MOE_TRY(check_mat(mb));
    MOE_TRY(check_mat(mc));
    if ((R > 0 && !a_scales) || !b_scales) return MOE_ERR_INVALID_ARG;
    if (gather_too_long(g, K / 2)) return MOE_ERR_UNSUPPORTED;
    for (const Mat &m : {ma, mas, mb, mbs})
        if (overlap(mc, m)) return MOE_ERR_INVALID_ARG;
    if (g->pairs == 0) return MOE_OK;
    GroupedArgs k = base_args(g);
    k.x = a_codes;
    k.xs = a_scales;
    k.x_ld = K / 2;
    k.y = b_codes;
    k.ys = b_scales;
    k.y_ld = K / 2;
    k.y_mat = N * K / 2;
    k.N = (int32_t)N;
    k.depth = (int32_t)K;
    k.out = c;
    k.out_ld = c_stride;
    return status_of(launch_grouped_mm(k, Elt::Fp4, c_dtype == MOE_DT_F32, (hipStream_t)stream));
}

int moe_swiglu(int32_t dtype, const void *gu, int64_t gu_stride, int64_t rows, int64_t ffn, void *h, int64_t h_stride,
               void *stream) {
    MOE_TRY(check_elementwise(dtype, rows, ffn, 8));
    const Mat mg{gu, rows, 2 * ffn, gu_stride, dt_bytes(dtype)}, mh{h, rows, ffn, h_stride, dt_bytes(dtype)};
    MOE_TRY(check_mat(mg));
    MOE_TRY(check_mat(mh));
    if (overlap(mh, mg)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    return status_of(launch_swiglu(dtype, gu, gu_stride, rows, ffn, h, h_stride, (hipStream_t)stream));
}

int moe_swiglu_mxfp4(int32_t dtype, const void *gu, int64_t gu_stride, int64_t rows, int64_t ffn, uint8_t *codes,
                     uint8_t *scales, void *stream) {
    MOE_TRY(check_elementwise(dtype, rows, ffn, 32));
    const Mat mg{gu, rows, 2 * ffn, gu_stride, dt_bytes(dtype)}, mq{codes, rows, ffn / 2, ffn / 2, 1},
        ms{scales, rows, ffn / 32, ffn / 32, 1};
    MOE_TRY(check_mat(mg));
    MOE_TRY(check_mat(mq));
    if (rows > 0 && !scales) return MOE_ERR_INVALID_ARG;
    if (overlap(mq, mg) || overlap(ms, mg) || overlap(ms, mq)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    return status_of(launch_swiglu_mxfp4(dtype, gu, gu_stride, rows, ffn, codes, scales, (hipStream_t)stream));
}

int moe_swiglu_grad(int32_t dtype, const void *dh, int64_t dh_stride, const void *gu, int64_t gu_stride, int64_t rows,
                    int64_t ffn, void *dgu, int64_t dgu_stride, void *stream) {
    MOE_TRY(check_elementwise(dtype, rows, ffn, 8));
    const int s = dt_bytes(dtype);
    const Mat md{dh, rows, ffn, dh_stride, s}, mg{gu, rows, 2 * ffn, gu_stride, s}, mo{dgu, rows, 2 * ffn, dgu_stride, s};
    MOE_TRY(check_mat(md));
    MOE_TRY(check_mat(mg));
    MOE_TRY(check_mat(mo));
    if (overlap(mo, md) || overlap(mo, mg)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    return status_of(launch_swiglu_grad(dtype, dh, dh_stride, gu, gu_stride, rows, ffn, dgu, dgu_stride,
                                        (hipStream_t)stream));
}

}  // extern "C"
