// Host side of the operators around the experts declared in include/moe.h
// (router, pairs' order, their sum, gradients, the update): argument checks and
// dispatch.
// Nothing is allocated and nothing synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "checks.hpp"
#include "ops.hpp"

using namespace qrmoe;

namespace {

static_assert(MOE_SCORE_SIGMOID == kSigmoid && MOE_SCORE_SOFTMAX == kSoftmax, "scores");

bool aligned(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// A dense array of n elements.
Mat array(const void *p, int64_t n, int bytes) { return Mat{p, n > 0 ? 1 : 0, n, n, bytes}; }

// Present (where it holds anything) and aligned to its elements.
int check_array(const Mat &m) {
    return m.rows > 0 && (!m.p || !aligned(m.p, m.bytes) || m.end() < m.begin()) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

// Rows of elements that need no more alignment than their own.
int check_rows(const Mat &m) {
    if (m.rows > 0 && (!m.p || !aligned(m.p, m.bytes))) return MOE_ERR_INVALID_ARG;
    if (m.stride < m.cols) return MOE_ERR_INVALID_ARG;
    if (m.stride > kMaxStride) return MOE_ERR_UNSUPPORTED;
    return m.rows > 0 && m.end() < m.begin() ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int check_pairs(int64_t tokens, int64_t top_k) {
    if (tokens < 0 || top_k < 1) return MOE_ERR_INVALID_ARG;
    return tokens > MOE_MAX_PAIRS || top_k > MOE_MAX_PAIRS || tokens * top_k > MOE_MAX_PAIRS ? MOE_ERR_TOO_MANY_TOKENS
                                                                                             : MOE_OK;
}

int check_router(const moe_router *r) {
    if (!r) return MOE_ERR_INVALID_ARG;
    if (r->n_experts < 1 || r->top_k < 1 || r->top_k > r->n_experts) return MOE_ERR_INVALID_ARG;
    if (r->score != MOE_SCORE_SIGMOID && r->score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (r->renormalize != 0 && r->renormalize != 1) return MOE_ERR_INVALID_ARG;
    if (r->n_experts > 1024 || r->top_k > kMaxTopK) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
int check_choice(const moe_router *r) {
    if (r->groups < 1 || r->n_experts % r->groups != 0 || r->keep_groups < 1 || r->keep_groups > r->groups)
        return MOE_ERR_INVALID_ARG;
    if (r->group_best != 1 && r->group_best != 2) return MOE_ERR_INVALID_ARG;
    if (r->top_k > r->keep_groups * (r->n_experts / r->groups)) return MOE_ERR_INVALID_ARG;
    if (r->groups > kMaxGroups) return MOE_ERR_UNSUPPORTED;
    return check_array(array(r->bias, r->bias ? r->n_experts : 0, 4));
}

// The order's arrays, apart from each other and from `others`.
template <int N>
int check_order(const moe_pair_order *o, int64_t tokens, int64_t pairs, int32_t E, const Mat (&others)[N], PairOrder &k) {
    if (!o) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_pair_order_bytes(tokens, E);
    const Mat m[] = {array(o->perm, pairs, 8), array(o->place, pairs, 8), array(o->rows, pairs, 4),
                     array(o->offsets, E + 1, 4), array(o->workspace, (int64_t)need, 1)};
    for (const Mat &x : m) MOE_TRY(check_array(x));
    if (need > 0 && (!aligned(o->workspace, 256) || o->workspace_bytes < need)) return MOE_ERR_WORKSPACE;
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(m[i], m[j])) return MOE_ERR_INVALID_ARG;
        for (const Mat &x : others)
            if (overlap(m[i], x)) return MOE_ERR_INVALID_ARG;
    }
    k.perm = o->perm;
    k.place = o->place;
    k.rows = o->rows;
    k.offsets = o->offsets;
    k.hist = (int32_t *)o->workspace;
    return MOE_OK;
}

int32_t order_chunks(int64_t tokens) {
    const int64_t c = order_chunk(tokens), n = (tokens + c - 1) / c;
    return (int32_t)(n < 1 ? 1 : n);
}

RouteArgs route_args(const moe_router *r, const void *logits, int64_t stride, int64_t tokens) {
    RouteArgs a{};
    a.logits = logits;
    a.ld = stride;
    a.T = (int32_t)tokens;
    a.E = r->n_experts;
    a.k = r->top_k;
    a.score = r->score;
    a.renorm = r->renormalize;
    a.scale = r->scale;
    return a;
}

// The combined rows' types: the pairs' own or fp32, of fp32 pairs any.
bool bad_out(int dt, int out) { return !known_dtype(dt) || !known_dtype(out) || (out != dt && out != MOE_DT_F32 && dt != MOE_DT_F32); }

int check_cols(int64_t cols) {
    if (cols < 1) return MOE_ERR_INVALID_ARG;
    return cols % 8 != 0 || cols > kMaxFeatures ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Matrices that one pass of the orthogonalised update takes: as many as fit 4 GiB of workspace (several rounds of
// tiles for 256 CUs at any size), one at least.
constexpr int64_t kOrthogonalBytes = (int64_t)4 << 30;
int64_t orthogonal_pass(const OrthogonalSizes &z, int64_t batch) {
    const int64_t each = 2 * z.x_mat + (z.gram ? 5 : 2) * z.a_mat;
    return std::max<int64_t>(1, std::min({batch, kOrthogonalBytes / each, (int64_t)65535}));
}

// The largest |c0 s + c1 s^3 + c2 s^5| (odd) or |c0 + c1 l + c2 l^2| over s in [0, u], l = s^2: at the ends or where
// the derivative is 0.
double largest(const float *c, double u, bool odd) {
    auto at = [&](double l) { return std::fabs(c[0] + c[1] * l + c[2] * l * l) * (odd ? std::sqrt(l) : 1.0); };
    // odd: c0 + 3 c1 l + 5 c2 l^2 = 0; even: c1 + 2 c2 l = 0
    double most = std::max(at(0), at(u * u));
    auto look = [&](double l) {
        if (l > 0 && l < u * u) most = std::max(most, at(l));
    };
    if (!odd) {
        if (c[2] != 0) look(-c[1] / (2.0 * c[2]));
    } else {
        const double A = 5.0 * c[2], B = 3.0 * c[1], C = c[0], D = B * B - 4 * A * C;
        if (A == 0) {
            if (B != 0) look(-C / B);
        } else if (D >= 0) {
            look((-B + std::sqrt(D)) / (2 * A));
            look((-B - std::sqrt(D)) / (2 * A));
        }
    }
    return most;
}
// The power of two that takes values of at most `most` to 2^14 .. 2^15, half of what fp16 holds.
int32_t scale_of(double most) { return most > 0 ? std::min(15, (int)std::floor(std::log2(32768.0 / most))) : 15; }

// Scales of every step from the largest singular values that can come up; past 64 the steps do not converge.  A P A is
// A of the step after, and P A has singular values of at most the two steps' X multiplied.
//
// Where a step on A alone is cheaper than one on X (gram), several are taken so, their P multiplied with each other,
// before X is formed anew.  But A holds squares: what its 22 bits lose of singular values that are still small beside
// the largest grows by P^2 a step, and is c1 / c0 of P's own value there.  A run ends before that passes an eighth of
// the result's rounding: with the quintic after three steps for 16-bit results, after one for fp32.  Norm of the error
// that runs of 1 / 3 / 5 add to the quintic's five steps: normal matrices 3e-6 / 1.2e-5 / 5.6e-5, one singular value of
// 1 and 511 of 1e-4 4e-5 / 4e-5 / 9e-3 (the rounding of bf16: 1.7e-3, of fp16: 2e-4).  16 x 4096 x 2048 bf16: 11.9 /
// 9.7 / 9.0 ms.
int plan_orthogonal(const float *c, int32_t steps, int32_t dtype, bool gram, OrthogonalArgs &o) {
    const double half_step = dtype == MOE_DT_F32 ? 0x1p-24 : dtype == MOE_DT_F16 ? 0x1p-11 : 0x1p-8;
    double u = 1, q = 1, lost = 0;
    for (int32_t k = 0; k < steps; ++k) {
        OrthogonalStep &t = o.step[k];
        const float *f = c + 3 * k;
        if (!std::isfinite(f[0]) || !std::isfinite(f[1]) || !std::isfinite(f[2])) return MOE_ERR_INVALID_ARG;
        const double p = largest(f, u, false), next = largest(f, u, true) * 1.001;  // fp32's rounding is far below that
        const bool anew = k == 0 || !gram || f[0] == 0 ||
                          !(lost * std::fabs(f[1]) <= half_step / 8 * std::fabs(f[0]));
        q = anew ? p : q * p;
        lost = (anew ? 0x1p-22 : lost) * p * p;
        t = OrthogonalStep{f[0], f[1], f[2], scale_of(u), scale_of(u * u), scale_of(p), scale_of(u * next), scale_of(q), anew};
        u = next;
        if (!(u <= 64)) return MOE_ERR_INVALID_ARG;
    }
    o.step[steps] = OrthogonalStep{0, 0, 0, scale_of(u), 0, 0, 0, 0, true};
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_orthogonalize_bytes(int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 1 || rows < 1 || cols < 1 || std::max(rows, cols) > kMaxFeatures || std::min(rows, cols) > kMaxOrthogonal)
        return 0;
    const OrthogonalSizes z = orthogonal_sizes(rows, cols);
    // a last, smaller pass may cut its tiles into more parts
    const int64_t pass = orthogonal_pass(z, batch), left = batch % pass;
    return (size_t)std::max(orthogonal_bytes(z, pass), left ? orthogonal_bytes(z, left) : 0);
}

int moe_orthogonalize(int32_t dtype, const void *g, int64_t batch, int64_t rows, int64_t cols, int32_t steps,
                      const float *coefficients, float eps, void *out, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (!known_dtype(dtype) || batch < 0 || rows < 1 || cols < 1 || steps < 1 || !coefficients) return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (std::max(rows, cols) > kMaxFeatures || std::min(rows, cols) > kMaxOrthogonal || steps > kMaxOrthogonalSteps)
        return MOE_ERR_UNSUPPORTED;
    const int bytes = dt_bytes(dtype);
    if (batch > INT64_MAX / (rows * cols * bytes)) return MOE_ERR_INVALID_ARG;
    const Mat mg = array(g, batch * rows * cols, bytes), mo = array(out, batch * rows * cols, bytes);
    MOE_TRY(check_array(mg));
    MOE_TRY(check_array(mo));
    OrthogonalArgs o{};
    const OrthogonalSizes z = orthogonal_sizes(rows, cols);
    MOE_TRY(plan_orthogonal(coefficients, steps, dtype, z.gram, o));
    if (g != out && overlap(mo, mg)) return MOE_ERR_INVALID_ARG;
    if (batch == 0) return MOE_OK;
    const size_t need = moe_orthogonalize_bytes(batch, rows, cols);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    const Mat mw = array(workspace, (int64_t)need, 1);
    MOE_TRY(check_array(mw));
    if (overlap(mw, mg) || overlap(mw, mo)) return MOE_ERR_INVALID_ARG;
    const int64_t pass = orthogonal_pass(z, batch);
    o.work = (uint8_t *)workspace;
    o.rows = (int32_t)rows;
    o.cols = (int32_t)cols;
    o.steps = steps;
    o.eps = eps;
    for (int64_t b = 0; b < batch; b += pass) {
        o.g = (const uint8_t *)g + b * rows * cols * bytes;
        o.out = (uint8_t *)out + b * rows * cols * bytes;
        o.batch = (int32_t)std::min(pass, batch - b);
        MOE_TRY(status_of(launch_orthogonal(dtype, o, (hipStream_t)stream)));
    }
    return MOE_OK;
}

size_t moe_pair_order_bytes(int64_t tokens, int32_t n_experts) {
    if (tokens < 0 || tokens > MOE_MAX_PAIRS || n_experts < 1 || n_experts > 1024) return 0;
    const int32_t chunks = order_chunks(tokens);
    return chunks > 1 ? (size_t)(chunks + 1) * (n_experts + 1) * 4 : 0;
}

int moe_route(const moe_router *r, int32_t dtype, const void *logits, int64_t stride, int64_t tokens, int32_t *ids,
              float *w, const moe_pair_order *order, void *stream) {
    MOE_TRY(check_router(r));
    MOE_TRY(check_choice(r));
    MOE_TRY(check_pairs(tokens, r->top_k));
    if (!known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t pairs = tokens * r->top_k;
    const Mat m[] = {{logits, tokens, r->n_experts, stride, dt_bytes(dtype)}, array(r->bias, r->bias ? r->n_experts : 0, 4),
                     array(ids, pairs, 4), array(w, pairs, 4)};
    MOE_TRY(check_rows(m[0]));
    MOE_TRY(check_array(m[2]));
    MOE_TRY(check_array(m[3]));
    for (int i = 0; i < 2; ++i)
        if (overlap(m[2], m[i]) || overlap(m[3], m[i])) return MOE_ERR_INVALID_ARG;
    if (overlap(m[2], m[3])) return MOE_ERR_INVALID_ARG;
    RouteArgs a = route_args(r, logits, stride, tokens);
    if (order) MOE_TRY(check_order(order, tokens, pairs, r->n_experts, m, a.o));
    a.o.chunk = order_chunk(tokens);
    a.o.chunks = order_chunks(tokens);
    // the kernel addresses the rows of a chunk with 31-bit offsets
    if (std::min<int64_t>(a.o.chunk, tokens) * stride > 0x7fffffff / dt_bytes(dtype)) return MOE_ERR_UNSUPPORTED;
    if (tokens == 0)  // no pairs: the offsets are zeros
        return order ? status_of(launch_sort_pairs(ids, false, 0, r->top_k, r->n_experts, a.o, (hipStream_t)stream))
                     : MOE_OK;
    a.bias = r->bias;
    a.groups = r->groups;
    a.keep = r->keep_groups;
    a.best = r->group_best;
    a.ids = ids;
    a.w = w;
    return status_of(launch_route(dtype, a, (hipStream_t)stream));
}

int moe_route_grad(const moe_router *r, int32_t dtype, const void *logits, int64_t stride, int64_t tokens,
                   const int32_t *ids, const float *dw, void *dlogits, int64_t d_stride, void *stream) {
    MOE_TRY(check_router(r));
    MOE_TRY(check_pairs(tokens, r->top_k));
    if (!known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t pairs = tokens * r->top_k;
    const int bytes = dt_bytes(dtype);
    const Mat ml{logits, tokens, r->n_experts, stride, bytes}, md{dlogits, tokens, r->n_experts, d_stride, bytes},
        mi = array(ids, pairs, 4), mw = array(dw, pairs, 4);
    MOE_TRY(check_rows(ml));
    MOE_TRY(check_rows(md));
    MOE_TRY(check_array(mi));
    MOE_TRY(check_array(mw));
    if (overlap(md, ml) || overlap(md, mi) || overlap(md, mw)) return MOE_ERR_INVALID_ARG;
    if (tokens == 0) return MOE_OK;
    RouteArgs a = route_args(r, logits, stride, tokens);
    a.ids = const_cast<int32_t *>(ids);
    a.dw = dw;
    a.dlogits = dlogits;
    a.d_ld = d_stride;
    return status_of(launch_route_grad(dtype, a, (hipStream_t)stream));
}

int moe_sort_pairs(const void *ids, int32_t id_bytes, int64_t tokens, int64_t top_k, int32_t n_experts,
                   const moe_pair_order *order, void *stream) {
    MOE_TRY(check_pairs(tokens, top_k));
    if (n_experts < 1 || (id_bytes != 4 && id_bytes != 8)) return MOE_ERR_INVALID_ARG;
    if (n_experts > 1024) return MOE_ERR_UNSUPPORTED;
    const int64_t pairs = tokens * top_k;
    const Mat m[] = {array(ids, pairs, id_bytes)};
    MOE_TRY(check_array(m[0]));
    PairOrder o{};
    MOE_TRY(check_order(order, tokens, pairs, n_experts, m, o));
    o.chunk = order_chunk(tokens);
    o.chunks = order_chunks(tokens);
    return status_of(
        launch_sort_pairs(ids, id_bytes == 8, tokens, (int32_t)top_k, n_experts, o, (hipStream_t)stream));
}

int moe_combine(int32_t dtype, const void *y, int64_t y_stride, int64_t pairs, const int64_t *place, const float *w,
                int64_t tokens, int64_t top_k, int64_t cols, void *out, int32_t out_dtype, int64_t out_stride,
                void *stream) {
    MOE_TRY(check_pairs(tokens, top_k));
    MOE_TRY(check_cols(cols));
    if (bad_out(dtype, out_dtype) || pairs < 0) return MOE_ERR_INVALID_ARG;
    if (pairs > MOE_MAX_PAIRS) return MOE_ERR_TOO_MANY_TOKENS;
    const int64_t n = tokens * top_k;
    const Mat my{y, pairs, cols, y_stride, dt_bytes(dtype)}, mo{out, tokens, cols, out_stride, dt_bytes(out_dtype)},
        mp = array(place, n, 8), mw = array(w, w ? n : 0, 4);
    MOE_TRY(check_mat(my));
    MOE_TRY(check_mat(mo));
    MOE_TRY(check_array(mp));
    MOE_TRY(check_array(mw));
    if (overlap(mo, my) || overlap(mo, mp) || overlap(mo, mw)) return MOE_ERR_INVALID_ARG;
    if (tokens == 0) return MOE_OK;
    CombineArgs a{};
    a.y = y;
    a.place = place;
    a.w = w;
    a.out = out;
    a.y_ld = y_stride;
    a.out_ld = out_stride;
    a.T = tokens;
    a.P = pairs;
    a.H = cols;
    a.k = (int32_t)top_k;
    return status_of(launch_combine_pairs(dtype, out_dtype, a, (hipStream_t)stream));
}

int moe_combine_grad(int32_t dtype, const void *dout, int32_t dout_dtype, int64_t dout_stride, const void *y,
                     int64_t y_stride, int64_t pairs, const int64_t *place, const float *w, int64_t tokens,
                     int64_t top_k, int64_t cols, void *dy, int64_t dy_stride, float *dw, void *stream) {
    MOE_TRY(check_pairs(tokens, top_k));
    MOE_TRY(check_cols(cols));
    if (!known_dtype(dtype) || (dout_dtype != dtype && dout_dtype != MOE_DT_F32) || pairs < 0) return MOE_ERR_INVALID_ARG;
    if (pairs > MOE_MAX_PAIRS) return MOE_ERR_TOO_MANY_TOKENS;
    const int64_t n = tokens * top_k;
    const int bytes = dt_bytes(dtype);
    const Mat md{dout, tokens, cols, dout_stride, dt_bytes(dout_dtype)}, my{y, dw ? pairs : 0, cols, dw ? y_stride : cols, bytes},
        mp = array(place, n, 8), mw = array(w, w ? n : 0, 4), mdy{dy, dy ? pairs : 0, cols, dy ? dy_stride : cols, bytes},
        mdw = array(dw, dw ? n : 0, 4);
    for (const Mat &x : {md, my, mdy}) MOE_TRY(check_mat(x));
    for (const Mat &x : {mp, mw, mdw}) MOE_TRY(check_array(x));
    for (const Mat &x : {md, my, mp, mw})
        if (overlap(mdy, x) || overlap(mdw, x)) return MOE_ERR_INVALID_ARG;
    if (overlap(mdy, mdw)) return MOE_ERR_INVALID_ARG;
    if (tokens == 0 || (!dy && !dw)) return MOE_OK;
    CombineArgs a{};
    a.dout = dout;
    a.y = y;
    a.place = place;
    a.w = w;
    a.dy = dy;
    a.dw = dw;
    a.out_ld = dout_stride;
    a.y_ld = y_stride;
    a.dy_ld = dy_stride;
    a.T = tokens;
    a.P = pairs;
    a.H = cols;
    a.k = (int32_t)top_k;
    return status_of(launch_combine_grad(dtype, dout_dtype, a, (hipStream_t)stream));
}

}  // extern "C"
