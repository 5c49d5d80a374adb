// Arguments and launchers of the operators around the experts' products: the
// router and the order of its pairs, the sum of a token's pairs, the
// orthogonalised update.
#pragma once

#include "grouped.hpp"

namespace qrmoe {

constexpr int kSigmoid = 1, kSoftmax = 2;
constexpr int kMaxTopK = 8, kMaxGroups = 16;

// The order of the pairs by expert; all null where it is not asked for.
struct PairOrder {
    int64_t *perm, *place;
    int32_t *rows, *offsets;
    int32_t *hist;         // [chunks + 1][E + 1] pairs of each expert (the last: of none) in each chunk; their sums
    int32_t chunk, chunks; // tokens of a chunk, number of chunks
};

struct RouteArgs {
    const void *logits;
    int64_t ld;  // elements
    const float *bias;
    int32_t *ids;
    float *w;
    const float *dw;   // gradient only
    void *dlogits;     // gradient only
    int64_t d_ld;
    int32_t T, E, k, score, groups, keep, best, renorm;
    float scale;
    PairOrder o;
};

struct CombineArgs {
    const void *y, *dout;
    const int64_t *place;
    const float *w;  // null: ones
    void *out, *dy;
    float *dw;
    int64_t y_ld, out_ld, dy_ld;  // elements; out_ld: of out or dout
    int64_t T, P, H;
    int32_t k;
};

// One step's coefficients and the powers of two by which its split matrices are scaled.
struct OrthogonalStep {
    float c0, c1, c2;
    int32_t x, a, p, pa, q;  // of X, A, P, P A and the product of the run's P so far
    bool anew;               // X is formed before this step: a new run of steps on A begins
};
constexpr int kMaxOrthogonalSteps = 32, kMaxOrthogonal = 16384;  // steps; the shorter side
struct OrthogonalArgs {
    const void *g;
    void *out;
    uint8_t *work;
    int32_t batch, rows, cols, steps;
    float eps;
    OrthogonalStep step[kMaxOrthogonalSteps + 1];  // the last: X only
};
// X is m x n, m <= n; strides in bytes.
struct OrthogonalSizes {
    int32_t m, n, parts;
    bool gram;  // steps may be taken on A: it is enough smaller than X
    int64_t x_ld, a_ld, x_mat, a_mat;
};

// Tokens of a chunk of the pairs' order, and the chunks of T tokens.
int32_t order_chunk(int64_t tokens);
hipError_t launch_route(int dt, const RouteArgs &a, hipStream_t s);
hipError_t launch_route_grad(int dt, const RouteArgs &a, hipStream_t s);
hipError_t launch_sort_pairs(const void *ids, bool wide, int64_t tokens, int32_t k, int32_t E, const PairOrder &o,
                             hipStream_t s);
hipError_t launch_combine_pairs(int dt, int out_dt, const CombineArgs &a, hipStream_t s);
OrthogonalSizes orthogonal_sizes(int64_t rows, int64_t cols);
int64_t orthogonal_bytes(const OrthogonalSizes &z, int64_t batch);  // of the workspace of a pass
hipError_t launch_orthogonal(int dt, const OrthogonalArgs &a, hipStream_t s);
hipError_t launch_combine_grad(int dt, int dout_dt, const CombineArgs &a, hipStream_t s);

}  // namespace qrmoe
