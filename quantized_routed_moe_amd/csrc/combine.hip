// The sum of a token's pairs and its gradients.
//
//   out[t] = sum_j w[t][j] y[place[t][j]]           (w absent: ones)
//   dy[place[t][j]] = w[t][j] dout[t],   dw[t][j] = <y[place[t][j]], dout[t]>
//
// Memory-bound: every row is touched once, eight elements a lane, the rows of
// a token's pairs in flight together.  Sums are in fp32, over j in order.  A
// place outside [0, P) stands for no pair: it adds nothing and gets nothing.
//
// Measured, bf16, 8192 tokens of six pairs x 4096: the sum to bf16 95 us (470
// MB, 4.95 TB/s; to fp32 110 us, 4.9), both gradients from fp32 191 us (940
// MB, 4.9 TB/s), as a large copy.  32 tokens: 3.9 and 7.0 us, launch and the
// latency of two loads in a row (the place, then the row).
#include <algorithm>

#include "mxfp4.hpp"
#include "ops.hpp"

namespace qrmoe {

namespace {

// Threads take eight columns each: whole workgroups of one token where rows are long, several tokens where not.  Up to
// seven pairs are loaded together, more by fours, twos and ones: six of 4096 to bf16 95 us against 98, eight of 2048 78
// against 72 (the registers of eight rows cost a wave a SIMD).
template <int DT, int OUT, int K>  // K pairs a token; 0: any number
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a) {
    const int per = (int)(a.H / 8), tid = threadIdx.x;
    int64_t t;
    int c;
    if (per >= kThreads) {
        const int blocks = (per + kThreads - 1) / kThreads;
        t = blockIdx.x / blocks;
        c = (blockIdx.x % blocks) * kThreads + tid;
        if (c >= per) return;
    } else {
        const int tokens = kThreads / per;
        t = (int64_t)blockIdx.x * tokens + tid / per;
        c = tid % per;
        if (tid >= tokens * per || t >= a.T) return;
    }
    const int64_t *place = a.place + t * a.k;
    const float *w = a.w ? a.w + t * a.k : nullptr;
    float sum[8] = {};
    auto some = [&](int j0, auto n_c) {
        constexpr int N = decltype(n_c)::value;
        float y[N][8], f[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t p = place[j0 + j];
            const bool there = (uint64_t)p < (uint64_t)a.P;
            f[j] = w ? w[j0 + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = 0;
            if (there) load8<DT>(a.y, p * a.y_ld + 8 * c, y[j]);
            else f[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(f[j], y[j][i], sum[i]);
    };
    if constexpr (K > 0) {
        some(0, std::integral_constant<int, K>{});
    } else {
        int j = 0;
        for (; j + 4 <= a.k; j += 4) some(j, std::integral_constant<int, 4>{});
        if (a.k - j >= 2) {
            some(j, std::integral_constant<int, 2>{});
            j += 2;
        }
        if (j < a.k) some(j, std::integral_constant<int, 1>{});
    }
    store8<OUT>(a.out, t * a.out_ld + 8 * c, sum);
}

// One workgroup a token, which reads its row of dout once.  The pairs are loaded together, so their number is a
// constant up to eight: 8192 tokens of six pairs of 4096 195 us, by predicated fours 198, by predicated eights 209; 32
// tokens 7.0 / 8.6 / 7.8.
template <int DT, int DOUT, int K>  // K pairs a token; 0: any number
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineArgs a) {
    constexpr int N = K > 0 ? K : 4;  // pairs whose rows are loaded together
    __shared__ float part[kThreads / 64][N];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
    const int per = (int)(a.H / 8), k = K > 0 ? K : a.k;
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < k; j0 += N) {
        int64_t p[N];
        float f[N], dot[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool in = K > 0 || j0 + j < k;
            p[j] = in ? a.place[t * k + j0 + j] : -1;
            if ((uint64_t)p[j] >= (uint64_t)a.P) p[j] = -1;
            f[j] = !in ? 0.0f : a.w ? a.w[t * k + j0 + j] : 1.0f;
            dot[j] = 0;
        }
        for (int c = tid; c < per; c += threads) {
            float d[8], y[N][8];
            load8<DOUT>(a.dout, t * a.out_ld + 8 * c, d);
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (p[j] >= 0) load8<DT>(a.y, p[j] * a.y_ld + 8 * c, y[j]);
            }
            if (a.dy) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (p[j] < 0) continue;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = f[j] * d[i];
                    store8<DT>(a.dy, p[j] * a.dy_ld + 8 * c, v);
                }
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (p[j] < 0) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(y[j][i], d[i], dot[j]);
                }
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float s = group_sum<64>(dot[j]);
            if (lane == 0) part[wave][j] = s;
        }
        __syncthreads();
        if (tid < N && j0 + tid < k) {
            float s = 0;
            for (int v = 0; v < threads / 64; ++v) s += part[v][tid];
            a.dw[t * k + j0 + tid] = s;
        }
        __syncthreads();
    }
}

constexpr int64_t kMaxBlocks = (((int64_t)1 << 32) - 1) / kThreads;  // of a launch of kThreads each

// f(integral_constant k) for k of at most MOST, else f(0).
template <int MOST, class F>
hipError_t by_pairs(int k, F &&f) {
    if constexpr (MOST == 0) return f(std::integral_constant<int, 0>{});
    else return k == MOST ? f(std::integral_constant<int, MOST>{}) : by_pairs<MOST - 1>(k, f);
}

}  // namespace

hipError_t launch_combine_pairs(int dt, int out_dt, const CombineArgs &all, hipStream_t s) {
    const int per = (int)(all.H / 8);
    const int64_t wide = (per + kThreads - 1) / kThreads;  // workgroups of a token, where it fills one
    // A launch has fewer than 2^32 threads (2^20 tokens of 30736 columns would be more): tokens are taken in turns.
    const int64_t most = kMaxBlocks / wide;
    auto go = [&](auto dt_c, auto out_c) {
        return by_pairs<7>(all.k, [&](auto k_c) {
            for (int64_t t = 0; t < all.T; t += most) {
                CombineArgs a = all;
                a.T = std::min(most, all.T - t);
                a.place += t * a.k;
                if (a.w) a.w += t * a.k;
                a.out = (uint8_t *)a.out + t * a.out_ld * dt_bytes(out_dt);
                const int64_t blocks = per >= kThreads ? a.T * wide : (a.T + kThreads / per - 1) / (kThreads / per);
                klaunch(combine_kernel<decltype(dt_c)::value, decltype(out_c)::value, decltype(k_c)::value>,
                        dim3((unsigned)blocks), dim3(kThreads), s, a);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            return hipSuccess;
        });
    };
    constexpr std::integral_constant<int, kDtF32> f32{};
    constexpr std::integral_constant<int, kDtBf16> bf16{};
    constexpr std::integral_constant<int, kDtF16> f16{};
    if (dt == kDtF32) return out_dt == kDtF32 ? go(f32, f32) : out_dt == kDtBf16 ? go(f32, bf16) : go(f32, f16);
    if (dt == kDtBf16) return out_dt == kDtF32 ? go(bf16, f32) : go(bf16, bf16);
    return out_dt == kDtF32 ? go(f16, f32) : go(f16, f16);
}

hipError_t launch_combine_grad(int dt, int dout_dt, const CombineArgs &a, hipStream_t s) {
    const int64_t per = a.H / 8;
    // The whole waves that a row of eight elements a lane fills, 256 threads at most.  8192 tokens, 64 / 128 / 256 threads:
    // three pairs of 520 14.8 / 16.8 / 18.9 us, six of 1024 38.6 / 37.4 / 46.6, six of 4096 215 / 199 / 195.
    const dim3 grid((unsigned)a.T), block(per < 128 ? 64 : per < 256 ? 128 : kThreads);
    auto go = [&](auto dt_c, auto dout_c) {
        return by_pairs<8>(a.k, [&](auto k_c) {
            klaunch(combine_grad_kernel<decltype(dt_c)::value, decltype(dout_c)::value, decltype(k_c)::value>, grid, block, s,
                    a);
            return hipGetLastError();
        });
    };
    constexpr std::integral_constant<int, kDtF32> f32{};
    constexpr std::integral_constant<int, kDtBf16> bf16{};
    constexpr std::integral_constant<int, kDtF16> f16{};
    if (dt == kDtF32) return go(f32, f32);
    if (dt == kDtBf16) return dout_dt == kDtF32 ? go(bf16, f32) : go(bf16, bf16);
    return dout_dt == kDtF32 ? go(f16, f32) : go(f16, f16);
}

}  // namespace qrmoe
