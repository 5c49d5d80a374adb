// The router of a mixture-of-experts layer on given logits, the order of its
// pairs by expert, and its gradient.
//
//   s = sigmoid(l) or softmax(l),  key = s + bias, -inf where l = -inf
//   groups: the sum of a group's `best` largest keys; the `keep` best groups stay
//   the k largest keys, equal ones by lower index; w = s / sum of chosen s * scale
//
// The choice is that of real numbers: fp32 decides where two keys are further
// apart than it can be wrong, 64 bits where they are not.  Without a bias the
// order of the scores is that of the logits, which needs no arithmetic at all.
//
// L lanes hold a token (4, 2 or 1 tokens a wave), PER keys each: expert
// lane + L i in slot i.  A key is the order-preserving image of its fp32 value
// with the low four bits replaced by the slot (lower slots larger), so that a
// lane sorts them with plain integer minima and maxima and the largest head
// of L lanes is found by a butterfly; of equal heads, which are of one slot,
// the lowest lane has the lowest expert.
#include <cfloat>
#include <type_traits>

#include "ops.hpp"

namespace qrmoe {

namespace {

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, class F>
__device__ __forceinline__ void unroll(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t at) {
    if constexpr (DT == kDtF32) return ((const float *)p)[at];
    else if constexpr (DT == kDtBf16) return (float)((const __bf16 *)p)[at];
    else return (float)((const _Float16 *)p)[at];
}
template <int DT>
__device__ __forceinline__ void store_logit(void *p, int64_t at, float v) {
    if constexpr (DT == kDtF32) ((float *)p)[at] = v;
    else if constexpr (DT == kDtBf16) ((__bf16 *)p)[at] = (__bf16)v;
    else ((_Float16 *)p)[at] = (_Float16)v;
}

// e^x for x <= 0 (or NaN) with a relative error of a few units of 2^-24: the integer part of x log2(e) is put on as an
// exponent, what is left is formed without the rounding of the product.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr double kLog2e = 1.4426950408889634;
    constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
    x = x < -256.0f ? -256.0f : x;
    const float n = rintf(x * kHi), f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
// sigmoid, within 2^-22
__device__ __forceinline__ float sigmoid_near(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * l));
}
__device__ __forceinline__ double sigmoid_f64(double l) { return 1.0 / (1.0 + exp(-l)); }

// What the wave's lanes have written to LDS is there for the others.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a NaN key counts as: behind every number, before -inf (an expert that is not there).
template <class T>
__device__ __forceinline__ T number(T key, T least) {
    return key != key ? least : key;
}
__device__ __forceinline__ uint32_t image_of(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t image) {
    return __uint_as_float(image & 0x80000000u ? image ^ 0x80000000u : ~image);
}
constexpr uint32_t kThere = 0x00800000u;  // the image of -FLT_MAX; that of -inf is below

// v sorted, the largest first (odd-even merge network)
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t a = v[i + j], b = v[i + j + q];
                        v[i + j] = umax(a, b);
                        v[i + j + q] = umin(a, b);
                    }
}

// ------------------------------------------------- one token in 64 bits
// The whole wave decides for token t: lanes r < k get the expert of rank r
// (-1: none left).  top, z: the row's largest logit and sum of e^(l - top).
// A function of its own, so that the registers of what hardly ever runs stay out of what always does.
template <int DT, int S>  // S slots of 64 experts
__device__ __attribute__((noinline)) int choose_f64(const RouteArgs &a, int64_t t, float top, int lane) {
    const int64_t row = t * a.ld;
    const bool soft = a.score == kSoftmax, by_logit = !a.bias && a.groups == 1;
    double key[S];
    double z = 0;
    if (soft && !by_logit) {
        for (int e = lane; e < a.E; e += 64) z += exp((double)load_logit<DT>(a.logits, row + e) - (double)top);
        z = wave_sum_f64(z);
        if (z == 0) z = 1;
    }
    auto key_of = [&](int e, bool score) -> double {
        const float lf = load_logit<DT>(a.logits, row + e);
        const double l = lf, b = a.bias ? (double)a.bias[e] : 0.0;
        if (lf == -INFINITY) return -INFINITY;
        if (!score) return number(l, -DBL_MAX);
        return number((soft ? exp(l - (double)top) / z : sigmoid_f64(l)) + b, -DBL_MAX);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) {
        key[i] = -INFINITY;
        if (64 * i < a.E && lane + 64 * i < a.E) key[i] = key_of(lane + 64 * i, !by_logit);
    }
    if (a.groups > 1) {
        const int size = a.E / a.groups;
        double mine = -INFINITY;  // of group `lane`
        for (int g = 0; g < a.groups; ++g) {
            double t1 = -INFINITY, t2 = -INFINITY;
            auto add = [&](double x) {
                t2 = fmax(t2, fmin(t1, x));
                t1 = fmax(t1, x);
            };
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (64 * i < a.E && (lane + 64 * i) / size == g) add(key[i]);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
                add(o1);
                add(o2);
            }
            const double v = a.best == 2 && t2 != -INFINITY ? t1 + t2 : t1;
            if (lane == g) mine = v;
        }
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl(mine, g);
            before += o > mine || (o == mine && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && before < a.keep);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int g = (lane + 64 * i) / size;
            if (64 * i < a.E && g < a.groups) {
                if (!((kept >> g) & 1)) key[i] = -INFINITY;
                // the scores of the chosen groups rank as their logits do
                else if (!a.bias && key[i] != -INFINITY) key[i] = key_of(lane + 64 * i, false);
            }
        }
    }
    int id = -1;
    for (int r = 0; r < a.k; ++r) {
        double m = key[0];
#pragma unroll
        for (int i = 1; i < S; ++i) m = fmax(m, key[i]);
        m = group_reduce<64>(m, [](double x, double y) { return fmax(x, y); });
        if (m == -INFINITY) break;
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = S - 1; i >= 0; --i) at = key[i] == m ? (uint32_t)(lane + 64 * i) : at;
        at = group_reduce<64>(at, umin);
#pragma unroll
        for (int i = 0; i < S; ++i)
            if ((uint32_t)(lane + 64 * i) == at) key[i] = -INFINITY;
        if (lane == r) id = (int)at;
    }
    return id;
}

// -------------------------------------------------------------- pair order
// Stable counting sort.  hist holds the pairs of each expert in each chunk of
// tokens; a chunk's workgroup adds up the chunks before its own by itself,
// which costs less than another launch.
struct SortShared {
    int fill[1025], before[1025], wcnt[kRouteWaves][1025];
    int tmp[kRouteWaves];
};

// fill[b] for b <= E: how many pairs stand before those of bucket b, from total[b] (LDS; the buckets' pairs).
__device__ __forceinline__ void exclusive_scan(const int *total, int *fill, int E, int *tmp) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int v = tid < E ? total[tid] : 0;
    const int inc = wave_incl_scan(v);
    if (lane == 63) tmp[wave] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wave; ++w) base += tmp[w];
    if (tid < E) fill[tid] = base + inc - v;
    if (tid == kRouteThreads - 1) fill[E] = base + inc;
    __syncthreads();
}

// Places pairs [p0, p1) in order; sh.fill[b] is the next free place of bucket b, sh.wcnt is zero.
template <class Id>
__device__ __forceinline__ void place_pairs(const Id *ids, int64_t p0, int64_t p1, int E, int k, const PairOrder &o,
                                            SortShared &sh) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    for (int64_t base = p0; base < p1; base += kRouteThreads) {
        const int64_t p = base + tid;
        const bool valid = p < p1;
        int e = 2047;  // no bucket's
        if (valid) {
            const Id id = ids[p];
            e = id < 0 || id >= (Id)E ? E : (int)id;
        }
        uint64_t same = ~0ull;
#pragma unroll
        for (int bit = 0; bit < 11; ++bit) {
            const uint64_t b = __ballot((e >> bit) & 1);
            same &= (e >> bit) & 1 ? b : ~b;
        }
        const int rank = __popcll(same & below);
        if (valid && rank == 0) sh.wcnt[wave][e] = __popcll(same);
        __syncthreads();
        if (valid) {
            int at = sh.fill[e] + rank;
            for (int w = 0; w < wave; ++w) at += sh.wcnt[w][e];
            o.perm[at] = p;
            o.rows[at] = (int32_t)(p / k);
            o.place[p] = at;
        }
        __syncthreads();
        if (valid && rank == 0) {
            atomicAdd(&sh.fill[e], sh.wcnt[wave][e]);
            sh.wcnt[wave][e] = 0;
        }
        __syncthreads();
    }
}

template <class Id>
__global__ __launch_bounds__(kRouteThreads) void place_kernel(const Id *ids, int64_t P, int E, int k, PairOrder o) {
    __shared__ SortShared sh;
    const int tid = threadIdx.x, c = blockIdx.x, buckets = E + 1;
    for (int i = tid; i < kRouteWaves * 1025; i += kRouteThreads) (&sh.wcnt[0][0])[i] = 0;
    for (int i = tid; i < buckets; i += kRouteThreads) sh.before[i] = sh.fill[i] = 0;
    __syncthreads();
    // rows of hist shared out over as many threads as there are for each bucket
    const int width = buckets <= 128 ? 128 : buckets <= 256 ? 256 : buckets <= 512 ? 512 : 1024;
    const int parts = kRouteThreads / width, part = tid / width;
    for (int b = tid % width; b < buckets; b += width) {
        int total = 0, before = 0;
#pragma unroll 8
        for (int i = part; i < o.chunks; i += parts) {
            const int v = o.hist[(int64_t)i * buckets + b];
            total += v;
            before += i < c ? v : 0;
        }
        atomicAdd(&sh.fill[b], total);
        atomicAdd(&sh.before[b], before);
    }
    __syncthreads();
    exclusive_scan(sh.fill, sh.fill, E, sh.tmp);
    for (int i = tid; i < buckets; i += kRouteThreads) {
        if (c == 0) o.offsets[i] = sh.fill[i];
        sh.fill[i] += sh.before[i];
    }
    __syncthreads();
    const int64_t p0 = (int64_t)c * o.chunk * k, p1 = min(P, p0 + (int64_t)o.chunk * k);
    place_pairs(ids, p0, p1, E, k, o, sh);
}

// The counts of one chunk; where it is the only one, the whole order.
template <class Id>
__global__ __launch_bounds__(kRouteThreads) void count_kernel(const Id *ids, int64_t P, int E, int k, PairOrder o) {
    __shared__ SortShared sh;
    const int tid = threadIdx.x, c = blockIdx.x;
    for (int i = tid; i <= E; i += kRouteThreads) sh.fill[i] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)c * o.chunk * k, p1 = min(P, p0 + (int64_t)o.chunk * k);
    for (int64_t p = p0 + tid; p < p1; p += kRouteThreads) {
        const Id id = ids[p];
        atomicAdd(&sh.fill[id < 0 || id >= (Id)E ? E : (int)id], 1);
    }
    __syncthreads();
    if (o.chunks > 1) {
        for (int i = tid; i <= E; i += kRouteThreads) o.hist[(int64_t)c * (E + 1) + i] = sh.fill[i];
        return;
    }
    for (int i = tid; i < kRouteWaves * 1025; i += kRouteThreads) (&sh.wcnt[0][0])[i] = 0;
    exclusive_scan(sh.fill, sh.fill, E, sh.tmp);
    for (int i = tid; i <= E; i += kRouteThreads) o.offsets[i] = sh.fill[i];
    place_pairs(ids, p0, p1, E, k, o, sh);
}

// ------------------------------------------------------------------ router
template <int DT, int L, int PER, bool GROUPS>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    constexpr int TW = 64 / L, TB = TW * kRouteWaves;  // tokens of a wave, of a workgroup's pass
    // keys of a wave's tokens by expert; afterwards, in a single workgroup, the order of the pairs
    __shared__ union Shared {
        float keys[GROUPS ? kRouteWaves : 1][GROUPS ? TW * L * PER : 1];
        SortShared sort;
    } sh;
    __shared__ int hist[1025];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & (L - 1), base = lane & ~(L - 1);  // this lane among its token's; the first of them
    const int E = a.E, k = a.k;
    const bool order = a.o.perm != nullptr, soft = a.score == kSoftmax;
    if (order) {
        for (int i = tid; i <= E; i += kRouteThreads) hist[i] = 0;
        __syncthreads();
    }
    const int t_end = min(a.T, (int)(blockIdx.x + 1) * a.o.chunk);
    for (int t0 = (int)blockIdx.x * a.o.chunk + wave * TW; t0 < t_end; t0 += TB) {
        const int t = t0 + lane / L;
        const bool live = t < t_end;
        const int64_t row = (int64_t)min(t, t_end - 1) * a.ld;

        // ---- logits, scores, keys
        float l[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = j + L * i;
            const float v = load_logit<DT>(a.logits, row + min(e, E - 1));
            l[i] = e < E ? v : -INFINITY;
        }
        float top = 0, z = 1;
        if (soft) {
            top = l[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) top = fmaxf(top, l[i]);
            top = group_max<L>(top);
            if (top == -INFINITY) top = 0;
        }
        // a key's error: of the score (sigmoid_near; e^x and the sum, against the largest probability, 1 / z)
        float slack = 0x1p-21f;
        const bool scored = a.bias || GROUPS;
        if (soft && (scored || !a.renorm)) {
            float part = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) part += exp_neg(l[i] - top);
            z = group_sum<L>(part);
            if (z == 0) z = 1;
            slack = 0x1p-20f / z;
        }
        auto score_of_l = [&](float x) { return soft ? exp_neg(x - top) / z : sigmoid_near(x); };
        uint32_t v[PER];
        bool unsure = false;
        if constexpr (GROUPS) {
            float *keys = sh.keys[wave] + (lane / L) * L * PER;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = j + L * i;
                float f = score_of_l(l[i]) + (a.bias && e < E ? a.bias[e] : 0.0f);
                f = l[i] == -INFINITY ? -INFINITY : number(f, -FLT_MAX);
                keys[e] = f;
                if (a.bias) v[i] = image_of(f);
            }
            // lane g < groups: group g's score; lanes start at places of their own in it (banks)
            wave_sync();
            const int size = E / a.groups;
            float t1 = -INFINITY, t2 = -INFINITY;
            if (j < a.groups) {
                int at = j % size;
                for (int n = 0; n < size; ++n) {
                    const float x = keys[j * size + at];
                    t2 = fmaxf(t2, fminf(t1, x));
                    t1 = fmaxf(t1, x);
                    at = at + 1 == size ? 0 : at + 1;
                }
            }
            wave_sync();
            const float mine = a.best == 2 && t2 != -INFINITY ? t1 + t2 : t1;
            // what the rounding of its sum is relative to
            const float size_of = (t1 == -INFINITY ? 0.0f : fabsf(t1)) + (t2 == -INFINITY ? 0.0f : fabsf(t2));
            int before = 0;
            for (int g = 0; g < a.groups; ++g) {
                const float o = __shfl(mine, base + g);
                before += o > mine || (o == mine && g < j);
            }
            const bool in = j < a.groups && before < a.keep;
            // the least of the kept must be clearly above the largest of the others
            const float least = -group_max<L>(in ? -mine : -INFINITY);
            const float most = group_max<L>(!in && j < a.groups ? mine : -INFINITY);
            if (most != -INFINITY)
                unsure = !(least - most > 4 * slack + 0x1p-20f * group_max<L>(size_of));
            const uint32_t kept = (uint32_t)(__ballot(in) >> base) & 0xffffu;
            const uint32_t recip = ((1u << 20) + size - 1) / size;  // e / size for e < 1024
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t g = ((uint32_t)(j + L * i) * recip) >> 20;
                if (!a.bias) v[i] = image_of(number(l[i] + 0.0f, -FLT_MAX));
                v[i] = (kept >> g) & 1 ? v[i] : 0;
            }
        } else if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = j + L * i;
                const float f = score_of_l(l[i]) + a.bias[min(e, E - 1)];
                v[i] = l[i] == -INFINITY ? 0 : image_of(number(f, -FLT_MAX));
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = image_of(number(l[i] + 0.0f, -FLT_MAX));  // -0 as 0
        }

        // ---- the k largest and the one after them
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = (v[i] & ~15u) | (15 - i);
        sort_keys(v);
        uint32_t last = 0;
        int id = -1;  // lane r of the token: its expert of rank r
        unroll<kMaxTopK + 1>([&](auto rank) {
            constexpr int r = decltype(rank)::value;
            if (r > k) return;
            const uint32_t m = group_reduce<L>(v[0], umax);
            const uint64_t hits = __ballot(v[0] == m) >> base;
            const int owner = __ffsll((long long)(L == 64 ? hits : hits & ((1ull << (L & 63)) - 1))) - 1;
            // is it clearly below the one before?
            if (r > 0 && m >= kThere) {
                if (a.bias) {
                    const float hi = value_of(last & ~15u), lo = value_of(m & ~15u);
                    unsure |= !(hi - lo > 2 * slack + 0x1p-18f * fmaxf(fabsf(hi), fabsf(lo)));
                } else if (DT == kDtF32) {
                    unsure |= (last ^ m) < 16;
                }
            }
            last = m;
            if (r < k && j == r && m >= kThere) id = owner + L * (int)(15 - (m & 15));
            const bool mine = j == owner;
#pragma unroll
            for (int i = 0; i + 1 < PER && i < kMaxTopK - r; ++i) v[i] = mine ? v[i + 1] : v[i];
            if (kMaxTopK - r >= PER) v[PER - 1] = mine ? 0 : v[PER - 1];
        });
        // ---- where fp32 cannot tell, the whole wave decides in 64 bits, a token at a time
        uint64_t todo = __ballot(unsure && live && j == 0);
        while (todo) {
            const int at = __ffsll((long long)todo) - 1;
            todo &= todo - 1;
            const int r = choose_f64<DT, L * PER / 64>(a, t0 + at / L, __shfl(top, at), lane);
            const int mine = __shfl(r, j);
            if (base == at) id = j < k ? mine : -1;
        }
        // ---- weights, in 64 bits
        double s = 0;
        if (id >= 0) {
            const double x = load_logit<DT>(a.logits, row + id);
            s = soft ? exp(x - (double)top) / (double)z : sigmoid_f64(x);
        }
        if (a.renorm) {
            const double sum = group_reduce<L>(s, [](double x, double y) { return x + y; });
            s = sum == 0 ? 0 : s / sum;
        }
        if (live && j < k) {
            const int64_t p = (int64_t)t * k + j;
            a.ids[p] = id;
            a.w[p] = (float)(s * a.scale);
            if (order) atomicAdd(&hist[id < 0 ? E : id], 1);
        }
    }
    if (!order) return;
    __syncthreads();
    if (a.o.chunks > 1) {
        for (int i = tid; i <= E; i += kRouteThreads) a.o.hist[(int64_t)blockIdx.x * (E + 1) + i] = hist[i];
        return;
    }
    // a single workgroup: its stores of ids have been made (the barrier waits for them)
    for (int i = tid; i < kRouteWaves * 1025; i += kRouteThreads) (&sh.sort.wcnt[0][0])[i] = 0;
    exclusive_scan(hist, sh.sort.fill, E, sh.sort.tmp);
    for (int i = tid; i <= E; i += kRouteThreads) a.o.offsets[i] = sh.sort.fill[i];
    place_pairs(a.ids, 0, (int64_t)a.T * k, E, k, a.o, sh.sort);
}

// ---------------------------------------------------------------- gradient
//   G_j = dw_j scale;  renormalised: G_j <- (G_j - sum_i G_i s_i / S) / S
//   sigmoid: dl_j = G_j s_j (1 - s_j) at the chosen, 0 elsewhere
//   softmax: dl_e = s_e (G_e - sum_j G_j s_j); renormalised the sum is 0
// One wave a token; what the chosen get passes through LDS, one after the
// other, so that an expert named twice gets both.
template <int DT>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteArgs a) {
    __shared__ float rows[kThreads / 64][1024];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, k = a.k;
    float *mine = rows[wave];
    for (int e = lane; e < E; e += 64) mine[e] = 0;
    const bool soft = a.score == kSoftmax, dense = soft && !a.renorm;
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wave; t < a.T; t += (int64_t)gridDim.x * (kThreads / 64)) {
        const int64_t row = t * a.ld;
        float top = -INFINITY, z = 0;
        if (soft) {
            for (int e = lane; e < E; e += 64) top = fmaxf(top, load_logit<DT>(a.logits, row + e));
            top = group_max<64>(top);
            if (top == -INFINITY) top = 0;
            if (dense) {
                for (int e = lane; e < E; e += 64) z += exp_neg(load_logit<DT>(a.logits, row + e) - top);
                z = group_sum<64>(z);
            }
        }
        if (!dense || z == 0) z = 1;
        int id = lane < k ? a.ids[t * k + lane] : -1;
        if ((uint32_t)id >= (uint32_t)E) id = -1;
        double s = 0, rest = 0, g = 0;  // score, its complement, the gradient of the score
        if (id >= 0) {
            const double x = load_logit<DT>(a.logits, row + id);
            if (soft) {
                s = exp(x - (double)top) / (double)z;
            } else {
                const double e = exp(-fabs(x)), q = 1.0 / (1.0 + e);
                s = x < 0 ? e * q : q;
                rest = x < 0 ? q : e * q;
            }
            g = (double)a.dw[t * k + lane] * a.scale;
        }
        double gs = wave_sum_f64(g * s);
        if (a.renorm) {
            double sum = wave_sum_f64(s);
            if (sum == 0) sum = 1;
            g = (g - gs / sum) / sum;
        }
        const float d = (float)(soft ? g * s : g * s * rest);
        for (int r = 0; r < k; ++r) {
            if (lane == r && id >= 0) mine[id] += d;
            wave_sync();
        }
        const float c = (float)gs;
        for (int e = lane; e < E; e += 64) {
            float v = mine[e];
            if (dense) v -= exp_neg(load_logit<DT>(a.logits, row + e) - top) / z * c;
            store_logit<DT>(a.dlogits, t * a.d_ld + e, v);
        }
        wave_sync();
        if (id >= 0) mine[id] = 0;
        wave_sync();
    }
}

template <int DT, bool GROUPS>
void route_by_size(const RouteArgs &a, dim3 grid, hipStream_t s) {
    const dim3 block(kRouteThreads);
    if (a.E <= 64) klaunch(route_kernel<DT, 16, 4, GROUPS>, grid, block, s, a);
    else if (a.E <= 128) klaunch(route_kernel<DT, 16, 8, GROUPS>, grid, block, s, a);
    else if (a.E <= 256) klaunch(route_kernel<DT, 16, 16, GROUPS>, grid, block, s, a);
    else if (a.E <= 512) klaunch(route_kernel<DT, 32, 16, GROUPS>, grid, block, s, a);
    else klaunch(route_kernel<DT, 64, 16, GROUPS>, grid, block, s, a);
}

template <class Id>
hipError_t place(const Id *ids, int64_t P, int E, int k, const PairOrder &o, hipStream_t s) {
    klaunch(place_kernel<Id>, dim3(o.chunks), dim3(kRouteThreads), s, ids, P, E, k, o);
    return hipGetLastError();
}

}  // namespace

// At most 256 chunks, which every one of them reads the counts of, of 64 tokens at least (a pass of a workgroup).
int32_t order_chunk(int64_t tokens) {
    const int64_t each = (tokens + 255) / 256;
    return (int32_t)((each < 64 ? 64 : each) + 63) / 64 * 64;
}

hipError_t launch_route(int dt, const RouteArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + a.o.chunk - 1) / a.o.chunk));
    auto go = [&](auto d) {
        constexpr int DT = decltype(d)::value;
        if (a.groups > 1) route_by_size<DT, true>(a, grid, s);
        else route_by_size<DT, false>(a, grid, s);
    };
    if (dt == kDtF32) go(std::integral_constant<int, kDtF32>{});
    else if (dt == kDtBf16) go(std::integral_constant<int, kDtBf16>{});
    else go(std::integral_constant<int, kDtF16>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.o.perm || a.o.chunks == 1) return e;
    return place(a.ids, (int64_t)a.T * a.k, a.E, a.k, a.o, s);
}

hipError_t launch_route_grad(int dt, const RouteArgs &a, hipStream_t s) {
    auto k = dt == kDtF32 ? route_grad_kernel<kDtF32>
                          : dt == kDtBf16 ? route_grad_kernel<kDtBf16> : route_grad_kernel<kDtF16>;
    const int64_t blocks = (a.T + kThreads / 64 - 1) / (kThreads / 64);
    klaunch(k, dim3((unsigned)(blocks > 8192 ? 8192 : blocks)), dim3(kThreads), s, a);
    return hipGetLastError();
}

hipError_t launch_sort_pairs(const void *ids, bool wide, int64_t tokens, int32_t k, int32_t E, const PairOrder &o,
                             hipStream_t s) {
    const dim3 grid(o.chunks), block(kRouteThreads);
    const int64_t P = tokens * k;
    if (wide) klaunch(count_kernel<int64_t>, grid, block, s, (const int64_t *)ids, P, (int)E, (int)k, o);
    else klaunch(count_kernel<int32_t>, grid, block, s, (const int32_t *)ids, P, (int)E, (int)k, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || o.chunks == 1) return e;
    return wide ? place((const int64_t *)ids, P, E, k, o, s) : place((const int32_t *)ids, P, E, k, o, s);
}

}  // namespace qrmoe
