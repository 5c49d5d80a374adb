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
// L lanes hold a token.  A key is a double: the fp32 key, which leaves 29 bits
// of it free, and the expert's number in the lowest ten, so that minima and
// maxima of 64-bit floats order keys and settle ties by themselves.  A lane
// takes eight experts at a time, sorts them with a network and merges them
// into its eight best so far; lanes then merge their lists with a butterfly
// (the larger of one list's i-th and the other's (7 - i)-th are the eight best
// of both) until all of them hold the token's.  The largest key that did not
// make it is kept beside the list: it is the ninth.
//
// What bounds it: vector instructions, 1360 for a wave's eight tokens of 256
// experts, half of them the network's, each waiting for the one before
// (65536 tokens of fp32: 29 us, the vector units busy 57% of it; reading the
// logits takes 14).  Eight lanes a token rather than more, as each doubling of
// the lanes adds a merge.  A softmax that is not renormalised, or has a bias,
// reads the logits three times and forms its sum in 64 bits (65536 x 256 bf16
// 36 and 47 us, the same renormalised sigmoids with a bias 26).  Arguments stay
// in scalar registers and logits come through buffer loads, whose addresses
// cost one instruction (63 -> 46 us); two workgroups of 512 threads have to fit
// a CU (128 registers), or the launch itself takes longer than the work
// (8192 tokens of eight groups 44 -> 25 us).  One token: 7.6 us, a wave's
// latency.  The order of many pairs is two launches behind it, 5 and 5 to 10
// us.
#include <cfloat>
#include <type_traits>

#include "ops.hpp"

namespace qrmoe {

namespace {

constexpr int kRouteThreads = 512, kRouteWaves = kRouteThreads / 64;
constexpr int kSortThreads = 1024;
constexpr int kMaxChunks = 512;  // of the pairs' order

__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t at) {
    if constexpr (DT == kDtF32) return ((const float *)p)[at];
    else if constexpr (DT == kDtBf16) return (float)((const __bf16 *)p)[at];
    else return (float)((const _Float16 *)p)[at];
}
// The same through a buffer descriptor, offsets in bytes; past its end: 0.
template <int DT>
__device__ __forceinline__ float load_logit(__amdgpu_buffer_rsrc_t r, int at) {
    if constexpr (DT == kDtF32) return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
    else if constexpr (DT == kDtBf16) return __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0) << 16);
    else return (float)__builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
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
// e^x for x <= 0 (or NaN) in 64 bits, to 2^-31: ln 2 is taken out n times, |r| <= ln 2 / 2, the first term left out of the
// series r^9 / 9!.
__device__ __forceinline__ double exp_neg(double x) {
    x = x < -700.0 ? -700.0 : x;
    const double n = rint(x * 1.4426950408889634), r = __builtin_fma(n, -0.6931471805599453, x);
    double p = 1.0 / 40320;
    constexpr double kTerms[] = {1.0 / 5040, 1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
#pragma unroll
    for (double t : kTerms) p = __builtin_fma(p, r, t);
    return ldexp(p, (int)n);
}
// sigmoid, within 2^-22: its argument's rounding, at most .225 |l| 2^-23 / |l|, and a unit each of 2^-23 s (1 - s) for the
// power, 2^-24 s for the sum and 2^-23 s for the reciprocal
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

// What a NaN key counts as: behind every number, before -inf (an expert that is not there).  In 64 bits so that two of
// them can be added.
constexpr double kLeast = -1e300;
template <class T>
__device__ __forceinline__ T number(T key, T least) {
    return key != key ? least : key;
}
// Of packed keys, which are never NaN.  (The builtins first make sure that a NaN would be a quiet one.)
__device__ __forceinline__ double larger(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double lesser(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
// fp32 keys as doubles that carry the expert in their low ten bits: of equal ones the lower expert is the larger.
// +-infinity, which has no room for it, is +-kFar, a NaN kNan; an expert that is not there has kAbsent.
constexpr double kFar = 0x1p200, kNan = -0x1p150, kAbsent = -0x1p300;
__device__ __forceinline__ double pack_key(float key, int e, bool in) {
    // (a NaN gives way to the other operand)
    const uint64_t u = (uint64_t)__double_as_longlong(lesser(larger((double)key, kNan), kFar));
    const uint32_t top = (uint32_t)(u >> 32), hi = in ? top : (uint32_t)((uint64_t)__builtin_bit_cast(uint64_t, kAbsent) >> 32);
    const uint32_t low = (uint32_t)u | ((uint32_t)e ^ (1023u & ~(uint32_t)((int)top >> 31)));
    return __longlong_as_double((long long)((uint64_t)hi << 32 | low));
}
__device__ __forceinline__ int expert_of(double k) {
    const uint64_t u = (uint64_t)__double_as_longlong(k);
    return (int)(((uint32_t)u ^ ~(uint32_t)((int)(u >> 32) >> 31)) & 1023u);
}
__device__ __forceinline__ bool there(double k) { return k > -0x1p299; }
__device__ __forceinline__ float value_of(double k) {  // the fp32 key (a NaN's: -infinity)
    return (float)__longlong_as_double(__double_as_longlong(k) & ~1023ll);
}

constexpr int kList = 8;
__device__ __forceinline__ void order2(double &a, double &b) {
    const double x = larger(a, b);
    b = lesser(a, b);
    a = x;
}
// The largest first: odd-even merge sort
__device__ __forceinline__ void sort_list(double (&v)[kList]) {
#pragma unroll
    for (int p = 1; p < kList; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < kList; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < kList && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order2(v[i + j], v[i + j + q]);
}
// v: the eight best of the sorted lists v and o; ninth: the largest of what either has lost, where it is asked for.
__device__ __forceinline__ void merge_list(double (&v)[kList], const double (&o)[kList], double &ninth, bool want) {
    if (want) {
#pragma unroll
        for (int i = 0; i < kList; ++i) ninth = larger(ninth, lesser(v[i], o[kList - 1 - i]));
    }
#pragma unroll
    for (int i = 0; i < kList; ++i) v[i] = larger(v[i], o[kList - 1 - i]);
#pragma unroll
    for (int q = kList / 2; q >= 1; q /= 2)  // falls, then rises (or any rotation of that): sorted by halves
#pragma unroll
        for (int i = 0; i < kList; ++i)
            if ((i & q) == 0) order2(v[i], v[i + q]);
}
template <int D>
__device__ __forceinline__ double partner(double v) {  // of the butterfly at distance D; DPP only where that is enough
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    uint32_t a, b, c, d;
    bfly_pair_u32<D>((uint32_t)u, a, b);
    bfly_pair_u32<D>((uint32_t)(u >> 32), c, d);
    const bool upper = (threadIdx.x & D) != 0;
    const uint32_t lo = D <= 8 ? b : upper ? a : b, hi = D <= 8 ? d : upper ? c : d;
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
template <int L, int D = 1>
__device__ __forceinline__ void merge_lanes(double (&v)[kList], double &ninth, bool want) {
    if constexpr (D < L) {
        double o[kList];
#pragma unroll
        for (int i = 0; i < kList; ++i) o[i] = partner<D>(v[i]);
        const double other = want ? partner<D>(ninth) : 0.0;
        merge_list(v, o, ninth, want);
        if (want) ninth = larger(ninth, other);
        merge_lanes<L, 2 * D>(v, ninth, want);
    }
}

// a - b + c with the right sign, so that comparing by it is an order: rounded differences could say that x is before y, y
// before z and z before x.  The roundings of both sums are added to the result.
__device__ __forceinline__ double difference(double a, double b, double c) {
    const double s = a - b, t = s + c;
    if (!(fabs(s) < INFINITY)) return s;  // one of them is not there
    const double u = s - a, v = t - s;
    return t + (((s - (t - v)) + (c - v)) + ((a - (s - u)) - (b + u)));
}

// ------------------------------------------------- one token in 64 bits
// The whole wave decides for token t: lanes r < k get the expert of rank r
// (-1: none left).  top, z: the row's largest logit and sum of e^(l - top).
// A function of its own, so that the registers of what hardly ever runs stay out of what always does.
template <int DT>
__device__ __attribute__((noinline)) int choose_f64(const RouteArgs &a, int64_t t, float top, bool biased, int lane) {
    const int S = (a.E + 63) / 64;  // slots of 64 experts
    const int64_t row = t * a.ld;
    const bool soft = a.score == kSoftmax, by_logit = !biased && a.groups == 1;
    double key[16];  // in memory: registers would cost every other token
    double z = 0;
    if (soft && !by_logit) {
        for (int e = lane; e < a.E; e += 64) z += exp((double)load_logit<DT>(a.logits, row + e) - (double)top);
        z = wave_sum_f64(z);
        if (z == 0) z = 1;
    }
    auto key_of = [&](int e, bool score) -> double {
        const float lf = load_logit<DT>(a.logits, row + e);
        const double l = lf, b = biased ? (double)a.bias[e] : 0.0;
        if (lf == -INFINITY) return -INFINITY;
        if (!score) return number(l, kLeast);
        return number((soft ? exp(l - (double)top) / z : sigmoid_f64(l)) + b, kLeast);
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
        key[i] = -INFINITY;
        if (64 * i < a.E && lane + 64 * i < a.E) key[i] = key_of(lane + 64 * i, !by_logit);
    }
    if (a.groups > 1) {
        const int size = a.E / a.groups;
        double mine = -INFINITY;  // of group `lane`
        int many = 0;             // the keys in it: a bias that is the same for all counts that often
        const double even = a.bias && !biased ? (double)a.bias[0] : 0.0;
        for (int g = 0; g < a.groups; ++g) {
            double t1 = -INFINITY, t2 = -INFINITY;
            auto add = [&](double x) {
                t2 = fmax(t2, fmin(t1, x));
                t1 = fmax(t1, x);
            };
#pragma unroll 1
            for (int i = 0; i < S; ++i)
                if (64 * i < a.E && (lane + 64 * i) / size == g) add(key[i]);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
                add(o1);
                add(o2);
            }
            const bool two = a.best == 2 && t2 != -INFINITY;
            const double v = two ? t1 + t2 : t1;
            if (lane == g) {
                mine = v;
                many = two ? 2 : t1 != -INFINITY;
            }
        }
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl(mine, g);
            const int n = __shfl(many, g) - many;
            const double d = o == mine ? n * even : difference(o, mine, n * even);
            before += d > 0 || (d == 0 && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && before < a.keep);
#pragma unroll 1
        for (int i = 0; i < S; ++i) {
            const int g = (lane + 64 * i) / size;
            if (64 * i < a.E && g < a.groups) {
                if (!((kept >> g) & 1)) key[i] = -INFINITY;
                // the scores of the chosen groups rank as their logits do
                else if (!biased && key[i] != -INFINITY) key[i] = key_of(lane + 64 * i, false);
            }
        }
    }
    int id = -1;
    for (int r = 0; r < a.k; ++r) {
        double m = key[0];
#pragma unroll 1
        for (int i = 1; i < S; ++i) m = fmax(m, key[i]);
        m = group_reduce<64>(m, [](double x, double y) { return fmax(x, y); });
        if (m == -INFINITY) break;
        uint32_t at = 0xffffffffu;
#pragma unroll 1
        for (int i = S - 1; i >= 0; --i) at = key[i] == m ? (uint32_t)(lane + 64 * i) : at;
        at = group_reduce<64>(at, umin);
#pragma unroll 1
        for (int i = 0; i < S; ++i)
            if ((uint32_t)(lane + 64 * i) == at) key[i] = -INFINITY;
        if (lane == r) id = (int)at;
    }
    return id;
}

// -------------------------------------------------------------- pair order
// Stable counting sort: the pairs of each expert in each chunk of tokens are
// counted, the counts summed over the chunks before, the pairs placed.  Ranks
// within a wave come from ballots on the bucket's bits, so that neither order
// nor places depend on timing.  65536 tokens of six pairs: the router counts on
// the way, the sums take 5 us, the placing 10 (a workgroup a chunk, three
// barriers for 1024 pairs).
template <int THREADS>
struct SortShared {
    int fill[1025], wcnt[THREADS / 64][1025];
    int tmp[THREADS / 64];
};

template <int THREADS>
__device__ __forceinline__ void zero_counts(SortShared<THREADS> &sh, int E) {
    for (int w = 0; w < THREADS / 64; ++w)
        for (int i = threadIdx.x; i <= E; i += THREADS) sh.wcnt[w][i] = 0;
}

// fill[b] for b <= E: how many pairs stand before those of bucket b, from total[b] (LDS; the buckets' pairs; may be fill).
template <int THREADS>
__device__ __forceinline__ void exclusive_scan(const int *total, int *fill, int E, int *tmp) {
    constexpr int N = (1024 + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    int v[N], sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = N * tid + i < E ? total[N * tid + i] : 0;
        sum += v[i];
    }
    const int inc = wave_incl_scan(sum);
    if (lane == 63) tmp[wave] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < wave; ++w) at += tmp[w];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (N * tid + i < E) fill[N * tid + i] = at;
        at += v[i];
    }
    if (tid == THREADS - 1) fill[E] = at;
    __syncthreads();
}

// Places pairs [p0, p1) in order; sh.fill[b] is the next free place of bucket b, sh.wcnt is zero.
template <int THREADS, class Id>
__device__ __forceinline__ void place_pairs(const Id *ids, int64_t p0, int64_t p1, int E, int k, const PairOrder &o,
                                            SortShared<THREADS> &sh) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    for (int64_t base = p0; base < p1; base += THREADS) {
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
            o.rows[at] = (int32_t)((uint32_t)p / (uint32_t)k);
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

// Turns the counts of the chunks into how many pairs of a bucket stand in the chunks before, and the row behind the last
// chunk into their totals.  A workgroup takes 32 buckets, 32 threads for the rows of each.
__global__ __launch_bounds__(kSortThreads) void scan_kernel(int E, PairOrder o) {
    __shared__ int part[32][33];
    constexpr int kEach = kMaxChunks / 32;
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, buckets = E + 1, b = blockIdx.x * 32 + c;
    const int each = (o.chunks + 31) / 32, r0 = g * each;
    auto mine = [&](int i) { return i < each && r0 + i < o.chunks && b < buckets; };
    int v[kEach], sum = 0;  // all on their way at once
#pragma unroll
    for (int i = 0; i < kEach; ++i) v[i] = mine(i) ? o.hist[(int64_t)(r0 + i) * buckets + b] : 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += v[i];
    part[g][c] = sum;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) at += i < g ? part[i][c] : 0;
    if (g == 31 && b < buckets) o.hist[(int64_t)o.chunks * buckets + b] = at + sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (mine(i)) o.hist[(int64_t)(r0 + i) * buckets + b] = at;
        at += v[i];
    }
}

template <class Id>
__global__ __launch_bounds__(kSortThreads) void place_kernel(const Id *ids, int64_t P, int E, int k, PairOrder o) {
    __shared__ SortShared<kSortThreads> sh;
    const int tid = threadIdx.x, c = blockIdx.x, buckets = E + 1;
    zero_counts<kSortThreads>(sh, E);
    for (int i = tid; i < buckets; i += kSortThreads) sh.fill[i] = o.hist[(int64_t)o.chunks * buckets + i];
    __syncthreads();
    exclusive_scan<kSortThreads>(sh.fill, sh.fill, E, sh.tmp);
    for (int i = tid; i < buckets; i += kSortThreads) {
        if (c == 0) o.offsets[i] = sh.fill[i];
        sh.fill[i] += o.hist[(int64_t)c * buckets + i];
    }
    __syncthreads();
    const int64_t p0 = (int64_t)c * o.chunk * k, p1 = min(P, p0 + (int64_t)o.chunk * k);
    place_pairs<kSortThreads>(ids, p0, p1, E, k, o, sh);
}

// The counts of one chunk; where it is the only one, the whole order.
template <class Id>
__global__ __launch_bounds__(kSortThreads) void count_kernel(const Id *ids, int64_t P, int E, int k, PairOrder o) {
    __shared__ SortShared<kSortThreads> sh;
    const int tid = threadIdx.x, c = blockIdx.x;
    for (int i = tid; i <= E; i += kSortThreads) sh.fill[i] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)c * o.chunk * k, p1 = min(P, p0 + (int64_t)o.chunk * k);
    for (int64_t p = p0 + tid; p < p1; p += kSortThreads) {
        const Id id = ids[p];
        atomicAdd(&sh.fill[id < 0 || id >= (Id)E ? E : (int)id], 1);
    }
    __syncthreads();
    if (o.chunks > 1) {
        for (int i = tid; i <= E; i += kSortThreads) o.hist[(int64_t)c * (E + 1) + i] = sh.fill[i];
        return;
    }
    zero_counts<kSortThreads>(sh, E);
    exclusive_scan<kSortThreads>(sh.fill, sh.fill, E, sh.tmp);
    for (int i = tid; i <= E; i += kSortThreads) o.offsets[i] = sh.fill[i];
    place_pairs<kSortThreads>(ids, p0, p1, E, k, o, sh);
}

// The order of few pairs by comparing each with all; `few` has the pairs' buckets.  Router and order of 1 / 4 / 5 tokens of
// six pairs, a hundred calls in a graph: so 7.7 / 8.1 / 8.6 us each, by counting 8.6 / 8.6 / 8.6.
constexpr int kFewPairs = 32;
__device__ __forceinline__ void order_few(const int *few, int P, int E, int k, const PairOrder &o) {
    const int tid = threadIdx.x;
    for (int e = tid; e <= E; e += kRouteThreads) {
        int n = 0;
        for (int q = 0; q < P; ++q) n += few[q] < e;
        o.offsets[e] = n;
    }
    if (tid < P) {
        const int e = few[tid];
        int at = 0;
        for (int q = 0; q < P; ++q) at += few[q] < e || (few[q] == e && q < tid);
        o.perm[at] = tid;
        o.rows[at] = (int32_t)((uint32_t)tid / (uint32_t)k);
        o.place[tid] = at;
    }
}

// ------------------------------------------------------------------ router
constexpr int kGroupKeys = 1024;  // keys that a wave keeps in LDS to choose groups: L = E / 16 lanes a token at least

template <int DT, int L, bool GROUPS, bool SOFT>
__global__ __launch_bounds__(kRouteThreads, 4) void route_kernel(RouteArgs a) {
    constexpr int TW = 64 / L, TB = TW * kRouteWaves;  // tokens of a wave, of a workgroup's pass
    // keys of a wave's tokens by expert; afterwards, in a single workgroup, the order of the pairs
    __shared__ union Shared {
        float keys[GROUPS ? kRouteWaves : 1][GROUPS ? kGroupKeys : 1];
        SortShared<kRouteThreads> sort;
    } sh;
    __shared__ int hist[1025];  // pairs of each expert; few pairs: the expert of each
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & (L - 1), base = lane & ~(L - 1);  // this lane among its token's; the first of them
    const int E = a.E, k = a.k;
    const bool order = a.o.perm != nullptr, few = order && a.T * k <= kFewPairs;
    if (order && !few) {
        for (int i = tid; i <= E; i += kRouteThreads) hist[i] = 0;
        __syncthreads();
    }
    constexpr int B = DT == kDtF32 ? 4 : 2;
    const int first_t = (int)blockIdx.x * a.o.chunk, t_end = min(a.T, first_t + a.o.chunk);
    // offsets are relative to the chunk's first row and have 31 bits (checked on the host)
    const uint8_t *const chunk = (const uint8_t *)a.logits + (int64_t)first_t * a.ld * B;
    const auto from = buf_rsrc(chunk, (uint32_t)(((int64_t)(t_end - first_t - 1) * a.ld + E) * B));
    const auto bias_from = buf_rsrc(a.bias, a.bias ? 4 * E : 0);  // no bias: zeros
    // the first logits are asked for before anything is waited for
    const float ahead = load_logit<DT>(from, (int)(min(wave * TW + lane / L, t_end - first_t - 1) * a.ld + min(j, E - 1)) * B);
    // a bias that is the same for every expert changes no order: then, as without one, the logits are the keys
    bool biased = false;
    float even = 0;  // what such a bias is
    if (a.bias) {
        const float first = even = a.bias[0];
        bool same = fabsf(first) < INFINITY;
        for (int e0 = 0; e0 < E; e0 += 256) {
            float b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = a.bias[min(e0 + 64 * i + lane, E - 1)];
#pragma unroll
            for (int i = 0; i < 4; ++i) same &= b[i] == first;
        }
        biased = __ballot(!same) != 0;
    }
    asm volatile("" ::"v"(ahead));
    const bool ninth_wanted = k == kList && biased;
    const bool scored = biased || GROUPS;
    for (int t0 = first_t + wave * TW; t0 < t_end; t0 += TB) {
        const int t = t0 + lane / L;
        const bool live = t < t_end;
        const int row = (int)((min(t, t_end - 1) - first_t) * a.ld) * B;  // bytes behind the chunk's first
        // this lane's logits of experts e0 + L i + j; -inf past the last
        auto logits = [&](int e0, float (&l)[kList]) {
#pragma unroll
            for (int i = 0; i < kList; ++i) l[i] = load_logit<DT>(from, row + (e0 + j) * B + L * i * B);
#pragma unroll
            for (int i = 0; i < kList; ++i) l[i] = e0 + L * i + j < E ? l[i] : -INFINITY;
        };

        float top = 0, rz = 1;
        double z = 1;
        // A key's error is that of its score, the bias's rounding apart.  Sigmoids: sigmoid_near.  Softmax: the sum, in 64
        // bits, has none to speak of: in one of 1024 terms that fp32 adds, what it loses of each can pass any bound that
        // leaves much to fp32 (1023 terms of e^-16.6 beside one of 1: 7.5e-6).  Left is e^x / z, to units of 2^-24 of the
        // largest probability, 1 / z: |x| e^x times 2.5 for the argument's roundings, one at most; two each for the power and
        // for 1 / z, one for the product.
        float slack = 0x1p-22f;
        if (SOFT && (scored || !a.renorm)) {
            float l[kList];
            top = -INFINITY;
            for (int e0 = 0; e0 < E; e0 += kList * L) {
                logits(e0, l);
#pragma unroll
                for (int i = 0; i < kList; ++i) top = fmaxf(top, l[i]);
            }
            top = group_max<L>(top);
            if (top == -INFINITY) top = 0;
            double part = 0;
            for (int e0 = 0; e0 < E; e0 += kList * L) {
                logits(e0, l);
#pragma unroll
                for (int i = 0; i < kList; ++i) part += exp_neg((double)l[i] - (double)top);
            }
            z = group_reduce<L>(part, [](double x, double y) { return x + y; });
            if (z == 0) z = 1;
            rz = 1.0f / (float)z;
            slack = 0x1p-21f * rz;
        }
        // fp32 keys by score; a logit of -inf needs its own look
        auto by_score = [&](int e0, const float (&l)[kList], float (&f)[kList]) {
            float b[kList];
#pragma unroll
            for (int i = 0; i < kList; ++i) b[i] = load_logit<kDtF32>(bias_from, (e0 + j) * 4 + L * i * 4);
#pragma unroll
            for (int i = 0; i < kList; ++i)
                f[i] = (SOFT ? __builtin_amdgcn_exp2f((l[i] - top) * 1.44269504f) * rz : sigmoid_near(l[i])) + b[i];
        };

        bool unsure = false;
        const int size = GROUPS ? E / a.groups : 1;
        float *const keys = GROUPS ? sh.keys[wave] + (lane / L) * (kGroupKeys / TW) : nullptr;
        if constexpr (GROUPS) {
            wave_sync();  // the tokens before are done with the keys
            for (int e0 = 0; e0 < E; e0 += kList * L) {
                float l[kList], f[kList];
                logits(e0, l);
                by_score(e0, l, f);
#pragma unroll
                for (int i = 0; i < kList; ++i)
                    if (e0 + L * i + j < E)
                        keys[e0 + L * i + j] = l[i] == -INFINITY ? -INFINITY : number(f[i], -FLT_MAX);
            }
            // lane g < groups: group g's score; lanes start at places of their own in it (banks)
            wave_sync();
            float t1 = -INFINITY, t2 = -INFINITY;
            if (j < a.groups) {
                int at = j % size;
#pragma unroll 1
                for (int n = 0; n < size; n += 8) {
                    float x[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        x[u] = n + u < size ? keys[j * size + at] : -INFINITY;
                        at = at + 1 == size ? 0 : at + 1;
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        t2 = fmaxf(t2, fminf(t1, x[u]));
                        t1 = fmaxf(t1, x[u]);
                    }
                }
            }
            const float mine = a.best == 2 && t2 != -INFINITY ? t1 + t2 : t1;
            // what its roundings are relative to: three of 2^-24 at most
            const float size_of = (t1 == -INFINITY ? 0.0f : fabsf(t1)) + (t2 == -INFINITY ? 0.0f : fabsf(t2));
            int before = 0;
#pragma unroll 1
            for (int g = 0; g < a.groups; ++g) {
                const float o = __shfl(mine, base + g);
                before += o > mine || (o == mine && g < j);
            }
            bool in = j < a.groups && before < a.keep;
            // the least of the kept must be clearly above the largest of the others that are there (their sum may be past
            // fp32: then size_of is too, and nothing is clear)
            const float least = -group_max<L>(in ? -mine : -INFINITY);
            const float most = group_max<L>(!in && j < a.groups ? mine : -INFINITY);
            const bool others = group_max<L>(!in && j < a.groups && t1 != -INFINITY ? 1.0f : 0.0f) > 0;
            unsure = others && !(least - most > 4 * slack + 0x1p-21f * group_max<L>(size_of));
            // Where it is not, the groups' best experts are scored in 64 bits (not with a softmax's sum and a bias: that
            // sum is good to 2^-31 only).  They have to be the best beyond doubt, else choose_f64 decides.
            if ((!SOFT || !biased) && __ballot(unsure) != 0) {
                // the best two by key (the third may be too near to tell), or without a bias by logit, which is exact
                int i1 = 0, i2 = 0;
                float b1 = -INFINITY, b2 = -INFINITY, t3 = -INFINITY;
                if (j < a.groups) {
#pragma unroll 1
                    for (int n = 0; n < size; ++n) {
                        float x = keys[j * size + n];
                        if (!biased && x != -INFINITY) x = load_logit<DT>(from, row + (j * size + n) * B);
                        t3 = fmaxf(t3, x > b2 ? b2 : x);
                        if (x > b1) b2 = b1, i2 = i1, b1 = x, i1 = n;
                        else if (x > b2) b2 = x, i2 = n;
                    }
                }
                // A bias that is the same for all is left out, and so is a softmax's sum: that orders groups which count it
                // equally often.  Where they do not, choose_f64 decides.
                auto exactly = [&](int n) -> double {
                    const double l = load_logit<DT>(from, row + (j * size + n) * B);
                    return (SOFT ? exp(l - (double)top) : sigmoid_f64(l)) +
                           (biased ? load_logit<kDtF32>(bias_from, (j * size + n) * 4) : 0.0f);
                };
                const bool two = a.best == 2 && t2 != -INFINITY, some = j < a.groups && t1 != -INFINITY;
                const bool unlike = !biased && even != 0 && group_max<L>(some && two ? 1.0f : 0.0f) > 0 &&
                                    group_max<L>(some && !two ? 1.0f : 0.0f) > 0;
                double score = -INFINITY;
                if (j < a.groups && t1 > -FLT_MAX) score = exactly(i1);
                if (j < a.groups && two && t2 > -FLT_MAX) score += exactly(i2);
                const float last = a.best == 2 ? t2 : t1, next = a.best == 2 ? t3 : t2;
                const bool clear = !biased || next == -INFINITY ||
                                   last - next > 2 * slack + 0x1p-23f * fmaxf(fabsf(last), fabsf(next));
                // (a NaN among a group's best counts as the least number: left to choose_f64)
                const bool vague = j < a.groups && (unlike || !clear || t1 == -FLT_MAX || (two && t2 == -FLT_MAX));
                before = 0;
#pragma unroll 1
                for (int g = 0; g < a.groups; ++g) {
                    const double o = __shfl(score, base + g);
                    before += o > score || (o == score && g < j);
                }
                if (unsure) in = j < a.groups && before < a.keep;  // the wave's other tokens are settled
                unsure = unsure && ((__ballot(vague) >> base) & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1)) != 0;
            }
            wave_sync();
            if (j < a.groups && !in)
                for (int n = 0; n < size; ++n) keys[j * size + n] = -INFINITY;
            wave_sync();
        }

        // ---- the eight largest keys, and the ninth
        double list[kList], ninth = kAbsent;
        for (int e0 = 0; e0 < E; e0 += kList * L) {
            double v[kList];
            float l[kList], f[kList];
            if constexpr (GROUPS) {  // keys of groups that are out have become -inf
#pragma unroll
                for (int i = 0; i < kList; ++i) f[i] = e0 + L * i + j < E ? keys[e0 + L * i + j] : -INFINITY;
#pragma unroll
                for (int i = 0; i < kList; ++i) v[i] = pack_key(f[i], e0 + L * i + j, f[i] != -INFINITY);
                if (!biased) {
                    logits(e0, l);
#pragma unroll
                    for (int i = 0; i < kList; ++i)
                        v[i] = pack_key(l[i] + 0.0f, e0 + L * i + j, f[i] != -INFINITY && l[i] != -INFINITY);
                }
            } else {
                logits(e0, l);
                if (biased) {
                    by_score(e0, l, f);
#pragma unroll
                    for (int i = 0; i < kList; ++i)
                        v[i] = pack_key(f[i], e0 + L * i + j, l[i] != -INFINITY && f[i] != -INFINITY);
                } else {
#pragma unroll
                    for (int i = 0; i < kList; ++i) v[i] = pack_key(l[i] + 0.0f, e0 + L * i + j, l[i] != -INFINITY);  // -0 as 0
                }
            }
            sort_list(v);
            if (e0 == 0) {
#pragma unroll
                for (int i = 0; i < kList; ++i) list[i] = v[i];
            } else {
                merge_list(list, v, ninth, ninth_wanted);
            }
        }
        merge_lanes<L>(list, ninth, ninth_wanted);
        // lanes 0 .. 7 of the token: a candidate each, its logit, its score in 64 bits
        double cand = kAbsent;
#pragma unroll
        for (int i = 0; i < kList; ++i) cand = j == i ? list[i] : cand;
        int id = there(cand) ? expert_of(cand) : -1, rank = j;
        if (biased) {
            // Keys by score may be off.  Sigmoids: the candidates are the right ones if a clear step comes between rank
            // k and what is not among them, and their order is settled below.  (Behind a softmax's key is a sum that
            // only choose_f64 has to the last bit: all steps have to be clear.)
            bool any = false, all = true;
#pragma unroll
            for (int i = 0; i < kList; ++i) {
                const double next = i + 1 < kList ? list[i + 1 < kList ? i + 1 : i] : ninth;
                const float hi = value_of(list[i]), lo = value_of(next);
                const bool clear = !there(next) || hi - lo > 2 * slack + 0x1p-23f * fmaxf(fabsf(hi), fabsf(lo));
                any |= i >= k - 1 && (i + 1 < kList || ninth_wanted) && clear;
                all &= i >= k || clear;
            }
            unsure |= SOFT ? !all : !any;
        }
        // where fp32 cannot tell, the whole wave decides in 64 bits, a token at a time
        uint64_t todo = __ballot(unsure && live && j == 0);
        while (todo) {
            const int at = __ffsll((long long)todo) - 1;
            todo &= todo - 1;
            const RouteArgs copy = a;  // in memory, where the call needs it; `a` itself stays in scalar registers
            const int r = choose_f64<DT>(copy, t0 + at / L, __shfl(top, at), biased, lane);
            const int theirs = __shfl(r, j);
            if (base == at) id = j < k ? theirs : -1;
        }
        // Weights, in 64 bits.  Renormalised, a softmax needs no sum over all.
        const float l = id >= 0 ? load_logit<DT>(from, row + id * B) : -INFINITY;
        const float about = SOFT && a.renorm ? group_max<L>(l) : top;
        double s = 0;
        if (id >= 0) s = SOFT ? exp((double)l - (double)about) / (a.renorm ? 1.0 : z) : sigmoid_f64(l);
        if (!SOFT && biased) {  // rank by the keys in 64 bits (a token that choose_f64 has ranked stays as it is)
            const double key = id < 0 ? -INFINITY : number(s + (double)a.bias[id], kLeast);
            int before = 0;
#pragma unroll 1
            for (int i = 0; i < kList; ++i) {
                const double o = __shfl(key, base + i);
                const int other = __shfl(id, base + i);
                before += o > key || (o == key && other < id);
            }
            rank = j >= kList ? L : id < 0 ? j : before;
        }
        const bool chosen = rank < k;
        if (!chosen) s = 0;
        if (a.renorm) {
            const double sum = group_reduce<L>(s, [](double x, double y) { return x + y; });
            s = sum == 0 ? 0 : s / sum;
        }
        if (live && chosen) {
            const int64_t p = (int64_t)t * k + rank;
            a.ids[p] = id;
            a.w[p] = (float)(s * a.scale);
            if (few) hist[p] = id < 0 ? E : id;
            else if (order) atomicAdd(&hist[id < 0 ? E : id], 1);
        }
    }
    if (!order) return;
    __syncthreads();
    if (few) {
        order_few(hist, a.T * k, E, k, a.o);
        return;
    }
    if (a.o.chunks > 1) {
        for (int i = tid; i <= E; i += kRouteThreads) a.o.hist[(int64_t)blockIdx.x * (E + 1) + i] = hist[i];
        return;
    }
    // a single workgroup: its stores of ids have been made (the barrier waits for them)
    zero_counts<kRouteThreads>(sh.sort, E);
    exclusive_scan<kRouteThreads>(hist, sh.sort.fill, E, sh.sort.tmp);
    for (int i = tid; i <= E; i += kRouteThreads) a.o.offsets[i] = sh.sort.fill[i];
    place_pairs<kRouteThreads>(a.ids, 0, (int64_t)a.T * k, E, k, a.o, sh.sort);
}

// ---------------------------------------------------------------- gradient
//   G_j = dw_j scale;  renormalised: G_j <- (G_j - sum_i G_i s_i / S) / S
//   sigmoid: dl_j = G_j s_j (1 - s_j) at the chosen, 0 elsewhere
//   softmax: dl_e = s_e (G_e - sum_j G_j s_j); renormalised the sum is 0
// What it has to move is the gradient of every logit, and the logits where all of them have one (DENSE: softmax, not
// renormalised); those are read once and their exponentials stay in registers.  L lanes a token, V consecutive experts
// a lane and access.  What the chosen get passes through LDS: an expert named twice has both's, by one after the other or
// (DENSE) by the first of them.  What those get is summed over pairs of experts, so that nothing is lost where one has all
// the weight.  65536 tokens of 256 experts, six chosen, bf16: DENSE 21.6 us (67 MB, 3.1 TB/s; the vector units are busy
// two thirds of the time, with the exponentials and the chosen's 64-bit sums), else 12.3 (34 MB and the chosen logits).
constexpr int kGradThreads = 256;
template <int DT, int V>
__device__ __forceinline__ void load_some(const void *p, int64_t at, float (&v)[V]) {
    typedef typename std::conditional<DT == kDtF32, float, typename std::conditional<DT == kDtBf16, __bf16, _Float16>::type>::type T;
    typedef T TV __attribute__((ext_vector_type(V)));
    if constexpr (V == 1) {
        v[0] = (float)((const T *)p)[at];
    } else {
        const TV x = *reinterpret_cast<const TV *>((const T *)p + at);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)x[i];
    }
}
template <int DT, int V>
__device__ __forceinline__ void store_some(void *p, int64_t at, const float (&v)[V]) {
    typedef typename std::conditional<DT == kDtF32, float, typename std::conditional<DT == kDtBf16, __bf16, _Float16>::type>::type T;
    typedef T TV __attribute__((ext_vector_type(V)));
    if constexpr (V == 1) {
        ((T *)p)[at] = (T)v[0];
    } else {
        TV x;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (T)v[i];
        *reinterpret_cast<TV *>((T *)p + at) = x;
    }
}

// f(integral_constant r) for the ranks r < k.
template <int R = 0, class F>
__device__ __forceinline__ void each_rank(int k, F &&f) {
    if constexpr (R < kMaxTopK) {
        if (R >= k) return;
        f(std::integral_constant<int, R>{});
        each_rank<R + 1>(k, f);
    }
}
// What the lane of rank R has: lane R of a row of 16, which is a token's row or, of 64 lanes a token, the one that its
// pairs are in.
template <int R>
__device__ __forceinline__ int of_rank(int v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x150 + R, 0xf, 0xf, false);  // row_newbcast
}
template <int R>
__device__ __forceinline__ double of_rank(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)of_rank<R>((int)u), hi = (uint32_t)of_rank<R>((int)(u >> 32));
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

template <int DT, int L, int PER, int V, bool DENSE>
__global__ __launch_bounds__(kGradThreads) void route_grad_kernel(RouteArgs a) {
    constexpr int TW = 64 / L, WAVES = kGradThreads / 64, N = PER / V;  // accesses of a lane
    __shared__ float rows[WAVES][TW][L * PER];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & (L - 1), E = a.E, k = a.k;
    float *mine = rows[wave][lane / L];
#pragma unroll
    for (int i = 0; i < PER; ++i) mine[L * i + j] = 0;
    wave_sync();
    const bool soft = DENSE || a.score == kSoftmax;
    const int64_t step = (int64_t)gridDim.x * WAVES * TW;
    for (int64_t t0 = ((int64_t)blockIdx.x * WAVES + wave) * TW; t0 < a.T; t0 += step) {
        const int64_t t = t0 + lane / L, tt = t < a.T ? t : a.T - 1;
        const int64_t row = tt * a.ld;
        int id = j < k ? a.ids[tt * k + j] : -1;
        if ((uint32_t)id >= (uint32_t)E) id = -1;
        const float dw = j < k ? a.dw[tt * k + j] : 0.0f;
        const float l = id >= 0 ? load_logit<DT>(a.logits, row + id) : -INFINITY;
        float ex[N][V], top = 0;
        double rest = 0;  // DENSE: the sum of the exponentials of what is not chosen
        if constexpr (DENSE) {
            if (id >= 0) mine[id] = 1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = (i * L + j) * V;  // all of the V or none are experts
                load_some<DT, V>(a.logits, row + min(e, E - V), ex[i]);
#pragma unroll
                for (int u = 0; u < V; ++u) ex[i][u] = e < E ? ex[i][u] : -INFINITY;
            }
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int u = 0; u < V; ++u) top = fmaxf(top, ex[i][u]);
            top = group_max<L>(top);
            if (top == -INFINITY) top = 0;
            wave_sync();
            float z = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    ex[i][u] = mine[(i * L + j) * V + u] != 0 ? 0.0f : exp_neg(ex[i][u] - top);
                    z += ex[i][u];
                }
            rest = group_reduce<L>((double)z, [](double x, double y) { return x + y; });
        }
        float d, c = 0;
        if constexpr (DENSE) {
            // G_j - sum_i G_i s_i = sum over all experts of (G_j - G_e) s_e, which keeps its precision where s_j is near 1.
            // What is not chosen has G = 0; an expert named twice has both's G, in the first lane that names it.
            const double g = id >= 0 ? (double)dw * a.scale : 0.0;
            double both = 0, s = id >= 0 ? exp((double)l - (double)top) : 0.0;
            bool first = id >= 0;
            each_rank(k, [&](auto r) {
                const bool same = of_rank<decltype(r)::value>(id) == id;
                both += same ? of_rank<decltype(r)::value>(g) : 0.0;
                first &= !same || decltype(r)::value >= j;
            });
            auto add = [](double x, double y) { return x + y; };
            s = first ? s : 0.0;
            const double z = rest + group_reduce<L>(s, add), rz = z == 0 ? 1.0 : 1.0 / z;
            s *= rz;
            c = (float)(group_reduce<L>(both * s, add) * rz);
            double sum = both * (rest * rz);
            each_rank(k, [&](auto r) {
                sum += (both - of_rank<decltype(r)::value>(both)) * of_rank<decltype(r)::value>(s);
            });
            d = (float)(s * sum);
            if (!first) id = -1;
            wave_sync();  // all have read what is named
            if (id >= 0) mine[id] = d;
            wave_sync();
        } else {
            double s = 0, rest = 0, g = id >= 0 ? (double)dw * a.scale : 0.0;  // score, its complement, the gradient of the score
            float about = soft ? group_max<L>(l) : 0.0f;
            if (about == -INFINITY) about = 0;  // every expert named has logit -inf: scores of 0
            if (id >= 0) {
                const double x = soft ? (double)l - (double)about : (double)l, e = exp(soft ? x : -fabs(x)), q = 1.0 / (1.0 + e);
                s = soft ? e : x < 0 ? e * q : q;
                rest = soft ? 1.0 : x < 0 ? q : e * q;
            }
            auto add = [](double x, double y) { return x + y; };
            if (a.renorm) {  // of s / S, and G_j - sum_i G_i s_i / S = sum_i (G_j - G_i) s_i / S, as above
                const double sum = group_reduce<L>(s, add);
                s = sum == 0 ? 0.0 : s / sum;
                double to = 0;
                each_rank(k, [&](auto i) {
                    to += (g - of_rank<decltype(i)::value>(g)) * of_rank<decltype(i)::value>(s);
                });
                g = to;
            }
            d = (float)(g * s * rest);
        }
        for (int r = 0; !DENSE && r < k; ++r) {
            if (j == r && id >= 0) mine[id] += d;
            wave_sync();
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = (i * L + j) * V;
            float v[V];
#pragma unroll
            for (int u = 0; u < V; ++u) {
                v[u] = mine[e + u];
                if constexpr (DENSE) v[u] = __builtin_fmaf(-c, ex[i][u], v[u]);
            }
            if (e < E && t < a.T) store_some<DT, V>(a.dlogits, t * a.d_ld + e, v);
        }
        wave_sync();
        if (id >= 0) mine[id] = 0;
        wave_sync();
    }
}

template <class Id>
hipError_t place(const Id *ids, int64_t P, int E, int k, const PairOrder &o, hipStream_t s) {
    klaunch(scan_kernel, dim3((E + 1 + 31) / 32), dim3(kSortThreads), s, E, o);
    klaunch(place_kernel<Id>, dim3(o.chunks), dim3(kSortThreads), s, ids, P, E, k, o);
    return hipGetLastError();
}

}  // namespace

// At most kMaxChunks of multiples of 32 tokens: a pass of a workgroup with groups of up to 256 experts, four passes with
// more, half of one without groups; a single one of up to 64 tokens, whose workgroup orders the pairs itself.  Router and order of 64 / 128 / 256 tokens of six pairs by one workgroup 8.8 /
// 13.6 / 23.1 us, by several and two more launches 13.8 / 13.7 / 14.1.
int32_t order_chunk(int64_t tokens) {
    const int64_t each = (tokens + kMaxChunks - 1) / kMaxChunks;
    return tokens <= 64 ? 64 : (int32_t)((each < 32 ? 32 : each) + 31) / 32 * 32;
}

hipError_t launch_route(int dt, const RouteArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + a.o.chunk - 1) / a.o.chunk));
    const dim3 block(kRouteThreads);
    auto go = [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto pick = [&](auto soft) {
            constexpr bool SOFT = decltype(soft)::value;
            // groups are scored by a lane each, and a wave's keys have to fit its LDS: 16 lanes a token up to 256 experts
            // (8192 x 256 bf16 12.9 us, with 64 lanes 34.4), 64 beyond
            if (a.groups == 1) klaunch(route_kernel<DT, 8, false, SOFT>, grid, block, s, a);
            else if (a.E <= 256) klaunch(route_kernel<DT, 16, true, SOFT>, grid, block, s, a);
            else klaunch(route_kernel<DT, 64, true, SOFT>, grid, block, s, a);
        };
        if (a.score == kSoftmax) pick(std::true_type{});
        else pick(std::false_type{});
    };
    if (dt == kDtF32) go(std::integral_constant<int, kDtF32>{});
    else if (dt == kDtBf16) go(std::integral_constant<int, kDtBf16>{});
    else go(std::integral_constant<int, kDtF16>{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.o.perm || a.o.chunks == 1) return e;
    return place(a.ids, (int64_t)a.T * a.k, a.E, a.k, a.o, s);
}

hipError_t launch_route_grad(int dt, const RouteArgs &a, hipStream_t s) {
    const bool dense = a.score == kSoftmax && !a.renorm;
    const uintptr_t at = (uintptr_t)a.logits | (uintptr_t)a.dlogits;
    // accesses of four elements: 65536 x 256 bf16 21.6 us against 25.5 (softmax), 12.2 against 14.2 (sigmoid)
    const bool four = (a.E | a.ld | a.d_ld) % 4 == 0 && at % (dt == kDtF32 ? 16 : 8) == 0;
    auto go = [&](auto d_c, auto dense_c, auto v_c) {
        constexpr int DT = decltype(d_c)::value, V = decltype(v_c)::value;
        constexpr bool DENSE = decltype(dense_c)::value;
        auto with = [&](auto k, int tokens) {
            const int64_t blocks = (a.T + tokens - 1) / tokens;
            klaunch(k, dim3((unsigned)(blocks > 4096 ? 4096 : blocks)), dim3(kGradThreads), s, a);
        };
        // 65536 x 64 bf16 softmax with 4 / 16 experts a lane: 11.7 / 17.0 us; x 256 with 16 / 64 lanes a token: 21.6 / 67
        if (a.E <= 64) with(route_grad_kernel<DT, 16, 4, V, DENSE>, 16);
        else if (a.E <= 256) with(route_grad_kernel<DT, 16, 16, V, DENSE>, 16);
        else with(route_grad_kernel<DT, 64, 16, V, DENSE>, 4);
    };
    auto pick = [&](auto d_c) {
        constexpr std::integral_constant<int, 1> one{};
        constexpr std::integral_constant<int, 4> some{};
        if (dense) four ? go(d_c, std::true_type{}, some) : go(d_c, std::true_type{}, one);
        else four ? go(d_c, std::false_type{}, some) : go(d_c, std::false_type{}, one);
    };
    if (dt == kDtF32) pick(std::integral_constant<int, kDtF32>{});
    else if (dt == kDtBf16) pick(std::integral_constant<int, kDtBf16>{});
    else pick(std::integral_constant<int, kDtF16>{});
    return hipGetLastError();
}

hipError_t launch_sort_pairs(const void *ids, bool wide, int64_t tokens, int32_t k, int32_t E, const PairOrder &o,
                             hipStream_t s) {
    const dim3 grid(o.chunks), block(kSortThreads);
    const int64_t P = tokens * k;
    if (wide) klaunch(count_kernel<int64_t>, grid, block, s, (const int64_t *)ids, P, (int)E, (int)k, o);
    else klaunch(count_kernel<int32_t>, grid, block, s, (const int32_t *)ids, P, (int)E, (int)k, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || o.chunks == 1) return e;
    return wide ? place((const int64_t *)ids, P, E, k, o, s) : place((const int32_t *)ids, P, E, k, o, s);
}

}  // namespace qrmoe
