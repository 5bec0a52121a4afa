// Routing of tokens to experts, and the grouping of rows.
//
// For each token, from its E logits l:
//   s = softmax(l) or 1 / (1 + exp(-l)),  c = s + bias
//   the experts lie in `groups` runs; a run's value is the sum of its group_top (1 or 2)
//   largest c; the top_groups best runs keep their experts
//   ids = the top_k largest c of those, in descending order (ties: the lower index first)
//   weights = scale * s[ids], divided by the sum of the chosen s on request
// then the (token, choice) pairs sorted by expert (group.cuh): what the ragged matmul
// takes its rows by.
//
// One warp per token.  A lane holds ceil(E / 32) neighbouring experts in registers, so
// runs are whole lanes and the lowest lane with the largest key has the lowest index.
// A key is a score's bits mapped to an unsigned number in the same order (NaN above
// all), its lowest bits replaced by the expert's slot in the lane.  Each lane sorts its
// keys (a network of minima and maxima); a round of the selection is then one warp
// maximum and one ballot, and the winning lane moves its keys up.
//
// Which expert is chosen is decided as the exact scores decide it.  Keys carry an
// error: the replaced bits, and where a bias makes the scores themselves be compared
// (without one their order is the logits', which are compared instead) their rounding,
// bounded below (`bound`).  Where two neighbours of the chosen order are nearer than
// that, the last choice and the best expert that stays behind among them, the choices and that
// expert are scored and ranked again as pairs of fp32 (refine), and so are the runs where the worst
// kept and the best dropped one are (near_groups).  Experts whose keys agree stand in any order, so the
// last choice is also compared with the key behind that expert, which bounds all the others;
// where that is as near, or pairs do not tell, the token is chosen in fp64 after all tokens
// (choose_exact).
//
// Instructions and latency bound it: 16384 tokens of 256 experts in fp32, 8 of 8 runs' 4, sigmoid and
// bias, 33 us, of which the placing of the pairs in a second launch is 5; 1000 instructions a
// token, 53 % of the issue slots.  One token 5.7 us, 64 6.3, 1013 of 160 experts 13.8.  Where
// nothing tells experts apart (logits of 0, groups by their two best) every token is decided in
// fp64: 16384 tokens 470 to 650 us, 64 76, one 36.
#include <algorithm>
#include <cstdio>

#include "../../include/w8a8_block_fp8.h"
#include "group.cuh"
#include "kernels.cuh"
#include "pair32.cuh"
#include "ptx.cuh"

namespace w8a8 {
w8a8_status record_error(w8a8_status st, const char *message);

namespace {

using namespace grp;

struct RouteParams {
    const void *logits;         // [T, ld]
    const float *bias;          // [E] or null
    const uint8_t *valid;       // [T] or null
    int *ids;                   // [T, k]
    float *weights;             // [T, k]
    long long T, ld;
    int E, k;
    int per;                    // experts of a lane
    int groups, top_groups, group_top;
    int group_lanes;            // lanes of a run where runs are whole lanes, a power of two; else 0
    int group_shift;            // its logarithm
    int sigmoid, renormalize;
    int vec;                    // a lane's logits can be loaded by 16 bytes
    float scale;
    int most;                   // tokens of a CTA at most
    GroupOut out;
};

constexpr uint32_t kAll = 0xffffffffu;

// Order-preserving maps; key 0 belongs to no number.  The addition makes -0 +0 and any NaN the
// canonical one, whose sign is plus: it ranks above infinity.
__device__ __forceinline__ uint32_t key_of_sum(float f)     // of a number that is a sum already
{
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t key_of(float f) { return key_of_sum(f + 0.f); }
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long key_of(double f)
{
    const unsigned long long u = __double_as_longlong(f + 0.0);
    return f != f ? ~0ull : u ^ (static_cast<unsigned long long>(static_cast<long long>(u) >> 63) | (1ull << 63));
}
__device__ __forceinline__ double value_of(unsigned long long k)
{
    return __longlong_as_double(k >> 63 ? k ^ (1ull << 63) : ~k);
}
// (A pair's lower part decides among equal upper ones.)
__device__ __forceinline__ unsigned long long key_of(Pair32 v)
{
    return static_cast<unsigned long long>(key_of(v.h)) << 32 | key_of(v.h == v.h ? v.l : 0.f);
}
__device__ __forceinline__ Pair32 pair_of(unsigned long long k)
{
    return {value_of(static_cast<uint32_t>(k >> 32)), value_of(static_cast<uint32_t>(k))};
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<unsigned long long>(hi) << 32 | lo;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d /= 2)
        v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d; d /= 2)
        v += __shfl_xor_sync(kAll, v, d);
    return v;
}

__device__ __forceinline__ float exp2_fast(float x)         // within 2 units of 2^-23
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x)          // within 1 unit
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504f;

// 0! .. 12!, inverted
__constant__ double kInverseFactorial[13] = {1.,           1.,            1. / 2.,       1. / 6.,       1. / 24.,
                                             1. / 120.,    1. / 720.,     1. / 5040.,    1. / 40320.,   1. / 362880.,
                                             1. / 3628800., 1. / 39916800., 1. / 479001600.};

// ln 2 as its first 40 bits, whose products with a quotient of up to 11 bits are exact, and the
// number nearest to the rest, which leaves 2^-102.
constexpr double kLn2High = 0x1.62e42fefa2p-1, kLn2Low = 0x1.9ef35793c7673p-41;

// exp of four numbers in fp64, to a few units of 2^-53, zero below -708: reduced by
// multiples of ln 2 in two parts (after W. J. Cody and W. Waite, "Software Manual for the
// Elementary Functions", 1980), then the power series up to f^13 / 13!, whose next term is
// below 2^-57.  Short and four at a time, because what decides a near tie once in
// thousands of tokens is never in the instruction cache, and fp64's latency is long: with
// the library's function unrolled over a lane's experts such a token took its warp 20 us.
constexpr int kQuad = 4;
__device__ __forceinline__ void exp64(double (&x)[kQuad])
{
    const double kMagic = 6755399441055744.;            // 1.5 2^52: the sum's low bits are the rounded quotient
    double f[kQuad], s[kQuad];
    int n[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        const double in = fmin(fmax(x[i], -708.), 709.);                // (a NaN is put back below)
        const double t = fma(in, 1.4426950408889634, kMagic), q = t - kMagic;
        f[i] = fma(q, -kLn2Low, fma(q, -kLn2High, in));
        n[i] = __double2loint(t);
        s[i] = 1. / 6227020800.;
    }
#pragma unroll 1
    for (int k = 12; k >= 0; --k) {
        const double c = kInverseFactorial[k];
#pragma unroll
        for (int i = 0; i < kQuad; ++i)
            s[i] = fma(s[i], f[i], c);
    }
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        const double v = __longlong_as_double(__double_as_longlong(s[i]) + (static_cast<long long>(n[i]) << 52));
        x[i] = x[i] != x[i] ? x[i] : x[i] < -708. ? 0. : x[i] > 709. ? INFINITY : v;
    }
}
// 1 / d for d from 1 to 2^20: two steps of Newton's method from fp32
__device__ __forceinline__ double inverse64(double d)
{
    double r = static_cast<double>(rcp_fast(static_cast<float>(d)));
    r = fma(r, fma(-d, r, 1.), r);
    return fma(r, fma(-d, r, 1.), r);
}

// (debug-bounds build: whether an access lies in its buffer)
template <int KIND> __device__ __forceinline__ bool is_logit(const RouteParams &p, const void *at, int bytes)
{
    return in_bounds(inside(at, bytes, p.logits, span(p.T, p.ld, p.E, KIND == W8A8_IN_FP32 ? 4 : 2)), p.out.status,
                     SITE_BOUNDS_A);
}
__device__ __forceinline__ bool is_expert(const RouteParams &p, int e)
{
    return in_bounds(e >= 0 && e < p.E, p.out.status, SITE_BOUNDS_B);
}
__device__ __forceinline__ float bias_of(const RouteParams &p, int e) { return is_expert(p, e) ? p.bias[e] : 0.f; }
__device__ __forceinline__ bool is_valid(const RouteParams &p, long long token)
{
    return !p.valid || (in_bounds(token >= 0 && token < p.T, p.out.status, SITE_BOUNDS_B) && p.valid[token]);
}
// (of the numbers that a CTA keeps)
__device__ __forceinline__ bool is_kept(const RouteParams &p, int i)
{
    return in_bounds(i >= 0 && i < p.most * p.k, p.out.status, SITE_BOUNDS_SMEM);
}

template <int KIND> __device__ __forceinline__ float load_logit(const RouteParams &p, const void *row, int e)
{
    constexpr int kBytes = KIND == W8A8_IN_FP32 ? 4 : 2;
    if (!is_logit<KIND>(p, static_cast<const char *>(row) + e * static_cast<long long>(kBytes), kBytes))
        return 0.f;
    if constexpr (KIND == W8A8_IN_FP32)
        return static_cast<const float *>(row)[e];
    else if constexpr (KIND == W8A8_IN_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
    else
        return __half2float(static_cast<const __half *>(row)[e]);
}

// A lane's logits, -infinity past E.
template <int KIND, int PER>
__device__ __forceinline__ void load_lane(const RouteParams &p, const void *row, int e0, float (&l)[PER])
{
    constexpr int kEach = KIND == W8A8_IN_FP32 ? 4 : 8;         // elements of 16 bytes
    if constexpr (PER % kEach == 0) {
        if (p.vec && PER == p.per) {
#pragma unroll
            for (int i = 0; i < PER; i += kEach) {
                uint4 w = make_uint4(0, 0, 0, 0);
                const bool in = e0 + i < p.E;
                if (in && is_logit<KIND>(p, static_cast<const char *>(row) + (e0 + i) * (16 / kEach), 16))
                    w = *reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (e0 + i) * (16 / kEach));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    float f;
                    if constexpr (KIND == W8A8_IN_FP32)
                        f = __uint_as_float(u[j]);
                    else if constexpr (KIND == W8A8_IN_BF16)
                        f = __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
                    else {
                        const __half2 h = *reinterpret_cast<const __half2 *>(&u[j >> 1]);
                        f = __half2float(j & 1 ? h.y : h.x);
                    }
                    l[i + j] = in ? f : -INFINITY;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        l[i] = i < p.per && e0 + i < p.E ? load_logit<KIND>(p, row, e0 + i) : -INFINITY;
}

// Descending order by odd-even merging (K. E. Batcher, "Sorting networks and their
// applications", AFIPS Spring Joint Computer Conference, 1968).
template <int N> __device__ __forceinline__ void sort_keys(uint32_t (&k)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (j + i + q < N && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
                        const uint32_t a = k[j + i], b = k[j + i + q];
                        k[j + i] = max(a, b);
                        k[j + i + q] = min(a, b);
                    }
}

// The two largest keys of a lane's experts, then of the lanes of its run.
template <class K> __device__ __forceinline__ void two_best(K &a, K &b, K x)
{
    const K lo = x < a ? x : a;
    a = x < a ? a : x;
    b = lo < b ? b : lo;
}

// Whether this lane's run g is kept, from its value (the same in all of its group_lanes
// lanes, a power of two), and the values at the border.  Each lane compares with its share
// of the runs.
template <class K>
__device__ __forceinline__ bool rank_groups(int groups, int group_lanes, int top, int g, K value, K *kept, K *dropped)
{
    const int share = (groups + group_lanes - 1) / group_lanes, from = (threadIdx.x & (group_lanes - 1)) * share;
    int above = 0;
    for (int i = 0; i < share; ++i) {
        const int j = from + i;
        const K v = __shfl_sync(kAll, value, min(j, groups - 1) * group_lanes);
        above += j < groups && (v > value || (v == value && j < g));
    }
    for (int d = 1; d < group_lanes; d *= 2)
        above += __shfl_xor_sync(kAll, above, d);
    const bool keep = g < groups && above < top;
    *kept = ~warp_max(keep ? ~value : K(0));
    *dropped = warp_max(keep || g >= groups ? K(0) : value);
    return keep;
}

template <class K> __device__ __forceinline__ K group_value(int group_top, K a, K b)
{
    return group_top == 2 ? key_of(value_of(a) + value_of(b)) : a;
}

// A softmax's sum in fp64 (1 for a sigmoid).
template <int KIND> __device__ __forceinline__ double softmax_sum(const RouteParams &p, const void *row, float m)
{
    if (p.sigmoid)
        return 1.;
    double z = 0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.E; e += 32 * kQuad) {
        double x[kQuad];
#pragma unroll
        for (int i = 0; i < kQuad; ++i)
            x[i] = e + 32 * i < p.E ? static_cast<double>(load_logit<KIND>(p, row, e + 32 * i)) - m : -1000.;
        exp64(x);
#pragma unroll
        for (int i = 0; i < kQuad; ++i)
            z += x[i];
    }
    return warp_sum(z);
}
// Scores of four logits, in their place.
__device__ __forceinline__ void score64(const RouteParams &p, double (&l)[kQuad], float m, double z)
{
    double e[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i)
        e[i] = p.sigmoid ? -fabs(l[i]) : l[i] - m;
    exp64(e);
    const double inv = p.sigmoid || z == 0 ? 0. : inverse64(z);
#pragma unroll
    for (int i = 0; i < kQuad; ++i) {
        if (p.sigmoid) {
            const double q = inverse64(1. + e[i]);
            l[i] = l[i] != l[i] ? l[i] : l[i] >= 0 ? q : e[i] * q;
        } else {
            l[i] = z == 0 ? 0. : e[i] * inv;
        }
    }
}

// The same as pairs of fp32.  Their scores are off by less than 2^-42, and sums with
// a bias by 2^-46 of their sizes: below kPairError (1 + the size).
constexpr float kPairError = 0x1p-40f;
template <int KIND> __device__ __forceinline__ Pair32 softmax_sum_pair(const RouteParams &p, const void *row, float m)
{
    Pair32 z = {0.f, 0.f};
    if (p.sigmoid)
        return z;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.E; e += 32)
        z = z + exp_pair(two_sum(load_logit<KIND>(p, row, e), -m));
#pragma unroll
    for (int d = 16; d; d /= 2) {
        const float h = __shfl_xor_sync(kAll, z.h, d), l = __shfl_xor_sync(kAll, z.l, d);
        // (the same in every lane: the lower lane's part first)
        z = threadIdx.x & d ? Pair32{h, l} + z : z + Pair32{h, l};
    }
    return z;
}
__device__ __forceinline__ Pair32 score_pair(const RouteParams &p, float l, float m, Pair32 z)
{
    if (p.sigmoid)
        return sigmoid(l);
    return z.h == 0.f ? z : exp_pair(two_sum(l, -m)) * inverse(z);
}

// The choice in fp64: lane j < k gets the j-th expert.  Rare, so one version for every
// E, its arrays in local memory.
template <int KIND> __device__ __noinline__ int choose_exact(const RouteParams &p, const void *row)
{
    using K = unsigned long long;
    const int lane = threadIdx.x & 31, e0 = lane * p.per, n = max(0, min(p.per, p.E - e0));
    K key[32], ck[32];
    float m = -INFINITY;
    for (int i = 0; i < n; ++i)
        m = fmaxf(m, load_logit<KIND>(p, row, e0 + i));
    m = value_of(warp_max(key_of(m)));
    m = m == -INFINITY ? 0.f : m;
    const double z = softmax_sum<KIND>(p, row, m);
    for (int i = 0; i < n; i += kQuad) {
        double x[kQuad], l[kQuad];
        for (int j = 0; j < kQuad; ++j)
            x[j] = l[j] = load_logit<KIND>(p, row, e0 + min(i + j, n - 1));
        score64(p, x, m, z);
        for (int j = 0; j < kQuad && i + j < n; ++j) {
            ck[i + j] = key_of(p.bias ? x[j] + bias_of(p, e0 + i + j) : x[j]);
            key[i + j] = p.bias ? ck[i + j] : key_of(l[j]);
        }
    }
    if (p.groups > 1) {
        const int size = p.E / p.groups;
        // every lane goes through every run's experts: no rule on sizes
        uint32_t keep = 0;
        K value = 0;
        for (int g = 0; g < p.groups; ++g) {
            K a = 0, b = 0;
            for (int i = 0; i < n; ++i)
                if ((e0 + i) / size == g)
                    two_best(a, b, p.group_top == 2 ? ck[i] : key[i]);
            const K top = warp_max(a);
            const uint32_t who = __ballot_sync(kAll, a == top);
            const K second = warp_max(lane == __ffs(who) - 1 ? b : a);
            const K v = group_value(p.group_top, top, second);
            value = lane == g ? v : value;
        }
        K kept, dropped;
        const bool mine = rank_groups<K>(p.groups, 1, p.top_groups, lane, value, &kept, &dropped);
        keep = __ballot_sync(kAll, mine);
        for (int i = 0; i < n; ++i)
            if (!(keep >> ((e0 + i) / size) & 1))
                key[i] = 0;
    }
    int id = 0;
    for (int j = 0; j < p.k; ++j) {
        K best = 0;
        int slot = 0;
        for (int i = 0; i < n; ++i)
            if (key[i] > best)
                best = key[i], slot = i;
        const K top = warp_max(best);
        const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
        const int e = __shfl_sync(kAll, e0 + slot, src);
        if (lane == src)
            key[slot] = 0;
        if (lane == j)
            id = e;
    }
    return id;
}

// The runs that are kept, as bits, from scores in pairs of fp32; *sure: whether they tell.
template <int KIND>
__device__ __forceinline__ uint32_t near_groups(const RouteParams &p, const void *row, float m, bool *sure)
{
    using K = unsigned long long;
    const int lane = threadIdx.x & 31, e0 = lane * p.per, n = max(0, min(p.per, p.E - e0)), size = p.E / p.groups;
    const Pair32 z = softmax_sum_pair<KIND>(p, row, m);
    K value = 0, a = 0, b = 0;
    auto key = [&](int e) {
        const float l = load_logit<KIND>(p, row, e);
        if (!p.bias && p.group_top == 1)
            return key_of(Pair32{l, 0.f});
        const Pair32 s = score_pair(p, l, m, z);
        return key_of(p.bias ? s + Pair32{bias_of(p, e), 0.f} : s);
    };
    auto value_of_run = [&](K first, K second) {
        return p.group_top == 2 ? key_of(pair_of(first) + pair_of(second)) : first;
    };
    float most = 0.f;
    if (p.group_lanes) {
#pragma unroll 1
        for (int i = 0; i < n; ++i)
            two_best(a, b, key(e0 + i));
        for (int d = 1; d < p.group_lanes; d *= 2) {
            const K oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
            two_best(a, b, oa);
            b = ob > b ? ob : b;
        }
        most = n ? fabsf(pair_of(a).h) + (p.group_top == 2 ? fabsf(pair_of(b).h) : 0.f) : 0.f;
        const K mine = value_of_run(a, b);
        value = __shfl_sync(kAll, mine, min(lane, p.groups - 1) * p.group_lanes);
    } else if (lane < p.groups) {
        for (int i = 0; i < size; ++i)
            two_best(a, b, key(lane * size + i));
        most = fabsf(pair_of(a).h) + (p.group_top == 2 ? fabsf(pair_of(b).h) : 0.f);
        value = value_of_run(a, b);
    }
    __syncwarp();
    K kept, dropped;
    const bool keep = rank_groups<K>(p.groups, 1, p.top_groups, lane, value, &kept, &dropped);
    most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(most)));
    const Pair32 hi = pair_of(kept), lo = pair_of(dropped);
    *sure = (hi.h - lo.h) + (hi.l - lo.l) > 4.f * kPairError * (1.f + most);
    return __ballot_sync(kAll, keep);
}

// Ranks `count` (at most 32) experts, lane j's being id, by their scores: returns the expert
// of rank `lane`.  *sure: whether pairs of fp32 tell neighbours apart.
template <class K> __device__ __forceinline__ int by_rank(K key, int id, int count, K *sorted)
{
    const int lane = threadIdx.x & 31;
    int above = 0;
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
        const K other = __shfl_sync(kAll, key, j);
        const int other_id = __shfl_sync(kAll, id, j);
        above += other > key || (other == key && other_id < id);
    }
    int mine = id;
    K its = key;
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
        const int rank = __shfl_sync(kAll, above, j), e = __shfl_sync(kAll, id, j);
        const K k = __shfl_sync(kAll, key, j);
        mine = rank == lane ? e : mine;
        its = rank == lane ? k : its;
    }
    *sorted = its;
    return mine;
}
template <int KIND>
__device__ __forceinline__ int refine(const RouteParams &p, const void *row, int id, int count, float m, bool *sure)
{
    using K = unsigned long long;
    const int lane = threadIdx.x & 31;
    const bool in = lane < count;
    const float l = in ? load_logit<KIND>(p, row, id) : 0.f;
    Pair32 c = {l, 0.f};                    // without a bias the logits rank
    if (p.bias) {
        const Pair32 z = softmax_sum_pair<KIND>(p, row, m);
        c = score_pair(p, l, m, z) + Pair32{in ? bias_of(p, id) : 0.f, 0.f};
    }
    K sorted;
    const int ranked = by_rank<K>(in ? key_of(c) : 0ull, id, count, &sorted);
    const K next = __shfl_down_sync(kAll, sorted, 1);
    const int next_id = __shfl_down_sync(kAll, ranked, 1);
    bool near = false;
    if (p.bias && lane + 1 < count) {
        const Pair32 x = pair_of(sorted), y = pair_of(next);
        near = !((x.h - y.h) + (x.l - y.l) > 2.f * kPairError * (1.f + fabsf(x.h)));
        // equal logits under equal biases are equal scores, in order of their index
        near = near && !(load_logit<KIND>(p, row, ranked) == load_logit<KIND>(p, row, next_id) && bias_of(p, ranked) == bias_of(p, next_id));
    }
    *sure = !__any_sync(kAll, near);
    return ranked;
}

// Shared memory of k_route beside the sort's.
struct RouteSmem {
    uint2 *won;                 // of a warp [batch, k + 1]: the choices' keys and experts, then what is behind
    uint32_t *hard;             // of a warp [32]: bits of its tokens that are left to fp64
    float4 *row;                // of a warp [batch]: a softmax's m and z, a score's bound, the key behind all
    float *bias;                // [32 per]
    int *run_keys;              // of a warp [E], where runs are not whole lanes
    static constexpr int kWon = 64;                     // 32 / k (k + 1) at most
    static __host__ __device__ size_t bytes(const RouteParams &p)
    {
        return kWarps * (sizeof(float4) * 32 + sizeof(uint2) * kWon + sizeof(uint32_t) * 32) + sizeof(float) * 32 * p.per +
               (p.groups > 1 && !p.group_lanes ? sizeof(int) * kWarps * p.E : 0);
    }
    __device__ __forceinline__ RouteSmem(const RouteParams &p, const GroupSmem &s, int warp)
    {
        float4 *const rows = reinterpret_cast<float4 *>(s.pairs + (p.most * p.k + 3) / 4 * 4);
        uint2 *const keys = reinterpret_cast<uint2 *>(rows + 32 * kWarps);
        row = rows + 32 * warp;
        won = keys + kWon * warp;
        uint32_t *const bits = reinterpret_cast<uint32_t *>(keys + kWon * kWarps);
        hard = bits + 32 * warp;
        bias = reinterpret_cast<float *>(bits + 32 * kWarps);
        run_keys = reinterpret_cast<int *>(bias + 32 * p.per) + warp * p.E;
    }
};

// A score as make_keys makes it.
__device__ __forceinline__ float score32(const RouteParams &p, float l, float m, float z)
{
    return p.sigmoid ? rcp_fast(1.f + exp2_fast(-kLog2e * l))
                     : exp2_fast(kLog2e * (l - m)) * (z == 0.f ? 0.f : rcp_fast(z));
}

// A token's scores as a lane's keys: sorted, of the open runs, and what the weights need.
template <int PER> struct Keys {
    static constexpr uint32_t kSlots = PER - 1;
    uint32_t key[PER];
    float m, z;                 // softmax: the largest logit (0 for -infinity) and the sum
    float bound;                // of a score's error
    bool hard;                  // which runs are open is left to fp64
};

template <int KIND, int PER>
__device__ __forceinline__ void make_keys(const RouteParams &p, const void *row, const float (&l)[PER], const float *bias,
                                          int *run_keys, Keys<PER> &out)
{
    constexpr uint32_t kSlots = Keys<PER>::kSlots;
    const int lane = threadIdx.x & 31, e0 = lane * p.per;
    const bool biased = p.bias != nullptr, sums = p.groups > 1 && p.group_top == 2;
    const bool scored = biased || sums || (!p.sigmoid && !p.renormalize);
    float c[PER];
    float m = 0.f, z = 1.f;
    // An upper bound of the error of an fp32 score, in units of 2^-23.  An exponential of x
    // is off by 2 units and by its argument's rounding, 0.75 |x|, relatively.
    //   sigmoid: s (1 - s) (2 + 0.75 |l|) <= 0.6 units, then one rounded sum and the
    //     quotient: 2.1 units, below 17/16 2^-22.
    //   softmax: with u = -x the terms' errors are at most 2 units of the largest term and,
    //     in the sum z, 2 + 0.75 u averaged with the terms as weights, where u averages at
    //     most ln E + 1 < 8; the sum's roundings (PER + 5) / 2 <= 18.5, the quotient 1.5: with
    //     s <= 1 / z at most 30 units of 1 / z, below 2^-18 / z.
    float bound = 0x1.1p-22f;
    if (scored) {
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                c[i] = rcp_fast(1.f + exp2_fast(-kLog2e * l[i]));
        } else {
            m = l[0];
#pragma unroll
            for (int i = 1; i < PER; ++i)
                m = fmaxf(m, l[i]);
            m = value_of(warp_max(key_of(m)));
            m = m == -INFINITY ? 0.f : m;
            z = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                z += c[i] = exp2_fast(kLog2e * (l[i] - m));
            z = warp_sum(z);
            const float inv = z == 0.f ? 0.f : rcp_fast(z);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                c[i] *= inv;
            bound = 0x1p-18f * inv;
        }
    }
    uint32_t (&key)[PER] = out.key;
    out.hard = false;
    const int mine = min(p.per, p.E - e0);      // experts of this lane
    if (biased) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] += i < p.per ? bias[i] : 0.f;
            key[i] = i < mine ? key_of_sum(c[i]) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = i < mine ? key_of(l[i]) : 0u;
    }
    if (p.groups > 1) {
        const int size = p.E / p.groups;
        uint32_t a = 0, b = 0, kept, dropped;
        const bool by_score = sums && !biased;          // (keys are the logits')
        bool keep;
        if (p.group_lanes) {
            if (by_score) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    two_best(a, b, i < mine ? key_of_sum(c[i]) : 0u);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    two_best(a, b, key[i]);
            }
            for (int d = 1; d < p.group_lanes; d *= 2) {
                const uint32_t oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
                two_best(a, b, oa);
                b = ob > b ? ob : b;
            }
            keep = rank_groups<uint32_t>(p.groups, p.group_lanes, p.top_groups, lane >> p.group_shift,
                                         group_value(p.group_top, a, b), &kept, &dropped);
        } else {
            // runs that do not begin with a lane: through shared memory, lane g takes run g
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i])
                    run_keys[e0 + i] = static_cast<int>(by_score ? key_of_sum(c[i]) : key[i]);
            __syncwarp();
            if (lane < p.groups)
                for (int i = 0; i < size; ++i)
                    two_best(a, b, static_cast<uint32_t>(run_keys[lane * size + i]));
            __syncwarp();
            keep = rank_groups<uint32_t>(p.groups, 1, p.top_groups, lane, group_value(p.group_top, a, b), &kept, &dropped);
        }
        bool near_group = false;        // which runs are open is nearer than the scores' errors
        if ((biased || sums) && p.top_groups < p.groups) {
            // Each value is off by two scores' errors, their sums' with the biases and the sum of
            // both: 2 bound + 2^-23 of the scores' sizes, taken as the largest run's.
            const float sizes = p.group_lanes || lane < p.groups ? fabsf(value_of(a)) + (sums ? fabsf(value_of(b)) : 0.f) : 0.f;
            const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(sizes)));
            near_group = !(value_of(kept) - value_of(dropped) > 4.f * bound + 0x1p-22f * most);
        }
        uint32_t open = 0;
        if (near_group) {
            bool sure;
            open = near_groups<KIND>(p, row, m, &sure);
            out.hard = !sure;
        }
        if (p.group_lanes) {
            if (near_group)
                keep = open >> (lane >> p.group_shift) & 1;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = keep ? key[i] : 0u;
        } else {
            const uint32_t lanes = __ballot_sync(kAll, keep);
            if (!near_group)
                open = lanes;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = open >> ((e0 + i) / size & 31) & 1 ? key[i] : 0u;
        }
    }
    // The slot takes the place of the key's lowest bits; 16-bit logits have zeros there.
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = key[i] ? (key[i] & ~kSlots) | (kSlots - i) : 0u;
    sort_keys(key);
    out.m = m;
    out.z = z;
    out.bound = bound;
}

__device__ __forceinline__ uint32_t lanes_below()
{
    uint32_t m;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
    return m;
}

// The best key that is left goes to *won with its expert, and from its lane; returns it.
template <int PER> __device__ __forceinline__ uint32_t take_best(uint32_t (&key)[PER], int e0, uint2 *won)
{
    constexpr uint32_t kSlots = PER - 1;
    // (the lane before the slot: the lower index first)
    const uint32_t bits = key[0] & ~kSlots, top = warp_max(bits);
    const uint32_t best = __ballot_sync(kAll, bits == top);
    if (bits == top && (best & lanes_below()) == 0) {
        *won = make_uint2(top, e0 + kSlots - (key[0] & kSlots));
#pragma unroll
        for (int i = 0; i + 1 < PER; ++i)
            key[i] = key[i + 1];
        key[PER - 1] = 0;
    }
    return top;
}

// Whether key a is not surely above key b, and so above whatever has b's kept bits or less: they
// differ by no more than `by` and `at` times their sizes, which is the errors of both scores and the bits
// that the keys lack.  (Without a bias, by and at 0: sure where the kept bits differ.)
template <int PER> struct Near {
    float by, at;
    __device__ __forceinline__ Near(bool biased, float bound)
        : by(biased ? 2.f * bound : 0.f), at(biased ? 0x1p-22f + PER * 0x1p-23f : 0.f)
    {
    }
    __device__ __forceinline__ bool operator()(uint32_t a, uint32_t b) const
    {
        constexpr uint32_t kSlots = PER - 1;
        const float hi = value_of(a & ~kSlots), lo = value_of(b & ~kSlots);
        return b > kSlots && !(hi - lo > by + at * (fabsf(hi) + fabsf(lo)));
    }
};

// The weight of a lane's choice, of k lanes from `first` on, from its logit, in full fp32; m
// and z are a softmax's.
__device__ __forceinline__ float weigh(const RouteParams &p, float x, int first, float m, float z)
{
    float w;
    if (p.renormalize) {
        // relative to the largest of them, so that small scores keep their ratios
        float top = -INFINITY;
        for (int j = 0; j < p.k; ++j)
            top = fmaxf(top, __shfl_sync(kAll, x, first + j));      // (leaves NaN aside)
        if (p.sigmoid) {
            top = fminf(top, 0.f);
            const float e = expf(-fabsf(x));        // 1 / (1 + exp(-x)) over exp(top)
            w = (x > 0.f ? 1.f : top == 0.f ? e : expf(x - top)) / (1.f + e);
            w = x != x ? x : w;
        } else {
            w = expf(x - top);
        }
        if (top == -INFINITY && x == -INFINITY)
            w = 0.f;            // (-infinity) - (-infinity)
        float sum = 0.f;
        for (int j = 0; j < p.k; ++j)
            sum += __shfl_sync(kAll, w, first + j);
        w = sum == 0.f ? 0.f : w / sum;
        if (!p.sigmoid && z != z)
            w = z;              // a NaN or an infinity in the row that was not chosen
    } else {
        w = p.sigmoid ? 1.f / (1.f + expf(-x)) : z == 0.f ? 0.f : expf(x - m) / z;
    }
    return w * p.scale;
}

template <int KIND, int PER> __global__ void __launch_bounds__(kThreads, PER <= 8 ? 2 : 1) k_route(const RouteParams p)
{
    extern __shared__ int smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = p.E + 1, e0 = lane * p.per;
    const GroupSmem s = carve(smem, bins);
    RouteSmem r(p, s, warp);
    const float *const bias = r.bias + e0;
    clear_hist(s, bins);
    grid_dependency_wait();
    grid_launch_dependents();
    if (p.bias) {
        for (int e = threadIdx.x; e < 32 * p.per; e += kThreads)
            r.bias[e] = e < p.E ? bias_of(p, e) : 0.f;
        __syncthreads();
    }
    // the CTA's tokens, and this warp's of them
    const int ctas = gridDim.x, cta = blockIdx.x;
    const long long cta_first = piece(p.T, ctas, cta);
    const int tokens = static_cast<int>(piece(p.T, ctas, cta + 1) - cta_first);
    const int lo = tokens * warp / kWarps, hi = tokens * (warp + 1) / kWarps;
    constexpr int kBytes = KIND == W8A8_IN_FP32 ? 4 : 2;
    const long long pitch = p.ld * kBytes;
    const char *const rows = static_cast<const char *>(p.logits) + cta_first * pitch;
    constexpr bool kAhead = PER <= 8;           // the next token's logits, while registers last
    float next[kAhead ? PER : 1];
    if constexpr (kAhead)
        if (lo < hi)
            load_lane<KIND, PER>(p, rows + lo * pitch, e0, next);
    // As many tokens at a time as have 32 choices: the choices one after the other, then
    // their check, the weights and the counts with a lane to each.
    const bool checked = p.bias || KIND == W8A8_IN_FP32;
    const int batch = 32 / p.k, in_batch = lane / p.k, choice = lane - in_batch * p.k;
    bool any_hard = false;
    r.hard[lane] = 0;
    for (int i0 = lo; i0 < hi; i0 += batch) {
        const int here = min(batch, hi - i0);
        uint32_t near_tokens = 0, hard_tokens = 0;
        for (int i = 0; i < here; ++i) {
            float l[PER];
            const char *const row = rows + (i0 + i) * pitch;
            if constexpr (kAhead) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    l[j] = next[j];
                if (i0 + i + 1 < hi)
                    load_lane<KIND, PER>(p, row + pitch, e0, next);
            } else {
                load_lane<KIND, PER>(p, row, e0, l);
            }
            if (!is_valid(p, cta_first + i0 + i))
                continue;
            Keys<PER> t;
            make_keys<KIND, PER>(p, row, l, bias, r.run_keys, t);
            hard_tokens |= t.hard ? 1u << i : 0u;
            uint2 *const won = r.won + i * (p.k + 1);
            // (one more where the choice is checked: the best that stays behind; and the key after it)
            for (int j = 0; j < (checked ? p.k + 1 : p.k); ++j)
                take_best(t.key, e0, won + j);
            const uint32_t after = checked ? warp_max(t.key[0]) : 0u;
            if (lane == 0)
                r.row[i] = make_float4(t.m, t.z, t.bound, __uint_as_float(after));
        }
        __syncwarp();
        const int token = i0 + in_batch;
        const bool in = in_batch < here, valid = in && is_valid(p, cta_first + token);
        const char *const row = rows + token * pitch;
        int id = p.E;
        float x = 0.f;
        if (valid) {
            const uint2 got = r.won[in_batch * (p.k + 1) + choice];
            id = static_cast<int>(got.y);
            x = load_logit<KIND>(p, row, id);
            if (checked) {
                const uint2 below = r.won[in_batch * (p.k + 1) + choice + 1];
                const float4 of = r.row[in_batch];
                const int other = static_cast<int>(below.y);
                bool near = below.x != 0;
                if (near && p.bias) {
                    // the fp32 scores anew, which the keys hold cut off: each off by the bound, and by half
                    // a unit for the sum with the bias
                    const float y = load_logit<KIND>(p, row, other);
                    const float hi = score32(p, x, of.x, of.y) + r.bias[id], lo = score32(p, y, of.x, of.y) + r.bias[other];
                    near = !(hi - lo > 2.f * of.z + 0x1p-23f * (fabsf(hi) + fabsf(lo)));
                    // equal logits under equal biases are equal scores, in order of their index
                    near = near && !(x == y && r.bias[id] == r.bias[other] && id < other && choice + 1 < p.k);
                    // what is behind that one has a key that is no larger, but may have a larger score: the
                    // last choice has to be surely above it too
                    near = near || (choice + 1 == p.k && Near<PER>(true, of.z)(got.x, __float_as_uint(of.w)));
                } else if (near) {
                    near = got.x == below.x;            // (the kept bits)
                    near = near && !(x == load_logit<KIND>(p, row, other) && id < other && choice + 1 < p.k);
                }
                near_tokens = near ? 1u << in_batch : 0u;
            }
        }
        near_tokens = __reduce_or_sync(kAll, near_tokens);
        while (near_tokens) {
            const int i = __ffs(near_tokens) - 1;
            near_tokens &= near_tokens - 1;
            const float4 of = r.row[i];
            const uint2 *const won = r.won + i * (p.k + 1);
            const char *const its = rows + (i0 + i) * pitch;
            // among the choices and the best behind them, where nothing is near that one
            const uint32_t behind = won[p.k].x;
            const int count = behind ? p.k + 1 : p.k;
            bool sure = false;
            int chosen = 0;
            if (count <= 32 && !Near<PER>(p.bias != nullptr, of.z)(behind, __float_as_uint(of.w)))
                chosen = refine<KIND>(p, its, lane < count ? static_cast<int>(won[lane].y) : 0, count, of.x, &sure);
            if (!sure) {
                hard_tokens |= 1u << i;
                continue;
            }
            const int again = __shfl_sync(kAll, chosen, choice);
            if (in_batch == i && valid) {
                id = again;
                x = load_logit<KIND>(p, row, id);
            }
        }
        if (hard_tokens) {
            any_hard = true;
            if (lane < here && hard_tokens >> lane & 1)
                atomicOr(r.hard + (i0 - lo + lane) / 32, 1u << ((i0 - lo + lane) & 31));
        }
        const float4 about = in ? r.row[in_batch] : make_float4(0.f, 1.f, 0.f, 0.f);
        const float w = weigh(p, x, in_batch * p.k, about.x, about.y);
        const bool writes = in && lane < batch * p.k;
        const long long pair = (cta_first + i0) * p.k + lane;
        if (writes && is_number(p.out, pair, SITE_BOUNDS_C)) {
            p.ids[pair] = valid ? id : -1;
            p.weights[pair] = valid ? w : 0.f;
        }
        if (writes && is_kept(p, i0 * p.k + lane))
            s.pairs[i0 * p.k + lane] = id;
        __syncwarp();
    }
    // What pairs of fp32 do not tell either.
    if (any_hard) {
        __syncwarp();
        for (int i = lo; i < hi; ++i) {
            if (!(r.hard[(i - lo) / 32] >> ((i - lo) & 31) & 1))
                continue;
            const char *const row = rows + i * pitch;
            const int id = choose_exact<KIND>(p, row);
            float m = -INFINITY, z = 0.f;
            for (int e = lane; e < p.E; e += 32)
                m = fmaxf(m, load_logit<KIND>(p, row, e));
            m = value_of(warp_max(key_of(m)));
            m = m == -INFINITY ? 0.f : m;
            for (int e = lane; e < p.E; e += 32)
                z += expf(load_logit<KIND>(p, row, e) - m);
            z = warp_sum(z);
            const float w = weigh(p, lane < p.k ? load_logit<KIND>(p, row, id) : 0.f, 0, m, z);
            const long long pair = (cta_first + i) * p.k + lane;
            if (lane < p.k && is_number(p.out, pair, SITE_BOUNDS_C) && is_kept(p, i * p.k + lane)) {
                p.ids[pair] = id;
                p.weights[pair] = w;
                s.pairs[i * p.k + lane] = id;
            }
            __syncwarp();
        }
    }
    // each choice's rank among the warp's of the same expert
    int *const h = s.hist + warp * bins;
    for (int i0 = lo * p.k; i0 < hi * p.k; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < hi * p.k;
        const int bin = in ? static_cast<int>(s.pairs[i]) : bins;
        const uint32_t same = __match_any_sync(kAll, bin), before = same & lanes_below();
        if (in)
            s.pairs[i] = static_cast<uint32_t>(bin) << 16 | (h[bin] + __popc(before));
        __syncwarp();
        if (in && !before)
            h[bin] += __popc(same);
        __syncwarp();
    }
    place_pairs(s, p.out, cta_first * p.k, lo * p.k, hi * p.k);
}

struct GroupParams {
    const int *ids;             // [n]
    GroupOut out;
};

__global__ void __launch_bounds__(kThreads) k_group(const GroupParams p)
{
    extern __shared__ int smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, groups = p.out.groups, bins = groups + 1;
    const GroupSmem s = carve(smem, bins);
    clear_hist(s, bins);
    grid_dependency_wait();
    grid_launch_dependents();
    // in units of 32 numbers
    const long long units = (p.out.n + 31) / 32;
    const long long cta_first = piece(units, gridDim.x, blockIdx.x) * 32;
    const int cta_units = static_cast<int>(piece(units, gridDim.x, blockIdx.x + 1) - cta_first / 32);
    const int count = static_cast<int>(min(p.out.n - cta_first, cta_units * 32ll));
    const int lo = min(cta_units * warp / kWarps * 32, count), hi = min(cta_units * (warp + 1) / kWarps * 32, count);
    int *const h = s.hist + warp * bins;
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        const int id = in && is_number(p.out, cta_first + i + lane, SITE_BOUNDS_A) ? p.ids[cta_first + i + lane] : 0;
        const int bin = !in ? bins : static_cast<uint32_t>(id) < static_cast<uint32_t>(groups) ? id : groups;
        const uint32_t same = __match_any_sync(kAll, bin);
        const uint32_t before = same & ((1u << lane) - 1u);
        if (in)
            s.pairs[i + lane] = static_cast<uint32_t>(bin) << 16 | (h[bin] + __popc(before));
        __syncwarp();
        if (in && !before)
            h[bin] += __popc(same);
        __syncwarp();
    }
    place_pairs(s, p.out, cta_first, lo, hi);
}

// The second launch of a sort over several clusters: places within a cluster, plus
// what earlier clusters hold.  Every cluster's numbers are shared by p.ctas CTAs.
struct PlaceParams {
    const int *ids;
    int clusters, ctas;
    long long units;            // of the first launch
    int per_unit, first_ctas;   // its numbers of a unit, and its CTAs
    GroupOut out;
};

__global__ void __launch_bounds__(kPlaceThreads) k_place(const PlaceParams p)
{
    extern __shared__ int smem[];
    const int groups = p.out.groups, bins = groups + 1;
    int *const total = smem, *const before = smem + bins, *const part = before + bins;
    const int cluster = blockIdx.x / p.ctas, slice = blockIdx.x % p.ctas;
    for (int b = threadIdx.x; b < bins; b += kPlaceThreads)
        total[b] = before[b] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    // the first number, fetched while the counts are
    const long long first = piece(p.units, p.first_ctas, cluster * kCluster) * p.per_unit + slice * kPlaceThreads + threadIdx.x;
    const long long last = min(p.out.n, piece(p.units, p.first_ctas, (cluster + 1) * kCluster) * p.per_unit);
    int id = 0, rank = 0;
    if (first < last && is_number(p.out, first, SITE_BOUNDS_A))
        id = p.ids[first], rank = p.out.rank[first];
    // Bins side by side in a warp, the clusters dealt to slices of the block.
    const int width = (bins + 31) / 32 * 32, slices = max(1, kPlaceThreads / width);
    const int mine = threadIdx.x / width;
    for (int b = threadIdx.x % width; b < bins && mine < slices; b += slices > 1 ? bins : kPlaceThreads) {
        int all = 0, early = 0;
#pragma unroll 8
        for (int c = mine; c < p.clusters; c += slices) {
            const long long at = static_cast<long long>(c) * bins + b;
            const int v = is_count(p.out, at) ? p.out.hist[at] : 0;
            all += v;
            early += c < cluster ? v : 0;
        }
        if (slices > 1) {
            atomicAdd(total + b, all);          // whole numbers: any order gives the same sums
            atomicAdd(before + b, early);
        } else {
            total[b] = all;
            before[b] = early;
        }
    }
    __syncthreads();
    // a thread takes up to two neighbouring bins
    const int q = bins <= kPlaceThreads ? 1 : 2, b0 = threadIdx.x * q;
    int t[2] = {}, sum = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i < q && b0 + i < bins)
            sum += t[i] = total[b0 + i];
    int run = thread_scan<kPlaceThreads>(sum, part);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i < q && b0 + i < bins) {
            if (blockIdx.x == 0 && is_offset(p.out, b0 + i))
                p.out.offsets[b0 + i] = run;
            before[b0 + i] += run;
            run += t[i];
        }
    __syncthreads();
    for (long long i = first; i < last; i += p.ctas * kPlaceThreads) {
        if (i > first && is_number(p.out, i, SITE_BOUNDS_A))
            id = p.ids[i], rank = p.out.rank[i];
        const int bin = static_cast<uint32_t>(id) < static_cast<uint32_t>(groups) ? id : groups;
        const int place = rank + before[bin];
        if (!is_number(p.out, i, SITE_BOUNDS_C) || !is_number(p.out, place, SITE_BOUNDS_C))
            continue;
        p.out.order[place] = static_cast<int>(i);
        if (p.out.rows)
            p.out.rows[i] = bin < groups ? place : -1;
    }
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

w8a8_status cuda_error(const char *what, cudaError_t e)
{
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return record_error(W8A8_ERR_CUDA, msg);
}

// How a sort is cut.  `units` of work (tokens, or 32 numbers) are dealt to CTAs, and to
// their warps, in equal runs: up to one cluster of sixteen CTAs while a warp's run is at
// most `deep` units (one launch; 512 tokens of 256 experts 12.0 us with sixteen, 16.6 with
// eight of twice the run; 768 in one launch of longer runs 14.6, in two 13.2), else to as many clusters as a GB300 holds at once (four of
// 8 CTAs, two to an SM, in each of eight parts; 38, which fill its 152 SMs in number, ran in
// two waves: 16384 tokens 56 us), or more where a CTA's run would not fit its shared memory.
struct Cut {
    int ctas;           // of the first launch
    int cluster;        // CTAs of a cluster
    int clusters;       // 1: one launch
    int most;           // units of a CTA at most
};
constexpr int kAtOnce = 32;
Cut cut(long long units, int deep, int per_warp)
{
    Cut c;
    if (units <= static_cast<long long>(kMaxCluster) * kWarps * deep) {
        c.cluster = 1;
        while (c.cluster < kMaxCluster && c.cluster * kWarps < units)
            c.cluster *= 2;
        c.ctas = c.cluster;
        c.clusters = 1;
    } else {
        const long long most = static_cast<long long>(kCluster) * kWarps * per_warp;
        c.cluster = kCluster;
        // (no warp without work: 1013 tokens by 8 clusters 13.7 us, by 32 15.9)
        const long long busy = (units + kCluster * kWarps - 1) / (kCluster * kWarps);
        c.clusters = static_cast<int>(std::max(std::min<long long>(kAtOnce, busy), (units + most - 1) / most));
        c.ctas = c.clusters * kCluster;
    }
    c.most = static_cast<int>((units + c.ctas - 1) / c.ctas);
    return c;
}
constexpr int kRouteDeep = 2, kGroupDeep = 8;
// (A CTA's numbers take at most 64 and 128 KB.)
Cut route_cut(long long T, int k) { return cut(T, kRouteDeep, 1024 / k); }
Cut group_cut(long long n) { return cut((n + 31) / 32, kGroupDeep, 64); }

size_t workspace_bytes(const Cut &c, long long n, int64_t groups, bool ranks)
{
    if (c.clusters == 1)
        return 0;
    return sizeof(int) * (static_cast<size_t>(c.clusters) * (groups + 1) + (ranks ? n : 0));
}

template <class Params>
cudaError_t launch(void (*kernel)(Params), const Params &p, int ctas, int cluster, int threads, size_t smem,
                   volatile int *smem_set, cudaStream_t stream)
{
    if (smem > 48 * 1024)
        if (const cudaError_t e = ensure_smem_limit(kernel, smem_set); e != cudaSuccess)
            return e;
    if (cluster > 8)                // more than every device has
        if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            e != cudaSuccess)
            return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(ctas, 1, 1);
    lc.blockDim = dim3(threads, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

cudaError_t launch_place(const GroupOut &out, const int *ids, const Cut &c, long long units, int per_unit,
                         cudaStream_t stream)
{
    PlaceParams p = {};
    p.ids = ids;
    p.clusters = c.clusters;
    p.units = units;
    p.per_unit = per_unit;
    p.first_ctas = c.ctas;
    const long long span = static_cast<long long>(c.most) * c.cluster * per_unit;
    p.ctas = static_cast<int>(std::max(1ll, std::min(8ll, (span + kPlaceThreads - 1) / kPlaceThreads)));
    p.out = out;
    static volatile int flags[kMaxDeviceFlags] = {};
    return launch(k_place, p, c.clusters * p.ctas, 1, kPlaceThreads, sizeof(int) * (2 * (out.groups + 1) + 32), flags,
                  stream);
}

template <int KIND, int PER>
cudaError_t launch_route(const RouteParams &p, const Cut &c, cudaStream_t stream)
{
    static volatile int flags[kMaxDeviceFlags] = {};
    const size_t smem = group_smem_bytes(p.E + 1, (p.most * p.k + 3) / 4 * 4) + RouteSmem::bytes(p);
    return launch(k_route<KIND, PER>, p, c.ctas, c.cluster, kThreads, smem, flags, stream);
}

template <int KIND> cudaError_t launch_route(const RouteParams &p, const Cut &c, cudaStream_t stream)
{
    if (p.per <= 1)
        return launch_route<KIND, 1>(p, c, stream);
    if (p.per <= 2)
        return launch_route<KIND, 2>(p, c, stream);
    if (p.per <= 4)
        return launch_route<KIND, 4>(p, c, stream);
    if (p.per <= 8)
        return launch_route<KIND, 8>(p, c, stream);
    if (p.per <= 16)
        return launch_route<KIND, 16>(p, c, stream);
    return launch_route<KIND, 32>(p, c, stream);
}

// The workspace's two parts.
w8a8_status take_workspace(GroupOut &out, const Cut &c, void *workspace, size_t bytes)
{
    out.hist = nullptr;
    out.rank = out.rows;
    const size_t need = workspace_bytes(c, out.n, out.groups, !out.rows);
    if (!need)
        return W8A8_OK;
    if (!workspace || bytes < need || !on(workspace, 4)) {
        char msg[160];
        snprintf(msg, sizeof(msg), "workspace of %zu bytes at %p: need %zu bytes, 4-byte aligned", bytes, workspace, need);
        return record_error(W8A8_ERR_WORKSPACE, msg);
    }
    out.hist = static_cast<int *>(workspace);
    out.hist_size = static_cast<long long>(c.clusters) * (out.groups + 1);
    if (!out.rank)
        out.rank = out.hist + out.hist_size;
    return W8A8_OK;
}

}  // namespace
}  // namespace w8a8

extern "C" size_t w8a8_route_workspace_size(int64_t T, int64_t E, int top_k)
{
    using namespace w8a8;
    if (T < 0 || E < 1 || E > W8A8_GROUPS_MAX || top_k < 1 || T > ((1ll << 31) - 1) / top_k)
        return 0;
    return workspace_bytes(route_cut(T, top_k), T * top_k, E, false);
}

extern "C" size_t w8a8_group_workspace_size(int64_t n, int64_t groups)
{
    using namespace w8a8;
    if (n < 0 || groups < 1 || groups > W8A8_GROUPS_MAX || n > (1ll << 31) - 1)
        return 0;
    return workspace_bytes(group_cut(n), n, groups, true);
}

extern "C" w8a8_status w8a8_route_experts(const void *logits_dev, w8a8_in_dtype dtype, int64_t ld,
                                          const float *bias_dev, const uint8_t *valid_dev, int64_t T, int64_t E,
                                          int top_k, w8a8_score scoring, int groups, int top_groups, int group_top,
                                          int renormalize, float scale, int32_t *ids_dev, float *weights_dev,
                                          int32_t *order_dev, int32_t *offsets_dev, int32_t *rows_dev,
                                          void *workspace_dev, size_t workspace_bytes, w8a8_stream_t stream)
{
    using namespace w8a8;
    if (T < 0 || E < 1 || top_k < 1)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size, or no expert to choose");
    if (dtype < W8A8_IN_BF16 || dtype > W8A8_IN_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown input dtype");
    if (scoring < W8A8_SCORE_SOFTMAX || scoring > W8A8_SCORE_SIGMOID)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown scoring");
    if (groups < 1 || E % groups || top_groups < 1 || top_groups > groups || group_top < 1 || group_top > 2 ||
        (groups > 1 && group_top > E / groups))
        return record_error(W8A8_ERR_INVALID_ARG, "groups must divide E, 1 <= top_groups <= groups, group_top be 1 or "
                                                  "2 and at most a group's experts");
    if (top_k > E / groups * top_groups)
        return record_error(W8A8_ERR_INVALID_ARG, "top_k above the experts of top_groups groups");
    ld = ld ? ld : E;
    if (ld < E)
        return record_error(W8A8_ERR_INVALID_ARG, "a row stride is shorter than its row");
    if (E > W8A8_GROUPS_MAX || top_k > W8A8_ROUTE_MAX_K || groups > W8A8_ROUTE_MAX_GROUPS ||
        T > ((1ll << 31) - 1) / top_k)
        return record_error(W8A8_ERR_UNSUPPORTED, "E above W8A8_GROUPS_MAX, top_k above W8A8_ROUTE_MAX_K, groups above "
                                                  "W8A8_ROUTE_MAX_GROUPS, or T * top_k of 2^31 or more");
    if (!offsets_dev || (T > 0 && (!logits_dev || !ids_dev || !weights_dev || !order_dev || !rows_dev)))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    const int bytes = dtype == W8A8_IN_FP32 ? 4 : 2;
    if (!on(logits_dev, bytes) || !on(bias_dev, 4) || !on(ids_dev, 4) || !on(weights_dev, 4) || !on(order_dev, 4) ||
        !on(offsets_dev, 4) || !on(rows_dev, 4))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    RouteParams p = {};
    p.logits = logits_dev;
    p.bias = bias_dev;
    p.valid = valid_dev;
    p.ids = ids_dev;
    p.weights = weights_dev;
    p.T = T;
    p.ld = ld;
    p.E = static_cast<int>(E);
    p.k = top_k;
    p.per = static_cast<int>((E + 31) / 32);
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_top = group_top;
    const int size = p.E / groups, lanes = size % p.per == 0 ? size / p.per : 0;
    p.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
    while (p.group_lanes >> p.group_shift > 1)
        ++p.group_shift;
    p.sigmoid = scoring == W8A8_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    const int each = 16 / bytes;
    p.vec = p.per % each == 0 && E % each == 0 && ld % each == 0 && on(logits_dev, 16);
    p.out.order = order_dev;
    p.out.offsets = offsets_dev;
    p.out.rows = rows_dev;
    p.out.groups = p.E;
    p.out.n = T * top_k;
    const Cut c = route_cut(T, top_k);
    p.most = c.most;
    if (const w8a8_status st = take_workspace(p.out, c, workspace_dev, workspace_bytes); st != W8A8_OK)
        return st;
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    p.out.status = dev.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == W8A8_IN_FP32   ? launch_route<W8A8_IN_FP32>(p, c, s)
                    : dtype == W8A8_IN_BF16 ? launch_route<W8A8_IN_BF16>(p, c, s)
                                            : launch_route<W8A8_IN_FP16>(p, c, s);
    if (e == cudaSuccess && p.out.hist)
        e = launch_place(p.out, ids_dev, c, T, top_k, s);
    return e == cudaSuccess ? W8A8_OK : cuda_error("kernel launch", e);
}

extern "C" w8a8_status w8a8_group_rows(const int32_t *ids_dev, int64_t n, int64_t groups, int32_t *order_dev,
                                       int32_t *offsets_dev, int32_t *rows_dev, void *workspace_dev,
                                       size_t workspace_bytes, w8a8_stream_t stream)
{
    using namespace w8a8;
    if (n < 0 || groups < 1)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size, or no group");
    if (groups > W8A8_GROUPS_MAX || n > (1ll << 31) - 1)
        return record_error(W8A8_ERR_UNSUPPORTED, "more than W8A8_GROUPS_MAX groups, or 2^31 ids or more");
    if (!offsets_dev || (n > 0 && (!ids_dev || !order_dev)))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (!on(ids_dev, 4) || !on(order_dev, 4) || !on(offsets_dev, 4) || !on(rows_dev, 4))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    GroupParams p = {};
    p.ids = ids_dev;
    p.out.order = order_dev;
    p.out.offsets = offsets_dev;
    p.out.rows = rows_dev;
    p.out.groups = static_cast<int>(groups);
    p.out.n = n;
    const Cut c = group_cut(n);
    if (const w8a8_status st = take_workspace(p.out, c, workspace_dev, workspace_bytes); st != W8A8_OK)
        return st;
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    p.out.status = dev.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    static volatile int flags[kMaxDeviceFlags] = {};
    cudaError_t e = launch(k_group, p, c.ctas, c.cluster, grp::kThreads,
                           group_smem_bytes(p.out.groups + 1, c.most * 32), flags, s);
    if (e == cudaSuccess && p.out.hist)
        e = launch_place(p.out, ids_dev, c, (n + 31) / 32, 32, s);
    return e == cudaSuccess ? W8A8_OK : cuda_error("kernel launch", e);
}
