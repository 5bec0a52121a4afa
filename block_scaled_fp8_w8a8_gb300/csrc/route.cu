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
// that, those that are too near are scored and ranked again in fp64 (refine); where the
// worst kept and the best dropped run are, the whole token is (choose_exact).
#include <algorithm>
#include <cstdio>

#include "../../include/w8a8_block_fp8.h"
#include "group.cuh"
#include "kernels.cuh"
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
    int sigmoid, renormalize;
    int vec;                    // a lane's logits can be loaded by 16 bytes
    float scale;
    int per_warp;               // tokens of a warp
    GroupOut out;
};

constexpr uint32_t kAll = 0xffffffffu;

// Order-preserving maps; key 0 belongs to no number.
__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __float_as_uint(f + 0.f);        // -0 -> +0
    return f != f ? 0xffffffffu : u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
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

template <int KIND> __device__ __forceinline__ float load_logit(const void *row, int e)
{
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
                if (in)
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
        l[i] = i < p.per && e0 + i < p.E ? load_logit<KIND>(row, e0 + i) : -INFINITY;
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

// Whether this lane's run is kept, from its value (the same in all of its lanes), and
// the values at the border.
template <class K>
__device__ __forceinline__ bool rank_groups(int groups, int group_lanes, int top, int g, K value, K *kept, K *dropped)
{
    int above = 0;
    for (int j = 0; j < groups; ++j) {
        const K v = __shfl_sync(kAll, value, j * group_lanes);
        above += v > value || (v == value && j < g);
    }
    const bool keep = g < groups && above < top;
    *kept = ~warp_max(keep ? ~value : K(0));
    *dropped = warp_max(keep || g >= groups ? K(0) : value);
    return keep;
}

template <class K> __device__ __forceinline__ K group_value(int group_top, K a, K b)
{
    return group_top == 2 ? key_of(value_of(a) + value_of(b)) : a;
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
        m = fmaxf(m, load_logit<KIND>(row, e0 + i));
    m = value_of(warp_max(key_of(m)));
    m = m == -INFINITY ? 0.f : m;
    double z = 0;
    if (!p.sigmoid) {
        for (int i = 0; i < n; ++i)
            z += exp(static_cast<double>(load_logit<KIND>(row, e0 + i)) - m);
        z = warp_sum(z);
    }
    for (int i = 0; i < n; ++i) {
        const float l = load_logit<KIND>(row, e0 + i);
        double s;
        if (p.sigmoid)
            s = 1 / (1 + exp(-static_cast<double>(l)));
        else
            s = z == 0 ? 0. : exp(static_cast<double>(l) - m) / z;
        ck[i] = key_of(p.bias ? s + p.bias[e0 + i] : s);
        key[i] = p.bias ? ck[i] : key_of(static_cast<double>(l));
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

// Ranks `count` (at most 32) experts, lane j's being id, by their scores in fp64: returns
// the expert of rank `lane`.
template <int KIND> __device__ __noinline__ int refine(const RouteParams &p, const void *row, int id, int count, float m)
{
    const int lane = threadIdx.x & 31;
    const bool in = lane < count;
    double s = 0;
    const double l = in ? static_cast<double>(load_logit<KIND>(row, id)) : 0.;
    if (p.sigmoid) {
        s = 1 / (1 + exp(-l));
    } else {
        double z = 0;
#pragma unroll 4
        for (int e = lane; e < p.E; e += 32)
            z += exp(static_cast<double>(load_logit<KIND>(row, e)) - m);
        z = warp_sum(z);
        s = z == 0 ? 0. : exp(l - m) / z;
    }
    // without a bias the logits rank
    const unsigned long long key = in ? key_of(p.bias ? s + p.bias[id] : l) : 0ull;
    int above = 0;
    for (int j = 0; j < count; ++j) {
        const unsigned long long other = __shfl_sync(kAll, key, j);
        const int other_id = __shfl_sync(kAll, id, j);
        above += other > key || (other == key && other_id < id);
    }
    int mine = id;
    for (int j = 0; j < count; ++j) {
        const int rank = __shfl_sync(kAll, above, j), e = __shfl_sync(kAll, id, j);
        mine = rank == lane ? e : mine;
    }
    return mine;
}

// One token: lane j < k gets the j-th expert and its weight.
template <int KIND, int PER>
__device__ __forceinline__ void route_token(const RouteParams &p, const void *row, const float (&l)[PER],
                                            const float *bias, int *run_keys, int &id, float &weight)
{
    const int lane = threadIdx.x & 31, e0 = lane * p.per;
    const bool biased = p.bias != nullptr;
    const bool scored = biased || (p.groups > 1 && p.group_top == 2) || (!p.sigmoid && !p.renormalize);
    float c[PER];
    float m = 0.f, z = 1.f;
    // An upper bound of the error of an fp32 score, in units of 2^-23.  An exponential of x
    // is off by 2 units and by its argument's rounding, 0.75 |x|, relatively.
    //   sigmoid: s (1 - s) (2 + 0.75 |l|) <= 0.6 units, then one rounded sum and the
    //     quotient: 2.1 units, below 2^-21.
    //   softmax: with u = -x the terms' errors are at most 2 units of the largest term and,
    //     in the sum z, 2 + 0.75 u averaged with the terms as weights, where u averages at
    //     most ln E + 1 < 8; the sum's roundings (PER + 5) / 2 <= 18.5, the quotient 1.5: with
    //     s <= 1 / z at most 30 units of 1 / z, below 2^-18 / z.
    float bound = 0x1p-21f;
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
    if (biased) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            c[i] += PER <= 8 ? bias[i] : i < p.per && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
    }
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = i < p.per && e0 + i < p.E ? key_of(biased ? c[i] : l[i]) : 0u;
    bool exact = false;             // decide the whole token again in fp64
    if (p.groups > 1) {
        const int size = p.E / p.groups;
        uint32_t a = 0, b = 0;
        uint32_t kept, dropped;
        const bool sums = p.group_top == 2;
        if (p.group_lanes) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                two_best(a, b, sums && !biased ? (key[i] ? key_of(c[i]) : 0u) : key[i]);
            for (int d = 1; d < p.group_lanes; d *= 2) {
                const uint32_t oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
                two_best(a, b, oa);
                b = ob > b ? ob : b;
            }
            const bool keep = rank_groups<uint32_t>(p.groups, p.group_lanes, p.top_groups, lane / p.group_lanes,
                                                    group_value(p.group_top, a, b), &kept, &dropped);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = keep ? key[i] : 0u;
        } else {
            // runs that do not begin with a lane: through shared memory, lane g takes run g
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i])
                    run_keys[e0 + i] = static_cast<int>(sums && !biased ? key_of(c[i]) : key[i]);
            __syncwarp();
            if (lane < p.groups)
                for (int i = 0; i < size; ++i)
                    two_best(a, b, static_cast<uint32_t>(run_keys[lane * size + i]));
            __syncwarp();
            const uint32_t keep = __ballot_sync(kAll, rank_groups<uint32_t>(p.groups, 1, p.top_groups, lane,
                                                                           group_value(p.group_top, a, b), &kept, &dropped));
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = keep >> ((e0 + i) / size & 31) & 1 ? key[i] : 0u;
        }
        if ((biased || sums) && p.top_groups < p.groups) {
            const float hi = value_of(kept), lo = value_of(dropped);
            exact = !(hi - lo > 4.f * bound + 0x1p-21f * (fabsf(hi) + fabsf(lo)));
        }
    }
    // The slot takes the place of the key's lowest bits; 16-bit logits have zeros there.
    constexpr uint32_t kSlots = PER - 1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = key[i] ? (key[i] & ~kSlots) | (kSlots - i) : 0u;
    sort_keys(key);
    const bool whole = !biased && KIND != W8A8_IN_FP32;
    const float near_by = biased ? 2.f * bound : 0.f, near_at = biased ? 0x1p-22f + PER * 0x1p-23f : 0.f;
    uint32_t mine = 0, last = 0;        // lane j: the j-th key
    id = 0;
    auto round = [&](int j) {
        // (the lane before the slot: the lower index first)
        const uint32_t kept_bits = key[0] & ~kSlots;
        const uint32_t top = warp_max(kept_bits);
        const int src = __ffs(__ballot_sync(kAll, kept_bits == top)) - 1;
        const uint32_t slot = kSlots - (__shfl_sync(kAll, key[0], src) & kSlots);
        if (lane == src) {
#pragma unroll
            for (int i = 0; i + 1 < PER; ++i)
                key[i] = key[i + 1];
            key[PER - 1] = 0;
        }
        if (lane == j)
            mine = top, id = src * p.per + static_cast<int>(slot);
        last = top;
    };
    for (int j = 0; j < p.k; ++j)
        round(j);
    if (!whole && !exact) {
        // Whether key `a` is surely above key `b`, the next.  (Without a bias that is so where
        // the kept bits differ.)
        auto near = [&](uint32_t a, uint32_t b) {
            const float hi = value_of(a), lo = value_of(b & ~kSlots);
            return b > kSlots && !(hi - lo > near_by + near_at * (fabsf(hi) + fabsf(lo)));
        };
        const uint32_t behind = warp_max(key[0]);
        const uint32_t below = __shfl_down_sync(kAll, mine, 1);         // (by every lane)
        const uint32_t next = lane == p.k - 1 ? behind : below;
        bool unsure = lane < p.k && near(mine, next);
        if (__any_sync(kAll, unsure)) {
            // Take on what is too near the last, as many as lanes hold.
            int count = p.k;
            while (count < 32 && near(last, warp_max(key[0])))
                round(count++);
            const int next_id = __shfl_down_sync(kAll, id, 1);
            const float own_l = lane < count ? load_logit<KIND>(row, id) : 0.f;
            const float own_b = biased && lane < count ? p.bias[id] : 0.f;
            const float next_l = __shfl_down_sync(kAll, own_l, 1), next_b = __shfl_down_sync(kAll, own_b, 1);
            // equal logits under equal biases are equal scores, in order of their index
            const uint32_t after = __shfl_down_sync(kAll, mine, 1);
            unsure = lane + 1 < count && near(mine, after) && !(own_l == next_l && own_b == next_b && id < next_id);
            if (near(last, warp_max(key[0])))
                exact = true;               // more than 32
            else if (__any_sync(kAll, unsure))
                id = refine<KIND>(p, row, id, count, m);
        }
    }
    if (exact)
        id = choose_exact<KIND>(p, row);
    // The weights from the chosen logits, in full fp32.
    const bool chosen = lane < p.k;
    const float x = chosen ? load_logit<KIND>(row, id) : -INFINITY;
    float s;
    if (p.renormalize) {
        // relative to the largest of them, so that small scores keep their ratios
        float r = value_of(warp_max(key_of(x != x ? -INFINITY : x)));
        if (p.sigmoid) {
            r = fminf(r, 0.f);
            s = x > 0.f ? 1.f / (1.f + expf(-x)) : expf(x - r) / (1.f + expf(x));
        } else {
            s = expf(x - r);
        }
        if (r == -INFINITY && x == -INFINITY)
            s = 0.f;            // (-infinity) - (-infinity)
        s = chosen ? s : 0.f;
        const float sum = warp_sum(s);
        s = sum == 0.f ? 0.f : s / sum;
        if (!p.sigmoid && z != z)
            s = z;              // a NaN or an infinity in the row that was not chosen
    } else {
        s = p.sigmoid ? 1.f / (1.f + expf(-x)) : z == 0.f ? 0.f : expf(x - m) / z;
    }
    weight = s * p.scale;
}

template <int KIND, int PER> __global__ void __launch_bounds__(kThreads, PER <= 8 ? 2 : 1) k_route(const RouteParams p)
{
    extern __shared__ int smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = p.E + 1, e0 = lane * p.per;
    const GroupSmem s = carve(smem, bins);
    const int pairs = p.per_warp * p.k;
    int *const run_keys = reinterpret_cast<int *>(s.pairs + kWarps * pairs) + warp * p.E;
    clear_hist(s, bins);
    grid_dependency_wait();
    grid_launch_dependents();
    float bias[PER <= 8 ? PER : 1];
    if constexpr (PER <= 8) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            bias[i] = p.bias && i < p.per && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
    }
    const long long cta_first = static_cast<long long>(blockIdx.x) * kWarps * p.per_warp;
    const long long first = cta_first + static_cast<long long>(warp) * p.per_warp;
    const int tokens = static_cast<int>(max(0ll, min(static_cast<long long>(p.per_warp), p.T - first)));
    constexpr int kBytes = KIND == W8A8_IN_FP32 ? 4 : 2;
    for (int i = 0; i < tokens; ++i) {
        const long long t = first + i;
        const void *row = static_cast<const char *>(p.logits) + t * p.ld * kBytes;
        int id = p.E, rank;
        float weight = 0.f;
        const bool valid = !p.valid || p.valid[t] != 0;
        if (valid) {
            float l[PER];
            load_lane<KIND, PER>(p, row, e0, l);
            route_token<KIND, PER>(p, row, l, bias, run_keys, id, weight);
        }
        int *const h = s.hist + warp * bins;
        if (lane < p.k) {
            p.ids[t * p.k + lane] = valid ? id : -1;
            p.weights[t * p.k + lane] = weight;
            rank = h[id] + (valid ? 0 : lane);          // a token's experts differ
            s.pairs[warp * pairs + i * p.k + lane] = static_cast<uint32_t>(id) << 16 | rank;
        }
        __syncwarp();
        if (valid ? lane < p.k : lane == 0)
            h[id] += valid ? 1 : p.k;
        __syncwarp();
    }
    const long long left = max(0ll, p.T - cta_first);
    place_pairs(s, p.out, cta_first * p.k,
                static_cast<int>(min(left, static_cast<long long>(kWarps) * p.per_warp)) * p.k, pairs);
}

struct GroupParams {
    const int *ids;             // [n]
    int per_warp;               // numbers of a warp, a multiple of 32
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
    const long long cta_first = static_cast<long long>(blockIdx.x) * kWarps * p.per_warp;
    const long long first = cta_first + static_cast<long long>(warp) * p.per_warp;
    const int count = static_cast<int>(max(0ll, min(static_cast<long long>(p.per_warp), p.out.n - first)));
    int *const h = s.hist + warp * bins;
    for (int i = 0; i < count; i += 32) {
        const bool in = i + lane < count;
        const int id = in ? p.ids[first + i + lane] : 0;
        const int bin = !in ? bins : static_cast<uint32_t>(id) < static_cast<uint32_t>(groups) ? id : groups;
        const uint32_t same = __match_any_sync(kAll, bin);
        const uint32_t before = same & ((1u << lane) - 1u);
        if (in)
            s.pairs[warp * p.per_warp + i + lane] = static_cast<uint32_t>(bin) << 16 | (h[bin] + __popc(before));
        __syncwarp();
        if (in && !before)
            h[bin] += __popc(same);
        __syncwarp();
    }
    const long long left = max(0ll, p.out.n - cta_first);
    place_pairs(s, p.out, cta_first, static_cast<int>(min(left, static_cast<long long>(kWarps) * p.per_warp)),
                p.per_warp);
}

// The second launch of a sort over several clusters: places within a cluster, plus
// what earlier clusters hold.  `span` numbers belong to a cluster, gridDim.x / clusters
// CTAs to each.
struct PlaceParams {
    const int *ids;
    int clusters, ctas;             // CTAs of a cluster's span
    long long span;
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
    // Bins side by side in a warp, the clusters dealt to slices of the block.
    const int width = (bins + 31) / 32 * 32, slices = max(1, kPlaceThreads / width);
    const int mine = threadIdx.x / width;
    for (int b = threadIdx.x % width; b < bins && mine < slices; b += slices > 1 ? bins : kPlaceThreads) {
        int all = 0, early = 0;
#pragma unroll 8
        for (int c = mine; c < p.clusters; c += slices) {
            const int v = p.out.hist[static_cast<long long>(c) * bins + b];
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
    block_scan(total, bins, part);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < bins; b += kPlaceThreads)
            p.out.offsets[b] = total[b];
    for (int b = threadIdx.x; b < bins; b += kPlaceThreads)
        before[b] += total[b];
    __syncthreads();
    const long long first = cluster * p.span, last = min(p.out.n, first + p.span);
    for (long long i = first + slice * kPlaceThreads + threadIdx.x; i < last; i += p.ctas * kPlaceThreads) {
        const int id = p.ids[i];
        const int bin = static_cast<uint32_t>(id) < static_cast<uint32_t>(groups) ? id : groups;
        const int place = p.out.rank[i] + before[bin];
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

// How a sort is cut.  `units` of work (tokens, or 32 numbers) go to warps in runs of
// per_warp: up to one cluster of eight CTAs while a warp's run is at most `deep` units
// (one launch), else runs that give two CTAs to every SM.
struct Cut {
    int per_warp;
    int ctas;           // of the first launch
    int cluster;        // CTAs of a cluster
    int clusters;       // 1: one launch
};
constexpr int kMaxPerWarp = 64;
Cut cut(long long units, int deep, int sm_count)
{
    Cut c;
    const long long warps = kMaxCluster * kWarps;
    if (units <= warps * deep) {
        c.per_warp = static_cast<int>(std::max(1ll, (units + warps - 1) / warps));
        c.ctas = static_cast<int>(std::max(1ll, (units + kWarps * c.per_warp - 1) / (kWarps * c.per_warp)));
        c.cluster = 1;
        while (c.cluster < c.ctas)
            c.cluster *= 2;
        c.ctas = c.cluster;
        c.clusters = 1;
        return c;
    }
    const long long want = 2ll * sm_count * kWarps;
    c.per_warp = static_cast<int>(std::min<long long>(kMaxPerWarp, (units + want - 1) / want));
    const long long span = static_cast<long long>(kMaxCluster) * kWarps * c.per_warp;
    c.cluster = kMaxCluster;
    c.clusters = static_cast<int>((units + span - 1) / span);
    c.ctas = c.clusters * kMaxCluster;
    return c;
}
constexpr int kRouteDeep = 4, kGroupDeep = 16;
Cut route_cut(long long T, int sm_count) { return cut(T, kRouteDeep, sm_count); }
Cut group_cut(long long n, int sm_count) { return cut((n + 31) / 32, kGroupDeep, sm_count); }

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

cudaError_t launch_place(const GroupOut &out, const int *ids, const Cut &c, long long span, cudaStream_t stream)
{
    PlaceParams p = {};
    p.ids = ids;
    p.clusters = c.clusters;
    p.span = span;
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
    size_t smem = group_smem_bytes(p.E + 1, p.per_warp * p.k);
    if (p.groups > 1 && !p.group_lanes)
        smem += sizeof(int) * kWarps * p.E;
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
    if (!out.rank)
        out.rank = out.hist + static_cast<size_t>(c.clusters) * (out.groups + 1);
    return W8A8_OK;
}

// The SMs that cuts go by: a GB300's, so that a workspace's size asks no device.
constexpr int kCutSms = 152;

}  // namespace
}  // namespace w8a8

extern "C" size_t w8a8_route_workspace_size(int64_t T, int64_t E, int top_k)
{
    using namespace w8a8;
    if (T < 0 || E < 1 || E > W8A8_GROUPS_MAX || top_k < 1 || T > ((1ll << 31) - 1) / top_k)
        return 0;
    return workspace_bytes(route_cut(T, kCutSms), T * top_k, E, false);
}

extern "C" size_t w8a8_group_workspace_size(int64_t n, int64_t groups)
{
    using namespace w8a8;
    if (n < 0 || groups < 1 || groups > W8A8_GROUPS_MAX || n > (1ll << 31) - 1)
        return 0;
    return workspace_bytes(group_cut(n, kCutSms), n, groups, true);
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
    const Cut c = route_cut(T, kCutSms);
    p.per_warp = c.per_warp;
    if (const w8a8_status st = take_workspace(p.out, c, workspace_dev, workspace_bytes); st != W8A8_OK)
        return st;
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == W8A8_IN_FP32   ? launch_route<W8A8_IN_FP32>(p, c, s)
                    : dtype == W8A8_IN_BF16 ? launch_route<W8A8_IN_BF16>(p, c, s)
                                            : launch_route<W8A8_IN_FP16>(p, c, s);
    if (e == cudaSuccess && p.out.hist)
        e = launch_place(p.out, ids_dev, c, static_cast<long long>(c.cluster) * grp::kWarps * c.per_warp * top_k, s);
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
    const Cut c = group_cut(n, kCutSms);
    p.per_warp = c.per_warp * 32;
    if (const w8a8_status st = take_workspace(p.out, c, workspace_dev, workspace_bytes); st != W8A8_OK)
        return st;
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    static volatile int flags[kMaxDeviceFlags] = {};
    cudaError_t e = launch(k_group, p, c.ctas, c.cluster, grp::kThreads,
                           group_smem_bytes(p.out.groups + 1, p.per_warp), flags, s);
    if (e == cudaSuccess && p.out.hist)
        e = launch_place(p.out, ids_dev, c, static_cast<long long>(c.cluster) * grp::kWarps * p.per_warp, s);
    return e == cudaSuccess ? W8A8_OK : cuda_error("kernel launch", e);
}
