// Grouping of rows, shared by the router and by group_rows: a stable counting
// sort of n small whole numbers ("bins") over thread-block clusters.
//
// Every warp takes a contiguous run of the numbers and counts, in its own
// histogram in shared memory, how many of each bin came before each of them.
// Sums over the warps of a CTA, then (through distributed shared memory) over the
// CTAs of the cluster turn these ranks into places.  Where one cluster holds all
// numbers, that is the whole sort, in one launch; else each cluster's counts go to a
// workspace and a second launch adds what the earlier clusters hold.  No atomics:
// the result is the same on every run.
#pragma once

#include "ptx.cuh"

namespace w8a8 {
namespace grp {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kPlaceThreads = 1024;

// Where a sort's results go.  Bin `groups` holds what belongs to no group: it is
// sorted behind offsets[groups], with -1 for its rows.
struct GroupOut {
    int *order;             // [n] the number in each place
    int *offsets;           // [groups + 1]
    int *rows;              // [n] each number's place; null: not wanted
    int *rank;              // [n] places within a cluster, between the launches: rows or workspace
    int *hist;              // [clusters, groups + 1] counts; null: one cluster, one launch
    int groups;
    long long n;
};

// Exclusive sums of a[0 .. n-1] in shared memory by all threads of the block;
// returns the total.  `part` holds one int per warp.
__device__ __forceinline__ int block_scan(int *a, int n, int *part)
{
    const int threads = blockDim.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int q = (n + threads - 1) / threads, from = min(t * q, n), to = min(from + q, n);
    int sum = 0;
    for (int i = from; i < to; ++i)
        sum += a[i];
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 31)
        part[warp] = scan;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < threads / 32; ++w) {
        const int v = part[w];
        before += w < warp ? v : 0;
        total += v;
    }
    int run = before + scan - sum;
    for (int i = from; i < to; ++i) {
        const int v = a[i];
        a[i] = run;
        run += v;
    }
    __syncthreads();
    return total;
}

// Shared memory of a sorting CTA.
struct GroupSmem {
    int *hist;              // [kWarps, bins]: counts, later each warp's first place
    int *tot;               // [bins] of this CTA, read by the cluster
    int *first;             // [bins] places before this CTA's
    int *part;              // [32]
    uint32_t *pairs;        // [kWarps, per_warp]: bin << 16 | rank within the warp
};
__host__ __device__ constexpr size_t group_smem_bytes(int bins, int per_warp)
{
    return sizeof(int) * (static_cast<size_t>(kWarps + 2) * bins + 32 + static_cast<size_t>(kWarps) * per_warp);
}
__device__ __forceinline__ GroupSmem carve(int *base, int bins)
{
    GroupSmem s;
    s.hist = base;
    s.tot = s.hist + kWarps * bins;
    s.first = s.tot + bins;
    s.part = s.first + bins;
    s.pairs = reinterpret_cast<uint32_t *>(s.part + 32);
    return s;
}

__device__ __forceinline__ void clear_hist(const GroupSmem &s, int bins)
{
    for (int i = threadIdx.x; i < kWarps * bins; i += kThreads)
        s.hist[i] = 0;
    __syncthreads();
}

// After every warp has counted its numbers [first_number, first_number + count):
// places of the CTA's numbers.  Called by all threads of all CTAs of the cluster.
__device__ __forceinline__ void place_pairs(const GroupSmem &s, const GroupOut &g, long long first_number,
                                            int count, int per_warp)
{
    const int bins = g.groups + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ctas, cluster;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
    const uint32_t me = cluster_ctarank();
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int v = s.hist[w * bins + b];
            s.hist[w * bins + b] = run;
            run += v;
        }
        s.tot[b] = run;
    }
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    // first[b]: what the cluster's earlier CTAs hold; and the cluster's total
    const int per_thread = (bins + kThreads - 1) / kThreads;       // at most 3
    int before[3], total[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int b = threadIdx.x + i * kThreads;
        before[i] = total[i] = 0;
        if (i < per_thread && b < bins) {
            int v[kMaxCluster];
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r) {
                v[r] = 0;
                if (r < ctas)
                    asm volatile("ld.shared::cluster.s32 %0, [%1];"
                                 : "=r"(v[r])
                                 : "r"(cluster_map(smem_addr(s.tot + b), r))
                                 : "memory");
            }
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r) {
                before[i] += r < me ? v[r] : 0;
                total[i] += v[r];
            }
            if (g.hist) {
                if (me == 0)
                    g.hist[static_cast<long long>(cluster) * bins + b] = total[i];
                s.first[b] = before[i];
            } else {
                s.first[b] = total[i];
            }
        }
    }
    __syncthreads();
    if (!g.hist) {
        block_scan(s.first, bins, s.part);
        if (me == 0)
            for (int b = threadIdx.x; b < bins; b += kThreads)
                g.offsets[b] = s.first[b];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int b = threadIdx.x + i * kThreads;
            if (i < per_thread && b < bins)
                s.first[b] += before[i];
        }
        __syncthreads();
    }
    const int lo = warp * per_warp, hi = min(lo + per_warp, count);
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t v = s.pairs[i];
        const int b = v >> 16;
        const int place = s.first[b] + s.hist[warp * bins + b] + static_cast<int>(v & 0xffffu);
        const long long p = first_number + i;
        if (g.hist) {
            g.rank[p] = place;
        } else {
            g.order[place] = static_cast<int>(p);
            if (g.rows)
                g.rows[p] = b < g.groups ? place : -1;
        }
    }
    if (ctas > 1)
        cluster_sync();         // tot is read until here
}

}  // namespace grp
}  // namespace w8a8
