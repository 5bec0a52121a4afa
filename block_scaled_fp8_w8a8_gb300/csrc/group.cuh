// Grouping of rows, shared by the router and by group_rows: a stable counting
// sort of n small whole numbers ("bins") over thread-block clusters.
//
// Every warp takes a contiguous run of the numbers and counts, in its own
// histogram in shared memory, how many of each bin came before each of them.
// Sums over the warps of a CTA, then (through distributed shared memory) over the
// CTAs of the cluster turn these ranks into places.  Where one cluster holds all
// numbers, that is the whole sort, in one launch; else each cluster's counts go to a
// workspace and a second launch adds what the earlier clusters hold.  No atomics but
// of whole numbers: the result is the same on every run.
#pragma once

#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {
namespace grp {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCluster = 8;             // CTAs of each cluster of many
constexpr int kMaxCluster = 16;         // and of one by itself at most
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
    long long hist_size;    // of hist, in counts
    unsigned *status;
};

// (debug-bounds build)
__device__ __forceinline__ bool is_number(const GroupOut &g, long long i, uint32_t site)
{
    return in_bounds(i >= 0 && i < g.n, g.status, site);
}
__device__ __forceinline__ bool is_count(const GroupOut &g, long long i)
{
    return in_bounds(i >= 0 && i < g.hist_size, g.status, SITE_BOUNDS_WORKSPACE);
}
__device__ __forceinline__ bool is_offset(const GroupOut &g, int b)
{
    return in_bounds(b >= 0 && b <= g.groups, g.status, SITE_BOUNDS_C);
}

// Exclusive scan over the block's threads of one number each; part holds one int per
// warp.  All threads call it, with a barrier between the writes and reads of part.
template <int THREADS> __device__ __forceinline__ int thread_scan(int sum, int *part)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 31)
        part[warp] = scan;
    __syncthreads();
    int before = lane < THREADS / 32 ? part[lane] : 0;
#pragma unroll
    for (int d = 1; d < THREADS / 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, d);
        before += lane >= d ? v : 0;
    }
    const int earlier = __shfl_sync(0xffffffffu, before, warp > 0 ? warp - 1 : 0);
    return scan - sum + (warp > 0 ? earlier : 0);
}

// Where unit `i` of n pieces of `units` begins.
__host__ __device__ __forceinline__ long long piece(long long units, int n, int i)
{
    return units * i / n;
}

// Shared memory of a sorting CTA.
struct GroupSmem {
    int *hist;              // [kWarps, bins]: counts, later each warp's first place
    int *tot;               // [bins] of this CTA, read by the cluster
    int *first;             // [bins] places before this CTA's
    int *part;              // [32]
    uint32_t *pairs;        // [numbers of the CTA]: bin << 16 | rank within the warp
};
__host__ __device__ constexpr size_t group_smem_bytes(int bins, int numbers)
{
    return sizeof(int) * ((static_cast<size_t>(kWarps + 2) * bins + 3) / 4 * 4 + 32 + numbers);
}
__device__ __forceinline__ GroupSmem carve(int *base, int bins)
{
    GroupSmem s;
    s.hist = base;
    s.tot = s.hist + kWarps * bins;
    s.first = s.tot + bins;
    s.part = base + ((kWarps + 2) * bins + 3) / 4 * 4;          // 16-byte boundary
    s.pairs = reinterpret_cast<uint32_t *>(s.part + 32);
    return s;
}

__device__ __forceinline__ void clear_hist(const GroupSmem &s, int bins)
{
    for (int i = threadIdx.x; i < kWarps * bins; i += kThreads)
        s.hist[i] = 0;
    __syncthreads();
}

// After every warp has counted its numbers, [lo, hi) of those that begin with
// first_number in the CTA: their places.  Called by all threads of all CTAs of the
// cluster.  A thread takes up to three neighbouring bins.
__device__ __forceinline__ void place_pairs(const GroupSmem &s, const GroupOut &g, long long first_number, int lo, int hi)
{
    constexpr int kMost = 3;
    const int bins = g.groups + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ctas, cluster;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
    const uint32_t me = cluster_ctarank();
    const int q = bins <= kThreads ? 1 : bins <= 2 * kThreads ? 2 : kMost, b0 = threadIdx.x * q;
    __syncthreads();
    int total[kMost], before[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        total[i] = before[i] = 0;
        const int b = b0 + i;
        if (i >= q || b >= bins)
            continue;
        int v[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v[w] = s.hist[w * bins + b];
        int run = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s.hist[w * bins + b] = run;
            run += v[w];
        }
        total[i] = run;
        s.tot[b] = run;
    }
    if (ctas > 1) {
        cluster_sync();
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int b = b0 + i;
            if (i >= q || b >= bins)
                continue;
            total[i] = 0;
            // (eight at a time: all sixteen at once 64 tokens 6.4 us, not 6.3, and 256 9.4, not 9.5)
#pragma unroll 1
            for (uint32_t r0 = 0; r0 < ctas; r0 += kCluster) {
                int v[kCluster];
#pragma unroll
                for (uint32_t r = 0; r < kCluster; ++r) {
                    v[r] = 0;
                    if (r0 + r < ctas)
                        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                                     : "=r"(v[r])
                                     : "r"(cluster_map(smem_addr(s.tot + b), r0 + r))
                                     : "memory");
                }
#pragma unroll
                for (uint32_t r = 0; r < kCluster; ++r) {
                    before[i] += r0 + r < me ? v[r] : 0;
                    total[i] += v[r];
                }
            }
        }
    }
    if (g.hist) {
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (i < q && b0 + i < bins) {
                if (me == 0 && is_count(g, static_cast<long long>(cluster) * bins + b0 + i))
                    g.hist[static_cast<long long>(cluster) * bins + b0 + i] = total[i];
                s.first[b0 + i] = before[i];
            }
    } else {
        int run = thread_scan<kThreads>(total[0] + total[1] + total[2], s.part);
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (i < q && b0 + i < bins) {
                if (me == 0 && is_offset(g, b0 + i))
                    g.offsets[b0 + i] = run;
                s.first[b0 + i] = run + before[i];
                run += total[i];
            }
    }
    __syncthreads();
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t v = s.pairs[i];
        const int b = v >> 16;
        const int place = s.first[b] + s.hist[warp * bins + b] + static_cast<int>(v & 0xffffu);
        const long long p = first_number + i;
        if (g.hist) {
            if (is_number(g, p, SITE_BOUNDS_WORKSPACE))
                g.rank[p] = place;
        } else if (is_number(g, p, SITE_BOUNDS_C) && is_number(g, place, SITE_BOUNDS_C)) {
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
