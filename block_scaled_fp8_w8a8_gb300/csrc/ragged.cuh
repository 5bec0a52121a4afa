// What the ragged grouped kernels share: the list of row tiles that a CTA makes
// of the device's offsets, and the walk over its items.
#pragma once

#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {

// Exclusive prefix over the CTA's threads with Op, in thread order.
template <int THREADS, typename Op>
__device__ __forceinline__ int block_prefix(int v, int neutral, volatile int *warp_part, Op op)
{
    const int lane = static_cast<int>(lane_index()), w = static_cast<int>(warp_index());
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc = op(inc, u);
    }
    if (lane == 31)
        warp_part[w] = inc;
    __syncthreads();
    int base = neutral;
    for (int i = 0; i < w; ++i)
        base = op(base, warp_part[i]);
    const int up = __shfl_up_sync(0xffffffffu, inc, 1);
    __syncthreads();
    return lane > 0 ? op(base, up) : base;
}

// The tile list in shared memory: each expert's first row (row0) and first tile of
// ROWS rows (tile0), and one past the last of both.  Offsets that decrease or leave
// [0, M] are bent into a non-decreasing sequence in [0, M] (a running maximum), so
// that nothing after this leaves a buffer whatever they hold.
template <int THREADS, int ROWS>
__device__ __forceinline__ void make_tile_list(const RaggedParams &p, int *row0, int *tile0,
                                               volatile int *warp_part)
{
    constexpr int kPerThread = (kRaggedMaxExperts + 1 + THREADS - 1) / THREADS;
    const int first = static_cast<int>(threadIdx.x) * kPerThread;
    auto max_op = [](int a, int b) { return max(a, b); };
    auto add_op = [](int a, int b) { return a + b; };
    int o[kPerThread], top = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        o[i] = first + i <= p.experts ? min(max(__ldg(p.offsets + first + i), 0), p.M) : 0;
        top = max(top, o[i]);
    }
    int run = block_prefix<THREADS>(top, 0, warp_part, max_op);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        run = max(run, o[i]);
        if (first + i <= p.experts)
            row0[first + i] = run;
    }
    __syncthreads();
    int tiles[kPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int e = first + i;
        tiles[i] = e < p.experts ? (row0[e + 1] - row0[e] + ROWS - 1) / ROWS : 0;
        sum += tiles[i];
    }
    int at = block_prefix<THREADS>(sum, 0, warp_part, add_op);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (first + i <= p.experts)
            tile0[first + i] = at;
        at += tiles[i];
    }
    __syncthreads();
}

// The items of a CTA (or cluster): `first`, first + step, ... over (row tile,
// column tile), column tiles innermost, so that the CTAs running at one time share
// row tiles of A and an expert's weights in L2.
template <int ROWS> struct RaggedWalk {
    const int *row0, *tile0;      // [experts + 1] first row and first tile of each expert
    int item, items, num_n, experts;
    int e, m0, rows, nb;          // the current item: expert, first row, valid rows, column tile
    __device__ RaggedWalk(const RaggedParams &p, const int *r, const int *t, int first)
        : row0(r), tile0(t), item(first), items(t[p.experts] * p.num_n_tiles),
          num_n(p.num_n_tiles), experts(p.experts)
    {
    }
    __device__ bool next(int step)
    {
        if (item >= items)
            return false;
        const int mt = item / num_n;
        nb = item - mt * num_n;
        int lo = 0, hi = experts - 1;            // last expert whose first tile is <= mt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile0[mid] <= mt)
                lo = mid;
            else
                hi = mid - 1;
        }
        e = lo;
        m0 = row0[lo] + (mt - tile0[lo]) * ROWS;
        rows = min(ROWS, row0[lo + 1] - m0);
        item = item < items - step ? item + step : items;
        return true;
    }
};

}  // namespace w8a8
