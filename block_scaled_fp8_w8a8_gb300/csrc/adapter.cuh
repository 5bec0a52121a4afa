// What the two forms of the adapter product share: the call's parameters, the search for
// a CTA's rows, the parts of an fp32 number.
#pragma once

#include <algorithm>

#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {
namespace lora {

struct AdapterParams {
    const uint16_t *x;          // [T, ld_x]
    const uint16_t *A;          // [L, r, K]
    const uint16_t *B;          // [L, N, r]
    const int *order;           // [T]
    const int *offsets;         // [L + 1]
    const float *scales;        // [L] or null
    const void *base;           // [T, ld_base]
    void *out;                  // [T, ld_out]; may be base
    long long ld_x, ld_base, ld_out;
    int T, L, r, K, N;
    int r_pad;                  // r up to whole 16
    int vec_k, vec_r;           // 16-byte pieces of x and A, of B
    unsigned *status;
    unsigned long long wait_limit;
    int vec_n;                  // eight columns of base and out at a time, by 16 bytes
};

// (debug-bounds build: whether an access lies in its buffer)
struct Buffer {
    const void *base;
    size_t size;
    unsigned *status;
    uint32_t site;
    __device__ __forceinline__ bool holds(const void *at, size_t bytes) const
    {
        return in_bounds(inside(at, bytes, base, size), status, site);
    }
};
__device__ __forceinline__ Buffer x_of(const AdapterParams &p)
{
    return {p.x, span(p.T, p.ld_x, p.K, 2), p.status, SITE_BOUNDS_A};
}
__device__ __forceinline__ Buffer a_of(const AdapterParams &p)
{
    return {p.A, span(static_cast<long long>(p.L) * p.r, p.K, p.K, 2), p.status, SITE_BOUNDS_B};
}
__device__ __forceinline__ Buffer b_of(const AdapterParams &p)
{
    return {p.B, span(static_cast<long long>(p.L) * p.N, p.r, p.r, 2), p.status, SITE_BOUNDS_B};
}
__device__ __forceinline__ Buffer base_of(const AdapterParams &p, int element)
{
    return {p.base, span(p.T, p.ld_base, p.N, element), p.status, SITE_BOUNDS_C};
}
__device__ __forceinline__ Buffer out_of(const AdapterParams &p, int element)
{
    return {p.out, span(p.T, p.ld_out, p.N, element), p.status, SITE_BOUNDS_C};
}
// The row in a place of the sort, -1 for one that is none.
__device__ __forceinline__ int row_in_place(const AdapterParams &p, int place)
{
    const int row = in_bounds(place >= 0 && place < p.T, p.status, SITE_BOUNDS_A) ? p.order[place] : -1;
    return static_cast<unsigned>(row) < static_cast<unsigned>(p.T) ? row : -1;
}
__device__ __forceinline__ float scale_of(const AdapterParams &p, int adapter)
{
    return p.scales && in_bounds(adapter >= 0 && adapter < p.L, p.status, SITE_BOUNDS_SCALES) ? p.scales[adapter] : 1.f;
}

// The power of two that brings a row of h, whose largest size is top, near 2^14: the
// factor that does, and the one that its sums are multiplied by afterwards.
__device__ __forceinline__ void power_of(float top, float *shrink, float *factor)
{
    // top in [2^e, 2^(e+1)); the power stays within the normal numbers
    const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int power = top == 0.f || e == 128 ? 0 : min(max(e - 14, -126), 126);
    *shrink = __uint_as_float(static_cast<uint32_t>(127 - power) << 23);
    *factor = __uint_as_float(static_cast<uint32_t>(127 + power) << 23);
}

// The item (adapter, first place, rows) of a cluster among tiles of `tile` rows:
// adapter L is the rows without one.  Every thread of the CTA calls it.
struct Item {
    int adapter, first, rows;       // rows 0: none
};
template <int THREADS>
__device__ __forceinline__ Item find_item(const AdapterParams &p, int index, int tile, int groups, int *scratch)
{
    // scratch: [12] sums of warps, then the item
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int q = (groups + THREADS - 1) / THREADS, from = min(t * q, groups), to = min(from + q, groups);
    auto offset = [&](int g) {
        return g > p.L || !in_bounds(g >= 0, p.status, SITE_BOUNDS_B) ? p.T : min(max(p.offsets[g], 0), p.T);
    };
    int sum = 0;
    for (int g = from; g < to; ++g)
        sum += (max(offset(g + 1) - offset(g), 0) + tile - 1) / tile;
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 31)
        scratch[warp] = scan;
    if (t == 0)
        scratch[14] = 0;
    __syncthreads();
    int run = scan - sum;
    for (int w = 0; w < warp; ++w)
        run += scratch[w];
    if (index >= run && index < run + sum) {
        for (int g = from; g < to; ++g) {
            const int first = offset(g), rows = max(offset(g + 1) - first, 0), tiles = (rows + tile - 1) / tile;
            if (index >= run && index < run + tiles) {
                const int skip = (index - run) * tile;
                scratch[12] = g;
                scratch[13] = first + skip;
                scratch[14] = min(tile, rows - skip);
            }
            run += tiles;
        }
    }
    __syncthreads();
    return Item{scratch[12], scratch[13], scratch[14]};
}

// v's leading 16-bit part, removed from v.  An infinity leaves nothing.
template <bool BF16> __device__ __forceinline__ uint32_t take_part(float &v)
{
    float part;
    uint32_t bits;
    if constexpr (BF16) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        part = __bfloat162float(h);
        bits = __bfloat16_as_ushort(h);
    } else {
        const __half h = __float2half_rn(v);
        part = __half2float(h);
        bits = __half_as_ushort(h);
    }
    v = fabsf(part) == INFINITY ? 0.f : v - part;
    return bits;
}

// Copies columns [from, to) of rows[0 .. count-1] (-1: none) of base to out, by all threads
// of the CTA; WORD is the piece that is copied at once.  Eight pieces of a thread are in
// flight: with one, 128 rows of 8 KB took a CTA 100 us.
template <typename WORD, int THREADS>
__device__ __forceinline__ void copy_rows(const AdapterParams &p, const int *rows, int count, int from, int to, int element)
{
    constexpr int kFlight = 8;
    const int each = static_cast<int>(sizeof(WORD)) / element, pieces = (to - from) / each;
    const long long all = static_cast<long long>(pieces) * count;
    for (long long i0 = threadIdx.x; i0 < all; i0 += THREADS * kFlight) {
        WORD v[kFlight];
        long long at[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const long long i = i0 + j * THREADS;
            at[j] = -1;
            if (i < all) {
                const int r = static_cast<int>(i / pieces), n = from + static_cast<int>(i - static_cast<long long>(r) * pieces) * each;
                if (const int row = rows[r]; row >= 0) {
                    const char *const from_at = static_cast<const char *>(p.base) + (row * p.ld_base + n) * element;
                    if (!base_of(p, element).holds(from_at, sizeof(WORD)))
                        continue;
                    at[j] = (row * p.ld_out + n) * element;
                    v[j] = *reinterpret_cast<const WORD *>(from_at);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (at[j] >= 0 && out_of(p, element).holds(static_cast<char *>(p.out) + at[j], sizeof(WORD)))
                *reinterpret_cast<WORD *>(static_cast<char *>(p.out) + at[j]) = v[j];
    }
}

// Up to `bytes` of dynamic shared memory for a kernel, and clusters of up to 16 CTAs,
// set once per device by its own flags.  (The device's most would leave nothing for the kernel's static arrays.)
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, size_t bytes, volatile int *set, bool large_clusters = false)
{
    int id = 0;
    cudaError_t e = cudaGetDevice(&id);
    if (e == cudaSuccess && (id < 0 || id >= kMaxDeviceFlags))
        e = cudaErrorInvalidDevice;
    if (e == cudaSuccess && !set[id]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e == cudaSuccess && large_clusters)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        set[id] = e == cudaSuccess;
    }
    return e;
}

// Tiles that T rows of `groups` adapters make at most: one unfilled each.
inline long long most_items(long long T, long long groups, int tile)
{
    const long long g = std::min(T, groups);
    return (T + g * (tile - 1)) / tile;
}

// Many rows: the two launches of adapter_tile.cu.
struct TileParams {
    AdapterParams a;
    float *h;                   // [splits, T, r_pad]: scales[l] x A^T of K's parts, by place
    int splits;
    int chunks;                 // CTAs that share a tile's columns
};
// Whether they take a problem (16-byte pieces everywhere, r in bounds), and by how
// many parts of K.
bool tile_takes(const AdapterParams &p);
int tile_splits(const AdapterParams &p);
cudaError_t launch_tile(const AdapterParams &p, int x_kind, int out_kind, float *h, const DeviceView &dev,
                        cudaStream_t stream);

}  // namespace lora
}  // namespace w8a8
