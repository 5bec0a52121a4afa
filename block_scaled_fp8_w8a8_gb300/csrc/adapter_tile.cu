// Low-rank adapters, many rows: tiles of 128 rows of one adapter on the tcgen05 tensor
// cores, in two launches with h = scales[l] x A[l]^T between them in fp32:
//
//   k_adapter_shrink   h[s] of a tile and the s-th part of K: x's rows (gathered by order)
//                      and A[l] through a ring of 64-column stages, r columns of TMEM
//   k_adapter_expand   a tile and some of the columns: the parts of K are added in order,
//                      h is split into 16-bit parts (adapter.cu says why) that are the MMA's
//                      A operand for all columns; tiles of B[l] and of base through a
//                      ring, the sums from TMEM added to base in shared memory, whole
//                      128-byte pieces of rows out
//
// HBM-bound: x, base and out pass once; the products' operands repeat from L2 and are small.
// Two launches, not one: either product then has as many CTAs as fill the SMs twice,
// whatever the number of tiles, and while one CTA of an SM fills its pipeline the other streams.
//
// 16384 rows of 16 adapters of rank 64, 4096x4096 in bf16: 88 us, 4.5 TB/s; the two launches' first
// loads and last stores are some 24 us of that, between them the copies run at HBM's rate.
//
// Rows lie anywhere, but mostly one after the other (a request's tokens): 32 rows of a tile
// that do are one TMA box, others are gathered four at a time.
#include "../../include/w8a8_block_fp8.h"
#include "adapter.cuh"

namespace w8a8 {
namespace {

using namespace lora;

constexpr uint32_t kTileRows = 128;
constexpr uint32_t kRowBytes = 128;                 // of an operand tile: 64 16-bit columns
constexpr uint32_t kTileBytes = kTileRows * kRowBytes;

// Instruction descriptor of kind::f16: idesc_f16_f32 with the operands' format.
template <bool BF16> __device__ __forceinline__ uint32_t idesc(uint32_t n)
{
    return idesc_f16_f32(128, n) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// (debug-bounds build)
__device__ __forceinline__ Buffer h_of(const TileParams &p)
{
    return {p.h, span(static_cast<long long>(p.splits) * p.a.T, p.a.r_pad, p.a.r_pad, 4), p.a.status, SITE_BOUNDS_WORKSPACE};
}

// Offset of 16-byte piece c of row r in a tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) { return r * kRowBytes + ((c ^ (r & 7u)) << 4); }

// Rows of a tile as a producer warp loads them: lane 8 i for the 32 rows of part i, if
// they follow one another (rows behind the item's last are then some others', whose sums go
// nowhere), else each of the part's lanes four of them, -1 as the row past the last: zeros.
// (All by four: 16384 rows in order, rank 64, 97 us; by boxes see k_adapter_expand.)
struct RowLoads {
    int row[4];
    uint32_t lane;
    bool box, any;
    __device__ __forceinline__ RowLoads(const int *list, int count, int T) : lane(lane_index())
    {
        const int first = list[lane / 8 * 32];
        bool follow = first >= 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = 4 * lane + i, r = list[at];
            follow = follow && (at >= count || r == first + (at & 31));
            row[i] = r >= 0 ? r : T;
        }
        const uint32_t yes = __ballot_sync(0xffffffffu, follow);
        box = (yes >> (lane & 24u) & 0xffu) == 0xffu;
        any = !box || (lane & 7u) == 0;
        if (box)
            row[0] = first;
    }
    __device__ __forceinline__ void operator()(uint32_t dst, const CUtensorMap *one, const CUtensorMap *boxes, uint32_t bar,
                                               int x, int cols, int T, unsigned *status, uint32_t site) const
    {
        const bool rows_in = box ? row[0] >= 0 && row[0] < T
                                 : min(min(row[0], row[1]), min(row[2], row[3])) >= 0 &&
                                       max(max(row[0], row[1]), max(row[2], row[3])) <= T;
        if (any && !in_bounds(rows_in && x >= 0 && x < cols, status, site))
            return;
        if (box && any)
            tma_load_2d(dst + lane * 4 * kRowBytes, boxes, bar, x, row[0]);
        else if (any)
            tma_gather4(dst + lane * 4 * kRowBytes, one, bar, x, row[0], row[1], row[2], row[3]);
    }
};

// After an abort: the loads still landing, the last into each stage of `issued` steps.
template <int STAGES> __device__ __forceinline__ void drain_loads(uint32_t full, int issued, unsigned *status,
                                                                  unsigned long long limit)
{
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        wait_drain(full + 8u * (i % STAGES), static_cast<uint32_t>(i / STAGES & 1), status, limit, (SITE_DRAIN << 8) | 4u);
}

// ------------------------------------------------------------------ x A^T

constexpr int kShrinkThreads = 192;         // warps 0-3 store h, 4 issues MMAs, 5 loads
constexpr int kMaxR = 128;

constexpr size_t shrink_smem(int r_pad, int stages)
{
    return 1024 + stages * (kTileBytes + static_cast<size_t>(r_pad) * kRowBytes);
}

template <bool BF16, int STAGES> __global__ void __launch_bounds__(kShrinkThreads) k_adapter_shrink(
    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_x32,
    const __grid_constant__ CUtensorMap map_a, const TileParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * STAGES + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, scratch[16], rows[kTileRows];
    const uint32_t warp = warp_uniform(warp_index()), lane = lane_index(), t = threadIdx.x;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8u * STAGES, done = empty + 8u * STAGES,
                   drain = done + 8u;
    const uint32_t stage_bytes = kTileBytes + p.a.r_pad * kRowBytes;
    uint32_t cols = 32;
    while (cols < static_cast<uint32_t>(p.a.r_pad))
        cols *= 2;
    if (t == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8u * s, 1);
            mbar_init(empty + 8u * s, 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        abort_word = 0;
        mbar_fence_init();
    }
    if (warp == 5 && lane == 0) {
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_x32);
        tma_prefetch_map(&map_a);
    }
    if (warp == 4) {
        tmem_alloc(smem_addr(&tmem_slot), cols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    // (only now: the second launch reads base and B before it waits for this one, so what
    // made those has to be finished when it starts; and only when this CTA has its TMEM,
    // which the second launch's CTAs hold while they wait)
    if (warp == 4)
        grid_launch_dependents();
    const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const Item item = find_item<kShrinkThreads>(p.a, tile, kTileRows, p.a.L, scratch);
    if (t < kTileRows) {
        rows[t] = static_cast<int>(t) < item.rows ? row_in_place(p.a, item.first + static_cast<int>(t)) : -1;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const WaitGuard guard{&abort_word, p.a.status, p.a.wait_limit};
    const int blocks = (p.a.K + 63) / 64;
    const int lo = static_cast<int>(static_cast<long long>(blocks) * split / p.splits);
    const bool some = item.rows && in_bounds(item.first >= 0 && item.first + item.rows <= p.a.T && item.adapter < p.a.L,
                                             p.a.status, SITE_BOUNDS_A);
    const int steps = some ? static_cast<int>(static_cast<long long>(blocks) * (split + 1) / p.splits) - lo : 0;
    if (warp < 4 && steps) {
        // h of this part of K
        if (__all_sync(0xffffffffu, wait_bounded(done, 0, guard, SITE_TILED_PROMOTE))) {
            tc_fence_after_sync();
            const float scale = scale_of(p.a, item.adapter);
            float *const h = p.h + (static_cast<long long>(split) * p.a.T + item.first + t) * p.a.r_pad;
            for (int j = 0; j < p.a.r_pad; j += 32) {
                float v[32];
                __syncwarp();
                tmem_load_32cols(tmem + ((warp * 32u) << 16) + j, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (static_cast<int>(t) < item.rows && j + i < p.a.r_pad && h_of(p).holds(h + j + i, 16))
                        *reinterpret_cast<float4 *>(h + j + i) =
                            make_float4(v[i] * scale, v[i + 1] * scale, v[i + 2] * scale, v[i + 3] * scale);
            }
        }
    } else if (warp == 4 && steps) {
        const uint32_t d = idesc<BF16>(p.a.r_pad);
        bool ok = true;
        for (int i = 0; i < steps && ok; ++i) {
            const int s = i % STAGES;
            ok = __all_sync(0xffffffffu, wait_bounded(full + 8u * s, static_cast<uint32_t>(i / STAGES & 1), guard,
                                                      SITE_TILED_MMA_FULL));
            if (!ok)
                break;
            tc_fence_after_sync();
            const uint64_t ad = sw128_kmajor_desc(smem + s * stage_bytes);
            const uint64_t bd = sw128_kmajor_desc(smem + s * stage_bytes + kTileBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_f16_elect<false>(tmem, ad + 2u * k, bd + 2u * k, d, i + k > 0);
            mma_commit_elect<false>(empty + 8u * s);
        }
        if (ok)
            mma_commit_elect<false>(done);
        // no commit arrives on this CTA's shared memory after it exits
        mma_commit_elect<false>(drain);
        wait_drain(drain, 0, p.a.status, p.a.wait_limit, (SITE_DRAIN << 8) | 4u);
    } else if (warp == 5 && steps) {
        const RowLoads load(rows, item.rows, p.a.T);
        int i = 0;
        for (; i < steps; ++i) {
            const int s = i % STAGES;
            if (!__all_sync(0xffffffffu, wait_bounded(empty + 8u * s, static_cast<uint32_t>(i / STAGES & 1) ^ 1u,
                                                      guard, SITE_TILED_PRODUCER)))
                break;
            const uint32_t dst = smem + s * stage_bytes, bar = full + 8u * s;
            const int k = (lo + i) * 64;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, stage_bytes);
                if (in_bounds(k >= 0 && k < p.a.K && item.adapter >= 0 && item.adapter < p.a.L, p.a.status, SITE_BOUNDS_B))
                    tma_load_3d(dst + kTileBytes, &map_a, bar, k, 0, item.adapter);
            }
            __syncwarp();
            load(dst, &map_x, &map_x32, bar, k, p.a.K, p.a.T, p.a.status, SITE_BOUNDS_A);
        }
        if (i < steps)
            drain_loads<STAGES>(full, i, p.a.status, p.a.wait_limit);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, cols);
    }
}

// ------------------------------------------------------------------ base + h B^T

constexpr int kExpandThreads = 192;         // warps 0-3 epilogue, 4 issues MMAs, 5 loads

template <bool BF16, int OUT> struct Expand {
    static constexpr int kTerms = BF16 && OUT == W8A8_OUT_FP32 ? 3 : 2;
    static constexpr int kEach = OUT == W8A8_OUT_FP32 ? 4 : 8;          // elements of 16 bytes
    static constexpr int kCols = 8 * kEach;                             // of a column tile
    static constexpr uint32_t kBBytes = kCols * kRowBytes;              // for 64 columns of r
    static __host__ __device__ constexpr uint32_t stage_bytes(int k_blocks) { return k_blocks * kBBytes + kTileBytes; }
    static constexpr size_t smem(int k_blocks, int stages)
    {
        return 1024 + static_cast<size_t>(kTerms) * k_blocks * kTileBytes + static_cast<size_t>(stages) * stage_bytes(k_blocks);
    }
};

template <bool BF16, int OUT, int STAGES>
__global__ void __launch_bounds__(kExpandThreads) k_adapter_expand(
    const __grid_constant__ CUtensorMap map_base, const __grid_constant__ CUtensorMap map_base32,
    const __grid_constant__ CUtensorMap map_b, const TileParams p)
{
    using X = Expand<BF16, OUT>;
    constexpr int kCols = X::kCols, kEach = X::kEach, kTerms = X::kTerms, kOut = 16 / kEach;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * STAGES + 6];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, scratch[16], rows[kTileRows];
    const uint32_t warp = warp_uniform(warp_index()), lane = lane_index(), t = threadIdx.x;
    const uint32_t pad = ((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw);
    const int k_blocks = (p.a.r_pad + 63) / 64;
    const uint32_t operand = smem_addr(smem_raw) + pad;
    const uint32_t ring_at = pad + kTerms * k_blocks * kTileBytes, ring = smem_addr(smem_raw) + ring_at;
    const uint32_t stage_bytes = X::stage_bytes(k_blocks), base_at = k_blocks * X::kBBytes;
    const uint32_t full = smem_addr(bars), empty = full + 8u * STAGES, h_full = empty + 8u * STAGES, d_full = h_full + 8u,
                   d_empty = d_full + 16u, drain = d_empty + 16u;
    if (t == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8u * s, 1);
            mbar_init(empty + 8u * s, 5);       // the MMAs' commit and four epilogue warps
        }
        mbar_init(h_full, 128);
        for (int b = 0; b < 2; ++b) {
            mbar_init(d_full + 8u * b, 1);
            mbar_init(d_empty + 8u * b, 4);
        }
        mbar_init(drain, 1);
        abort_word = 0;
        mbar_fence_init();
    }
    if (warp == 5 && lane == 0) {
        tma_prefetch_map(&map_base);
        tma_prefetch_map(&map_base32);
        tma_prefetch_map(&map_b);
    }
    if (warp == 4) {
        tmem_alloc(smem_addr(&tmem_slot), 2 * kCols);
        tmem_relinquish();
    }
    const int tile = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const Item item = find_item<kExpandThreads>(p.a, tile, kTileRows, p.a.out == p.a.base ? p.a.L : p.a.L + 1, scratch);
    if (t < kTileRows) {
        rows[t] = static_cast<int>(t) < item.rows ? row_in_place(p.a, item.first + static_cast<int>(t)) : -1;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const WaitGuard guard{&abort_word, p.a.status, p.a.wait_limit};
    const int col_tiles = (p.a.N + kCols - 1) / kCols;
    const int lo = static_cast<int>(static_cast<long long>(col_tiles) * chunk / p.chunks);
    const int hi = static_cast<int>(static_cast<long long>(col_tiles) * (chunk + 1) / p.chunks);
    const bool some = item.rows && item.adapter < p.a.L &&
                      in_bounds(item.first >= 0 && item.first + item.rows <= p.a.T, p.a.status, SITE_BOUNDS_B);
    const int steps = some ? hi - lo : 0;
    char *const out = static_cast<char *>(p.a.out);
    if (warp == 5 && steps) {
        // (h alone is the first launch's: nothing here waits for it)
        const RowLoads load(rows, item.rows, p.a.T);
        int i = 0;
        for (; i < steps; ++i) {
            const int s = i % STAGES;
            if (!__all_sync(0xffffffffu, wait_bounded(empty + 8u * s, static_cast<uint32_t>(i / STAGES & 1) ^ 1u, guard,
                                                      SITE_TILED_PRODUCER)))
                break;
            const uint32_t dst = ring + s * stage_bytes, bar = full + 8u * s;
            const int n0 = (lo + i) * kCols;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, stage_bytes);
                for (int q = 0; q < k_blocks; ++q)
                    if (in_bounds(n0 >= 0 && n0 < p.a.N && 64 * q < p.a.r && item.adapter >= 0 && item.adapter < p.a.L,
                                  p.a.status, SITE_BOUNDS_B))
                        tma_load_3d(dst + q * X::kBBytes, &map_b, bar, 64 * q, n0, item.adapter);
            }
            __syncwarp();
            load(dst + base_at, &map_base, &map_base32, bar, n0, p.a.N, p.a.T, p.a.status, SITE_BOUNDS_C);
        }
        if (i < steps)
            drain_loads<STAGES>(full, i, p.a.status, p.a.wait_limit);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp < 4 && steps) {
        // ---------------------------------------------------- h's parts, then the epilogue
        const uint32_t e = warp, row = e * 32 + lane;
        const float *const h = p.h + (static_cast<long long>(item.first) + row) * p.a.r_pad;
        const bool mine = static_cast<int>(row) < item.rows;
        const long long plane = static_cast<long long>(p.a.T) * p.a.r_pad;
        // 32 columns at a time, the loads of a part of K together (r_pad is a multiple of 16)
        auto load = [&](int k, float (&v)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = 0.f;
            if (!mine)
                return;
            for (int s = 0; s < p.splits; ++s) {
                float4 a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    a[i] = (i < 4 || k + 16 < p.a.r_pad) && h_of(p).holds(h + s * plane + k + 4 * i, 16)
                               ? *reinterpret_cast<const float4 *>(h + s * plane + k + 4 * i)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[4 * i] += a[i].x, v[4 * i + 1] += a[i].y, v[4 * i + 2] += a[i].z, v[4 * i + 3] += a[i].w;
            }
        };
        float factor = 1.f, shrink = 1.f;
        if constexpr (!BF16) {
            float top = 0.f;
            for (int k = 0; k < p.a.r_pad; k += 32) {
                float v[32];
                load(k, v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    top = fmaxf(top, fabsf(v[i]));
            }
            power_of(top, &shrink, &factor);
        }
#pragma unroll 2
        for (int k = 0; k < p.a.r_pad; k += 32) {
            float v[32];
            load(k, v);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (k + 8 * c >= p.a.r_pad)
                    continue;
#pragma unroll
                for (int q = 0; q < kTerms; ++q) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!BF16 && q == 0)
                            v[8 * c + i] *= shrink;
                        w[i] = take_part<BF16>(v[8 * c + i]);
                    }
                    const uint32_t at = operand + (q * k_blocks + k / 64) * kTileBytes + swizzled(row, (k & 63) / 8 + c);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[1] << 16 | w[0]),
                                 "r"(w[3] << 16 | w[2]), "r"(w[5] << 16 | w[4]), "r"(w[7] << 16 | w[6])
                                 : "memory");
                }
            }
        }
        fence_async_smem();
        mbar_arrive(h_full);
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int s = i % STAGES, b = i & 1;
            ok = __all_sync(0xffffffffu,
                            wait_bounded(full + 8u * s, static_cast<uint32_t>(i / STAGES & 1), guard, SITE_TILED_PROMOTE) &&
                                wait_bounded(d_full + 8u * b, static_cast<uint32_t>(i / 2 & 1), guard, SITE_TILED_PROMOTE));
            if (!ok)
                break;
            tc_fence_after_sync();
            const uint32_t tile_at = ring_at + s * stage_bytes + base_at;
            uint8_t *const tile_rows = smem_raw + tile_at;
#pragma unroll
            for (int j = 0; j < kCols; j += 32) {
                float v[32];
                tmem_load_32cols(tmem + ((e * 32u) << 16) + b * kCols + j, v);
                if (j + 32 == kCols) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(d_empty + 8u * b);
                }
#pragma unroll
                for (int q = 0; q < 32; q += kEach) {
                    uint4 *const piece = reinterpret_cast<uint4 *>(tile_rows + swizzled(row, (j + q) / kEach));
                    const uint4 u = *piece;
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    uint32_t o[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        if constexpr (OUT == W8A8_OUT_FP32) {
                            o[z] = __float_as_uint(fmaf(v[q + z], factor, __uint_as_float(w[z])));
                        } else if constexpr (BF16) {
                            o[z] = pack_bf16x2(v[q + 2 * z] + __uint_as_float(w[z] << 16),
                                               v[q + 2 * z + 1] + __uint_as_float(w[z] & 0xffff0000u));
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[z]));
                            o[z] = pack_f16x2(fmaf(v[q + 2 * z], factor, f.x), fmaf(v[q + 2 * z + 1], factor, f.y));
                        }
                    }
                    *piece = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            __syncwarp();
            // out: eight lanes to a row's 128 bytes
            const uint32_t c = lane & 7u;
            const int col = (lo + i) * kCols + static_cast<int>(c) * kEach;
            if (col < p.a.N)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t r = e * 32 + (lane >> 3) + 4 * j;
                    const int to = rows[r];
                    if (to >= 0 && out_of(p.a, kOut).holds(out + (to * p.a.ld_out + col) * kOut, 16))
                        *reinterpret_cast<uint4 *>(out + (to * p.a.ld_out + col) * kOut) =
                            *reinterpret_cast<const uint4 *>(tile_rows + swizzled(r, c));
                }
            fence_async_smem();         // these accesses before the next load's
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty + 8u * s);
        }
    } else if (warp == 4 && steps) {
        // ---------------------------------------------------- MMAs
        const uint32_t d = idesc<BF16>(kCols);
        bool ok = __all_sync(0xffffffffu, wait_bounded(h_full, 0, guard, SITE_TILED_MMA_FULL));
        for (int i = 0; i < steps && ok; ++i) {
            const int s = i % STAGES, b = i & 1;
            ok = __all_sync(0xffffffffu, wait_bounded(d_empty + 8u * b, static_cast<uint32_t>(i / 2 & 1) ^ 1u, guard,
                                                      SITE_TILED_MMA_TMEM) &&
                                             wait_bounded(full + 8u * s, static_cast<uint32_t>(i / STAGES & 1), guard,
                                                          SITE_TILED_MMA_FULL));
            if (!ok)
                break;
            tc_fence_after_sync();
            uint32_t more = 0;
            for (int q = 0; q < k_blocks; ++q) {
                const uint64_t bd = sw128_kmajor_desc(ring + s * stage_bytes + q * X::kBBytes);
                const int ks = min(4, (p.a.r_pad - 64 * q) / 16);
                for (int z = 0; z < kTerms; ++z) {
                    const uint64_t ad = sw128_kmajor_desc(operand + (z * k_blocks + q) * kTileBytes);
                    for (int k = 0; k < ks; ++k) {
                        mma_f16_elect<false>(tmem + b * kCols, ad + 2u * k, bd + 2u * k, d, more);
                        more = 1;
                    }
                }
            }
            mma_commit_elect<false>(empty + 8u * s);
            mma_commit_elect<false>(d_full + 8u * b);
        }
        // no commit arrives on this CTA's shared memory, and none reads it, after it exits
        mma_commit_elect<false>(drain);
        wait_drain(drain, 0, p.a.status, p.a.wait_limit, (SITE_DRAIN << 8) | 4u);
    }
    if (item.rows && item.adapter == p.a.L) {
        // rows without an adapter
        copy_rows<uint4, kExpandThreads>(p.a, rows, item.rows, lo * kCols, min(hi * kCols, p.a.N), kOut);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 2 * kCols);
    }
}

// Tiles of a problem where half of the adapters' last ones are full (the most there can be are
// launched; those without rows leave at once).
long long likely_tiles(const AdapterParams &p) { return p.T / kTileRows + std::min(p.T, p.L) / 2 + 1; }

template <class Kernel>
cudaError_t launch(Kernel kernel, const CUtensorMap (&rows)[2], const CUtensorMap &weights, const TileParams &p,
                   long long ctas, int threads, size_t smem, volatile int *flags, cudaStream_t stream)
{
    if (const cudaError_t e = allow_smem(kernel, 224 * 1024, flags); e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    lc.blockDim = dim3(threads, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, rows[0], rows[1], weights, p);
}

template <bool BF16, int OUT, int STAGES>
cudaError_t launch_expand(const CUtensorMap (&rows)[2], const CUtensorMap &weights, const TileParams &p, long long ctas,
                          cudaStream_t s)
{
    static volatile int flags[kMaxDeviceFlags] = {};
    return launch(k_adapter_expand<BF16, OUT, STAGES>, rows, weights, p, ctas, kExpandThreads,
                  Expand<BF16, OUT>::smem((p.a.r_pad + 63) / 64, STAGES), flags, s);
}

template <bool BF16, int STAGES>
cudaError_t launch_shrink(const CUtensorMap (&rows)[2], const CUtensorMap &weights, const TileParams &p, long long ctas,
                          cudaStream_t s)
{
    static volatile int flags[kMaxDeviceFlags] = {};
    return launch(k_adapter_shrink<BF16, STAGES>, rows, weights, p, ctas, kShrinkThreads, shrink_smem(p.a.r_pad, STAGES), flags,
                  s);
}

// Rows of 128 bytes: boxes of one row, which are gathered, and of 32.
cudaError_t rows_maps(CUtensorMap (&map)[2], int kind, const void *base, int64_t rows, int64_t cols, int64_t ld)
{
    const int element = kind == W8A8_OUT_FP32 ? 4 : 2;
    const uint64_t sizes[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)},
                   strides[1] = {static_cast<uint64_t>(ld) * element};
    const uint32_t one[2] = {kRowBytes / element, 1}, boxes[2] = {kRowBytes / element, 32};
    const cudaError_t e = encode_rows_map(&map[0], kind, 2, base, sizes, strides, one);
    return e == cudaSuccess ? encode_rows_map(&map[1], kind, 2, base, sizes, strides, boxes) : e;
}

// The adapters' weights [L, rows, cols]: boxes of 64 columns of `high` rows.
cudaError_t weights_map(CUtensorMap *map, int kind, const void *base, int64_t L, int64_t rows, int64_t cols, int high)
{
    const uint64_t sizes[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(L)},
                   strides[2] = {static_cast<uint64_t>(cols) * 2, static_cast<uint64_t>(cols) * rows * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(high), 1};
    return encode_rows_map(map, kind, 3, base, sizes, strides, box);
}

template <bool BF16, int OUT> cudaError_t launch_both(TileParams p, const DeviceView &dev, cudaStream_t stream)
{
    using X = Expand<BF16, OUT>;
    constexpr int kKind = BF16 ? W8A8_OUT_BF16 : W8A8_OUT_FP16;
    CUtensorMap map_x[2], map_base[2], map_a, map_b;
    cudaError_t e = rows_maps(map_x, kKind, p.a.x, p.a.T, p.a.K, p.a.ld_x);
    if (e == cudaSuccess)
        e = weights_map(&map_a, kKind, p.a.A, p.a.L, p.a.r, p.a.K, p.a.r_pad);
    if (e == cudaSuccess)
        e = rows_maps(map_base, OUT, p.a.base, p.a.T, p.a.N, p.a.ld_base);
    if (e == cudaSuccess)
        e = weights_map(&map_b, kKind, p.a.B, p.a.L, p.a.N, p.a.r, X::kCols);
    if (e != cudaSuccess)
        return e;
    const long long tiles = most_items(p.a.T, p.a.L, kTileRows);
    // stages that leave room for two CTAs on an SM
    e = p.a.r_pad <= 64 ? launch_shrink<BF16, 4>(map_x, map_a, p, tiles * p.splits, stream)
                        : launch_shrink<BF16, 3>(map_x, map_a, p, tiles * p.splits, stream);
    if (e != cudaSuccess)
        return e;
    const long long all = most_items(p.a.T, p.a.out == p.a.base ? p.a.L : p.a.L + 1, kTileRows);
    const int col_tiles = (p.a.N + X::kCols - 1) / X::kCols;
    const int k_blocks = (p.a.r_pad + 63) / 64;
    // Two CTAs to an SM where three stages leave room for them; as many CTAs as fill the
    // SMs, with at least four column tiles each.
    const bool two = X::smem(k_blocks, 3) + 2048 <= 113 * 1024;
    p.chunks = static_cast<int>(
        std::max(1ll, std::min<long long>((two ? 2ll : 1ll) * dev.sm_count / likely_tiles(p.a), col_tiles / 4)));
    return two ? launch_expand<BF16, OUT, 3>(map_base, map_b, p, all * p.chunks, stream)
               : launch_expand<BF16, OUT, 4>(map_base, map_b, p, all * p.chunks, stream);
}

}  // namespace

namespace lora {

bool tile_takes(const AdapterParams &p)
{
    return p.r >= 8 && p.r <= kMaxR && p.r % 8 == 0 && p.K >= 64 && p.vec_k && p.vec_n &&
           reinterpret_cast<uintptr_t>(p.B) % 16 == 0;
}

// (The workspace's size goes by it: a GB300's SMs, so that no device is asked.)
constexpr int kSms = 152;
int tile_splits(const AdapterParams &p)
{
    // CTAs that fill the SMs twice, with at least four steps of 64 columns each
    return static_cast<int>(std::max(1ll, std::min<long long>({2ll * kSms / likely_tiles(p), p.K / 256, 8})));
}

cudaError_t launch_tile(const AdapterParams &a, int x_kind, int out_kind, float *h, const DeviceView &dev, cudaStream_t stream)
{
    TileParams p = {};
    p.a = a;
    p.h = h;
    p.splits = tile_splits(a);
    if (x_kind == W8A8_IN_BF16)
        return out_kind == W8A8_OUT_FP32 ? launch_both<true, W8A8_OUT_FP32>(p, dev, stream)
                                         : launch_both<true, W8A8_OUT_BF16>(p, dev, stream);
    return out_kind == W8A8_OUT_FP32 ? launch_both<false, W8A8_OUT_FP32>(p, dev, stream)
                                     : launch_both<false, W8A8_OUT_FP16>(p, dev, stream);
}

}  // namespace lora
}  // namespace w8a8
