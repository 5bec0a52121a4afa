// The ragged grouped matmul (see gemm_ragged.cu for the formula and the offsets)
// where experts have few rows: k_ragged_few.
//
// The weights of the experts that have rows bound the time, so nothing else may
// take longer than their bytes: weights lie on the MMA's M side (128 of them: one
// scale block) and up to 32 rows of A on its N side, which makes a K group's MMAs,
// its partial in tensor memory and its promotion a quarter of the row-major
// tile's, and a pipeline stage 20 KB.  Two CTAs fit an SM; each walks items of
// (32-row tile, 128 weight rows), and its ring runs across them, so the stream of
// weights does not pause between experts.
// Where that leaves SMs without an item (a few rows of a few experts), the CTAs of
// a cluster share one: each takes a range of its K groups, leaves its fp32 partial
// rows in shared memory, and they are added in rank order through distributed
// shared memory.
//
// Bound by the weights' bytes where the items fill the GPU (512 rows of 256 experts,
// 1536 x 4096: 186 to 190 us, 6.8 TB/s); otherwise by the latency of launch, offsets, first
// loads and the cluster's sum, some 7 us, and by what a K group takes to pass from
// load to promotion in one CTA, some 600 cycles (8 rows of 256 experts, 1536 x 4096,
// split over two CTAs: 14.6 to 15.6 us; unsplit 17.3).
//
// Roles: warps 0 and 3 TMA producers, warp 1 MMA issuer, warp 2 scale loader, warps 4..7
// promotion (a thread owns one weight row, the partial's columns are rows of A).
#include "kernels.cuh"
#include "ptx.cuh"
#include "ragged.cuh"

namespace w8a8 {

namespace {

constexpr int kRows = 32;                  // rows of A per tile
constexpr int kStages = 4;                 // even: a stage has one producer
constexpr int kBufs = 8;                   // partials in tensor memory, 32 columns each
constexpr int kSlots = 8, kSlotFloats = 40;     // 32 a_s values, one b_s, padding
constexpr int kThreads = 256;
constexpr uint32_t kWBytes = 128 * 128, kXBytes = kRows * 128;
constexpr size_t kStageBytes = kStages * (kWBytes + kXBytes);
constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 1;
constexpr size_t kSmem = 1024 + kStageBytes + kSlots * kSlotFloats * 4 + kBars * 8 + 8 + 16 + 64 +
                         2 * (kRaggedMaxExperts + 1) * 4;
static_assert(kSmem <= 115712, "two CTAs per SM");
static_assert(kRows * 128 * 4 <= kStageBytes, "the partial rows take the stages' place");

__global__ void __launch_bounds__(kThreads, 2)
    k_ragged_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const RaggedParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sW = smem_addr(smem), sX = sW + kStages * kWBytes;
    float *scales = reinterpret_cast<float *>(smem + kStageBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(scales + kSlots * kSlotFloats);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + kBufs + b); };
    auto sfull_bar = [&](int q) { return bar0 + 8u * (2 * kStages + 2 * kBufs + q); };
    auto sempty_bar = [&](int q) { return bar0 + 8u * (2 * kStages + 2 * kBufs + kSlots + q); };
    const uint32_t drain_bar = bar0 + 8u * (kBars - 1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *warp_part = reinterpret_cast<volatile int *>(tmem_slot + 2);    // 8 words
    int *row0 = reinterpret_cast<int *>(tmem_slot + 18);
    int *tile0 = row0 + kRaggedMaxExperts + 1;
    const uint32_t warp = warp_uniform(warp_index()), lane = lane_index();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);
        }
        for (int q = 0; q < kSlots; ++q) {
            mbar_init(sfull_bar(q), 32);
            mbar_init(sempty_bar(q), 4);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), kBufs * kRows);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = warp_uniform(*tmem_slot);
    const WaitGuard guard{abort_flag, p.status, p.wait_limit};

    grid_launch_dependents();
    grid_dependency_wait();

    // The cluster's items, and this CTA's K groups of each.  With a split the grid
    // holds a cluster for every item there can be.
    const int S = p.split, rank = static_cast<int>(blockIdx.x) % S;
    const int first = static_cast<int>(blockIdx.x) / S, step = static_cast<int>(gridDim.x) / S;
    const int g0 = p.G * rank / S, g1 = p.G * (rank + 1) / S;
    make_tile_list<kThreads, kRows>(p, row0, tile0, warp_part);

    if (warp == 0 || warp == 3) {
        // -------------------------------------------------------------- TMA producers
        // One for the even groups, one for the odd: two loads take a warp some 500
        // cycles, the MMAs and the promotion of a group less.
        const int me = warp == 0 ? 0 : 1;
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;             // groups so far, both producers'
        bool ok = true;
        RaggedWalk<kRows> w(p, row0, tile0, first);
        while (ok && w.next(step)) {
            for (int g = g0; g < g1; ++g) {
                if ((stage & 1) == me) {
                    ok = __all_sync(0xffffffffu, wait_bounded(empty_bar(stage), phase ^ 1u, guard,
                                                              SITE_TILED_PRODUCER));
                    if (!ok)
                        break;
                    const int arow = w.m0 + ((W8A8_DEBUG_BOUNDS && issued == 0 &&
                                              p.debug_skip_tma == kDebugBadFirstLoad)
                                                 ? (1 << 28)
                                                 : 0);
                    const bool in =
                        in_bounds(arow >= 0 && arow < p.M && g * 128 < p.K, p.status, SITE_BOUNDS_A) &&
                        in_bounds(w.nb * 128 < p.N && w.e < p.experts, p.status, SITE_BOUNDS_B);
                    if (issued != p.debug_skip_tma && in && elect_one()) {
                        mbar_arrive_expect_tx(full_bar(stage), kWBytes + kXBytes);
                        tma_load_3d(sW + stage * kWBytes, &tmB, full_bar(stage), g * 128, w.nb * 128,
                                    w.e);
                        tma_load_2d(sX + stage * kXBytes, &tmA, full_bar(stage), g * 128, arow);
                    }
                }
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        const int next_stage = stage;
        const uint32_t next_phase = phase;
        // Tail: wait until the MMA has released every stage, so that no commit
        // arrives on this CTA's shared memory after it exits.
        for (int s = 0; s < kStages && ok; ++s) {
            if ((stage & 1) == me)
                ok = __all_sync(0xffffffffu, wait_bounded(empty_bar(stage), phase ^ 1u, guard,
                                                          SITE_TILED_PRODUCER));
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {
            // Drain: this producer's loads still landing (the last into each stage).
            for (int s = me; s < kStages; s += 2) {
                const bool this_round = s < next_stage;
                if (!this_round && issued < kStages && s >= issued)
                    continue;
                wait_drain(full_bar(s), this_round ? next_phase : (next_phase ^ 1u), p.status,
                           p.wait_limit, (SITE_DRAIN << 8) | 4u);
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA issuer
        constexpr uint32_t idesc = idesc_e4m3_f32(128, kRows);
        int stage = 0;
        uint32_t phase = 0, it = 0;
        bool ok = true;
        const int items = tile0[p.experts] * p.num_n_tiles;
        for (int item = first; ok && item < items; item = item < items - step ? item + step : items) {
            for (int g = g0; g < g1; ++g, ++it) {
                const uint32_t buf = it % kBufs;
                ok = __all_sync(0xffffffffu,
                                wait_bounded(tempty_bar(buf), ((it / kBufs) & 1u) ^ 1u, guard,
                                             SITE_TILED_MMA_TMEM) &&
                                    wait_bounded(full_bar(stage), phase, guard, SITE_TILED_MMA_FULL));
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + buf * kRows;
                const uint64_t wd = sw128_kmajor_desc(sW + stage * kWBytes);
                const uint64_t xd = sw128_kmajor_desc(sX + stage * kXBytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_e4m3_elect(d, wd + 2u * kk, xd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                mma_commit_elect<false>(empty_bar(stage));
                mma_commit_elect<false>(tfull_bar(buf));
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
            // an aborting CTA frees its tensor memory only after its MMAs have completed
            mma_commit_elect<false>(drain_bar);
            wait_drain(drain_bar, 0, p.status, p.wait_limit, (SITE_DRAIN << 8) | 4u);
        }
    } else if (warp == 2) {
        // -------------------------------------------------------------- scale loader
        int slot = 0;
        uint32_t sphase = 0;
        bool ok = true;
        RaggedWalk<kRows> w(p, row0, tile0, first);
        while (ok && w.next(step)) {
            const bool mine = static_cast<int>(lane) < w.rows;
            const float *a = p.a_s + static_cast<size_t>(w.m0 + (mine ? lane : 0)) * p.G;
            const float *b = p.b_s + (static_cast<size_t>(w.e) * p.NB + w.nb) * p.G;
            for (int g = g0; g < g1; ++g) {
                ok = __all_sync(0xffffffffu,
                                wait_bounded(sempty_bar(slot), sphase ^ 1u, guard, SITE_TILED_SCALES));
                if (!ok)
                    break;
                const uint32_t dst = smem_addr(scales + slot * kSlotFloats);
                if (mine)
                    cp_async_4(dst + 4u * lane, a + g, 4u);
                if (lane == 0)
                    cp_async_4(dst + 4u * kRows, b + g, 4u);
                cp_async_arrive(sfull_bar(slot));
                if (++slot == kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
        }
        // Let every gather land before the CTA can exit.
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        // -------------------------------------------------------------- promotion + stores
        const uint32_t q = warp & 3u;
        const int col = static_cast<int>(q * 32 + lane);
        const bool fp32 = p.out_kind == OUT_FP32, bf = p.out_kind == OUT_BF16;
        int slot = 0;
        uint32_t sphase = 0, it = 0;
        RaggedWalk<kRows> w(p, row0, tile0, first);
        while (w.next(step)) {
            const int n = w.nb * 128 + col;
            const bool idle = w.nb * 128 + static_cast<int>(q * 32) >= p.N;
            uint64_t acc[kRows / 2];
#pragma unroll
            for (int j = 0; j < kRows / 2; ++j)
                acc[j] = 0ull;
            bool ok = true;
            for (int g = g0; g < g1; ++g, ++it) {
                const uint32_t buf = it % kBufs;
                ok = __all_sync(
                    0xffffffffu,
                    wait_bounded(sfull_bar(slot), sphase, guard, SITE_TILED_PROMOTE) &&
                        wait_bounded(tfull_bar(buf), (it / kBufs) & 1u, guard, SITE_TILED_PROMOTE));
                if (!ok)
                    break;
                tc_fence_after_sync();
                const float *sl = scales + slot * kSlotFloats;
                if (!idle) {
                    uint32_t v[kRows];
                    tmem_ld32_async(tmem_base + ((q * 32u) << 16) + buf * kRows, v);
                    const uint64_t b2 = pack2f(sl[kRows], sl[kRows]);
                    tmem_wait_ld32(v);
                    // eight rows at a time, as far as there are any
#pragma unroll
                    for (int c = 0; c < kRows / 8; ++c)
                        if (8 * c < w.rows) {
                            const float4 x = *reinterpret_cast<const float4 *>(sl + 8 * c);
                            const float4 y = *reinterpret_cast<const float4 *>(sl + 8 * c + 4);
                            fma2(acc[4 * c], mul2_rn(pack2f(x.x, x.y), b2), pack2(v[8 * c], v[8 * c + 1]));
                            fma2(acc[4 * c + 1], mul2_rn(pack2f(x.z, x.w), b2),
                                 pack2(v[8 * c + 2], v[8 * c + 3]));
                            fma2(acc[4 * c + 2], mul2_rn(pack2f(y.x, y.y), b2),
                                 pack2(v[8 * c + 4], v[8 * c + 5]));
                            fma2(acc[4 * c + 3], mul2_rn(pack2f(y.z, y.w), b2),
                                 pack2(v[8 * c + 6], v[8 * c + 7]));
                        }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(sempty_bar(slot));
                    mbar_arrive(tempty_bar(buf));
                }
                if (++slot == kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
            if (!ok)
                break;
            float *part = reinterpret_cast<float *>(smem) + col;
            const bool store = n < p.N && in_bounds(w.m0 >= 0 && w.m0 + w.rows <= p.M, p.status,
                                                    SITE_BOUNDS_C);
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (j < w.rows) {
                    float x, y;
                    unpack2f(acc[j / 2], x, y);
                    const float v = (j & 1) ? y : x;
                    const size_t to = static_cast<size_t>(w.m0 + j) * p.N + n;
                    if (S > 1)
                        // Every group's MMA has completed (its partial was read), so
                        // the stages are free.
                        part[128 * j] = v;
                    else if (store && fp32)
                        static_cast<float *>(p.C)[to] = v;
                    else if (store && bf)
                        static_cast<__nv_bfloat16 *>(p.C)[to] = __float2bfloat16_rn(v);
                    else if (store)
                        static_cast<__half *>(p.C)[to] = __float2half_rn(v);
                }
        }
    }
    __syncwarp();

    if (S > 1) {
        cluster_sync();               // the partial rows are in shared memory
        RaggedWalk<kRows> w(p, row0, tile0, first);
        if (warp >= 4 && w.next(step)) {
            // The CTAs share the tile's rows, in pieces of four columns.
            const bool fp32 = p.out_kind == OUT_FP32, bf = p.out_kind == OUT_BF16;
            const uint32_t base = smem_addr(smem);
            for (int u = rank * 128 + static_cast<int>(threadIdx.x) - 128; u < w.rows * 32; u += S * 128) {
                const int r = u / 32, n = w.nb * 128 + 4 * (u % 32);
                if (n >= p.N || !in_bounds(w.m0 + r < p.M && n + 4 <= p.N, p.status, SITE_BOUNDS_C))
                    continue;
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)          // every load before the first addition
                    if (i < S)
                        v[i] = ld_cluster_f4(cluster_map(base + 16u * u, static_cast<uint32_t>(i)));
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i < S) {
                        v[0].x += v[i].x;
                        v[0].y += v[i].y;
                        v[0].z += v[i].z;
                        v[0].w += v[i].w;
                    }
                const size_t to = static_cast<size_t>(w.m0 + r) * p.N + n;
                if (fp32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + to) = v[0];
                else
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + to) =
                        bf ? make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[0].z, v[0].w))
                           : make_uint2(pack_f16x2(v[0].x, v[0].y), pack_f16x2(v[0].z, v[0].w));
            }
        }
        __syncwarp();
        cluster_sync();               // and have been read
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, kBufs * kRows);
    }
}

cudaError_t launch(const CUtensorMap &tmA, const CUtensorMap &tmB, const RaggedParams &p, int grid,
                   cudaStream_t stream, int *clusters)
{
    static volatile int smem_set[kMaxDeviceFlags] = {};
    cudaError_t e = ensure_smem_limit(k_ragged_few, smem_set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid, 1, 1);
    lc.blockDim = dim3(kThreads, 1, 1);
    lc.dynamicSmemBytes = kSmem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    // the kernel waits for the work before it ahead of its first access
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = clusters ? 0 : 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = p.split > 1 || clusters ? 2 : 1;
    if (clusters)
        return cudaOccupancyMaxActiveClusters(clusters, k_ragged_few, &lc);
    return cudaLaunchKernelEx(&lc, k_ragged_few, tmA, tmB, p);
}

}  // namespace

int ragged_few_clusters(int split)
{
    static volatile int cached[kMaxDeviceFlags][9] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDeviceFlags)
        return 0;
    if (cached[dev][split])
        return cached[dev][split];
    const CUtensorMap none = {};
    RaggedParams p = {};
    p.split = split;
    if (launch(none, none, p, split, nullptr, &n) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    // The query counts one CTA per SM for kernels that allocate tensor memory; the
    // shared memory, registers and columns above leave room for two.
    cached[dev][split] = 2 * n;
    return 2 * n;
}

cudaError_t launch_ragged_few(const CUtensorMap &tmA, const CUtensorMap &tmB, const RaggedParams &p,
                              const LaunchCfg &cfg)
{
    return launch(tmA, tmB, p, cfg.grid, cfg.stream, nullptr);
}

}  // namespace w8a8
