// Grouped W8A8 block-FP8 matmul over ragged groups on sm_103a: the rows of A
// lie expert after expert, each expert's in offsets[e] .. offsets[e+1]-1, with
// no padding between them.
//
//   C[i,n] = cast( sum_g a_s[i,g] * b_s[e,n/128,g] * sum_{k in g} A[i,k] B[e,n,k] )
//
// The offsets are read on the device, after the dependency wait, so no host
// code waits for a routing.  One persistent CTA per SM turns them into a list
// of 128-row tiles in shared memory (a prefix sum of the experts' tile counts)
// and walks the (row tile, BN weight rows) items of it; an item finds its
// expert by binary search.  Tokens sit on the MMA's M side: where experts have
// many rows this is the tiled kernel's work.  Of a tile with fewer rows only the
// 32-row boxes of A that hold valid ones are loaded; the MMA still runs 128 rows
// (the others hold whatever the stage last held: a row of the product depends on
// its own row of A alone, and those rows are neither promoted nor stored).  The
// ring runs across items.  Where experts have a few rows only, k_ragged_few
// (gemm_ragged_few.cu) takes over.
// Bound by the promotion out of tensor memory, some 1130 cycles per 128 x 256 group
// against the MMA's 512, and by the padding of the experts' last tiles: 16384 rows
// of 64 experts, 4096 x 4096 (a quarter of the tiles' rows padding), 328 us, 1.68
// PFLOP/s, as captured calls (324 to 334 by the clock that the power cap leaves; 370
// called in a loop); 128-column tiles take 404.  1013 rows of 16 experts, 520 x 1088:
// 7.4 us, the latency of launch, offsets and nine groups in series.
//
// Roles per CTA, promotion and scale ring are those of the tiled kernel (see
// gemm_tiled.cu): warp 0 TMA producer, warps 1 and 3 MMA issuers, warp 2 scale
// loader, warps 4.. promotion and epilogue.
#include "epilogue.cuh"
#include "kernels.cuh"
#include "promote.cuh"
#include "ptx.cuh"
#include "ragged.cuh"

namespace w8a8 {

namespace {

constexpr int kScaleSlots = 8;
constexpr int kSlotFloats = 144;   // 128 a_s values + up to 2 b_s values, padded
constexpr int kBoxRows = 32;       // rows of A per TMA box

template <int BN, int STAGES, int CPW, int EB> struct RaggedLayout {
    static constexpr int kPromoWG = BN / CPW;
    static constexpr int kPairs = CPW / 2;
    static constexpr int kThreads = 128 + 128 * kPromoWG;
    static constexpr uint32_t kABytes = 128u * 128u;
    static constexpr uint32_t kBBytes = static_cast<uint32_t>(BN) * 128u;
    static constexpr int kBufs = 512 / BN;
    static constexpr uint32_t kTmemCols = 512;
    // Issuer threads and register split: as for the tiled kernel's layouts.
    static constexpr uint32_t kIssuers = (BN == 128 && STAGES % 2 == 0) ? 2u : 1u;
    static constexpr size_t kStageBytes = STAGES * (kABytes + kBBytes);
    static constexpr size_t kEpiBytes = 4 * kPromoWG * 2048 * EB;
    static constexpr int kRegsLow = BN == 128 ? 72 : 56;
    static constexpr int kRegsHigh = BN == 128 ? 200 : 224;
    static_assert(kThreads == 384 && 128 * kRegsLow + 256 * kRegsHigh <= 384 * 168,
                  "register split exceeds the launch's registers");
    static constexpr size_t kScaleBytes = kScaleSlots * kSlotFloats * 4;
    static constexpr int kBars = 2 * STAGES + 2 * kBufs + 2 * kScaleSlots + 2;
    // tile list: the experts' first rows and first tiles, one past the last each
    static constexpr size_t kListBytes = 2 * (kRaggedMaxExperts + 1) * 4;
    static constexpr size_t kSmem =
        1024 + kStageBytes + kEpiBytes + kScaleBytes + kBars * 8 + 16 + 64 + kListBytes;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int BN, int STAGES, int CPW, int EB>
__global__ void __launch_bounds__(RaggedLayout<BN, STAGES, CPW, EB>::kThreads, 1)
    k_ragged(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmTile,
             const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmC,
             const RaggedParams p)
{
    using L = RaggedLayout<BN, STAGES, CPW, EB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sA = smem_addr(smem);
    const uint32_t sB = sA + STAGES * L::kABytes;
    const uint32_t sEpi = sA + static_cast<uint32_t>(L::kStageBytes);
    float *scales = reinterpret_cast<float *>(smem + L::kStageBytes + L::kEpiBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kStageBytes + L::kEpiBytes +
                                                  L::kScaleBytes);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + L::kBufs + b); };
    auto sfull_bar = [&](int q) { return bar0 + 8u * (2 * STAGES + 2 * L::kBufs + q); };
    auto sempty_bar = [&](int q) {
        return bar0 + 8u * (2 * STAGES + 2 * L::kBufs + kScaleSlots + q);
    };
    auto drain_bar = [&](int w) {
        return bar0 + 8u * (2 * STAGES + 2 * L::kBufs + 2 * kScaleSlots + w);
    };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *warp_part = reinterpret_cast<volatile int *>(tmem_slot + 4);    // 16 words
    int *row0 = reinterpret_cast<int *>(tmem_slot + 20);
    int *tile0 = row0 + kRaggedMaxExperts + 1;

    const uint32_t warp = warp_index(), lane = lane_index();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < L::kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4 * L::kPromoWG);
        }
        for (int q = 0; q < kScaleSlots; ++q) {
            mbar_init(sfull_bar(q), 32);
            mbar_init(sempty_bar(q), 4 * L::kPromoWG);
        }
        mbar_init(drain_bar(0), 1);
        mbar_init(drain_bar(1), 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmTile);
        tma_prefetch_map(&tmB);
        tma_prefetch_map(&tmC);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const WaitGuard guard{abort_flag, p.status, p.wait_limit};

    grid_launch_dependents();
    grid_dependency_wait();

    make_tile_list<L::kThreads, 128>(p, row0, tile0, warp_part);

    if (warp < 4) {
        regs_dealloc<L::kRegsLow>();
        if (warp == 0) {
            // ---------------------------------------------------------- TMA producer
            // The whole warp walks the stages and an elected lane issues.
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            RaggedWalk<128> w(p, row0, tile0, static_cast<int>(blockIdx.x));
            while (ok && w.next(static_cast<int>(gridDim.x))) {
                // All 128 rows at once, or the boxes of 32 that hold valid ones (an
                // issue takes the producer some hundred cycles: with four boxes for
                // a whole tile, 128-column tiles took 476 us instead of 412 for
                // 16384 rows of 64 experts, N = K = 4096).
                const bool whole = w.rows > 128 - kBoxRows;
                const CUtensorMap *const map_a = whole ? &tmTile : &tmA;
                const int loads = whole ? 1 : (w.rows + kBoxRows - 1) / kBoxRows;
                const uint32_t a_bytes = (whole ? 128 : loads * kBoxRows) * 128u;
                for (int g = 0; g < p.G; ++g) {
                    ok = __all_sync(0xffffffffu, wait_bounded(empty_bar(stage), phase ^ 1u, guard,
                                                              SITE_TILED_PRODUCER));
                    if (!ok)
                        break;
                    const int arow = w.m0 + ((W8A8_DEBUG_BOUNDS && issued == 0 &&
                                              p.debug_skip_tma == kDebugBadFirstLoad)
                                                 ? (1 << 28)
                                                 : 0);
                    const bool in = in_bounds(arow >= 0 && arow < p.M && g * 128 < p.K, p.status,
                                              SITE_BOUNDS_A) &&
                                    in_bounds(w.nb * BN < p.N && w.e < p.experts, p.status,
                                              SITE_BOUNDS_B);
                    if (issued != p.debug_skip_tma && in && elect_one()) {
                        mbar_arrive_expect_tx(full_bar(stage), a_bytes + L::kBBytes);
                        tma_load_3d(sB + stage * L::kBBytes, &tmB, full_bar(stage), g * 128,
                                    w.nb * BN, w.e);
                        for (int b = 0; b < loads; ++b)
                            tma_load_2d(sA + stage * L::kABytes + b * kBoxRows * 128u, map_a,
                                        full_bar(stage), g * 128, arow + b * kBoxRows);
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            const int next_stage = stage;
            const uint32_t next_phase = phase;
            if (ok) {
                // Tail: wait until the MMA has released every stage, so that no
                // commit arrives on this CTA's shared memory after it exits.
                for (int s = 0; s < STAGES && ok; ++s) {
                    ok = wait_bounded(empty_bar(stage), phase ^ 1u, guard, SITE_TILED_PRODUCER);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // Drain: the loads still landing (the last issue into each stage).
                for (int s = 0; s < STAGES; ++s) {
                    const bool this_round = s < next_stage;
                    if (!this_round && issued < STAGES && s >= issued)
                        continue;
                    wait_drain(full_bar(s), this_round ? next_phase : (next_phase ^ 1u), p.status,
                               p.wait_limit, (SITE_DRAIN << 8) | 4u);
                }
            }
        } else if ((warp == 1 || (warp == 3 && L::kIssuers == 2)) && lane == 0) {
            // ---------------------------------------------------------- MMA issuers
            const uint32_t me = warp == 1 ? 0u : 1u;
            constexpr uint32_t idesc = idesc_e4m3_f32(128, BN);
            int stage = 0;
            uint32_t phase = 0;
            uint32_t it = 0;
            bool ok = true;
            const int items = tile0[p.experts] * p.num_n_tiles;
            for (int item = static_cast<int>(blockIdx.x); ok && item < items;
                 item += static_cast<int>(gridDim.x)) {
                for (int g = 0; g < p.G; ++g) {
                    if (it % L::kIssuers == me) {
                        const uint32_t buf = it % L::kBufs;
                        const uint32_t bphase = (it / L::kBufs) & 1u;
                        if (!wait_bounded(tempty_bar(buf), bphase ^ 1u, guard,
                                          SITE_TILED_MMA_TMEM) ||
                            !wait_bounded(full_bar(stage), phase, guard, SITE_TILED_MMA_FULL)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t d = tmem_base + buf * BN;
                        const uint64_t ad = sw128_kmajor_desc(sA + stage * L::kABytes);
                        const uint64_t bd = sw128_kmajor_desc(sB + stage * L::kBBytes);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_e4m3(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                        mma_commit(empty_bar(stage));
                        mma_commit(tfull_bar(buf));
                    }
                    ++it;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok || *abort_flag) {
                // an aborting CTA frees its tensor memory only after both
                // issuers' MMAs have completed
                mma_commit(drain_bar(me));
                wait_drain(drain_bar(me), 0, p.status, p.wait_limit, (SITE_DRAIN << 8) | 4u);
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------- scale loader
            int slot = 0;
            uint32_t sphase = 0;
            bool ok = true;
            RaggedWalk<128> w(p, row0, tile0, static_cast<int>(blockIdx.x));
            while (ok && w.next(static_cast<int>(gridDim.x))) {
                const size_t b_row0 = static_cast<size_t>(w.e) * p.NB;
                for (int g = 0; g < p.G; ++g) {
                    ok = __all_sync(0xffffffffu, wait_bounded(sempty_bar(slot), sphase ^ 1u, guard,
                                                              SITE_TILED_SCALES));
                    if (!ok)
                        break;
                    const uint32_t dst = smem_addr(scales + slot * kSlotFloats);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = static_cast<int>(lane) + 32 * i;
                        if (r < w.rows)
                            cp_async_4(dst + 4u * r,
                                       p.a_s + static_cast<size_t>(w.m0 + r) * p.G + g, 4u);
                    }
                    if (lane < static_cast<uint32_t>(L::kPromoWG)) {
                        const int col0 = w.nb * BN + static_cast<int>(lane) * CPW;
                        const bool in = col0 < p.N;
                        cp_async_4(dst + 4u * (128 + lane),
                                   p.b_s + (b_row0 + (in ? col0 / 128 : 0)) * p.G + g,
                                   in ? 4u : 0u);
                    }
                    cp_async_arrive(sfull_bar(slot));
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            // Let every gather land before the CTA can exit.
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // -------------------------------------------------------------- promotion + epilogue
        regs_alloc<L::kRegsHigh>();
        const int h = static_cast<int>(warp / 4) - 1;
        const uint32_t q = warp & 3u;
        const int row = static_cast<int>(q * 32 + lane);
        const uint32_t epi_buf = sEpi + (warp - 4u) * 2048u * EB;
        const bool fp32 = p.out_kind == OUT_FP32, bf = p.out_kind == OUT_BF16;
        uint32_t it = 0;
        int slot = 0;
        uint32_t sphase = 0;
        RaggedWalk<128> w(p, row0, tile0, static_cast<int>(blockIdx.x));
        while (w.next(static_cast<int>(gridDim.x))) {
            const int col0 = w.nb * BN + h * CPW;
            const int mine = min(32, w.rows - static_cast<int>(q * 32));   // rows of this warp
            const bool idle = mine <= 0 || col0 >= p.N;
            uint64_t acc[L::kPairs];
#pragma unroll
            for (int j = 0; j < L::kPairs; ++j)
                acc[j] = 0ull;
            bool ok = true;
            for (int g = 0; g < p.G; ++g) {
                const uint32_t buf = it % L::kBufs;
                const uint32_t bphase = (it / L::kBufs) & 1u;
                ok = __all_sync(0xffffffffu,
                                wait_bounded(sfull_bar(slot), sphase, guard, SITE_TILED_PROMOTE) &&
                                    wait_bounded(tfull_bar(buf), bphase, guard, SITE_TILED_PROMOTE));
                if (!ok)
                    break;
                const float *sl = scales + slot * kSlotFloats;
                const float s = sl[row] * sl[128 + h];
                const uint64_t s2 = pack2f(s, s);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sempty_bar(slot));
                if (++slot == kScaleSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                tc_fence_after_sync();
                const uint32_t taddr = tmem_base + ((q * 32u) << 16) + buf * BN + h * CPW;
                auto release = [&]() {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(tempty_bar(buf));
                };
                if (!idle)
                    promote_group<L::kPairs>(acc, taddr, s2, release);
                else
                    release();
                ++it;
            }
            if (!ok)
                break;
            const int y = w.m0 + static_cast<int>(q * 32);
            if (!idle && in_bounds(y >= 0 && y + mine <= p.M, p.status, SITE_BOUNDS_C)) {
                auto pack = [&](int k, int j) {
                    if (fp32) {
                        const uint64_t a = acc[8 * k + 2 * j], b = acc[8 * k + 2 * j + 1];
                        return make_uint4(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32),
                                          static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32));
                    }
                    const int b = (16 * k + 4 * j) % L::kPairs;
                    return make_uint4(pack_out2(acc[b], bf), pack_out2(acc[b + 1], bf),
                                      pack_out2(acc[b + 2], bf), pack_out2(acc[b + 3], bf));
                };
                // A warp with all of its 32 rows stores by TMA; the last rows of
                // an expert leave in 16-byte pieces, so that nothing is written
                // over the next expert's.
                store_warp_rows<CPW, EB>(pack, &tmC, epi_buf, lane, col0, y, p.N, fp32, mine == 32,
                                         true, mine, p.C, p.N);
            }
        }
        if (lane == 0)
            tma_store_wait_read();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

template <int BN, int STAGES, int CPW, int EB>
cudaError_t launch_ragged_t(const CUtensorMap &tmA, const CUtensorMap &tmTile,
                            const CUtensorMap &tmB, const CUtensorMap &tmC, const RaggedParams &p,
                            const LaunchCfg &cfg)
{
    using L = RaggedLayout<BN, STAGES, CPW, EB>;
    auto kernel = k_ragged<BN, STAGES, CPW, EB>;
    static volatile int smem_set[kMaxDeviceFlags] = {};
    cudaError_t e = ensure_smem_limit(kernel, smem_set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(cfg.grid, 1, 1);
    lc.blockDim = dim3(L::kThreads, 1, 1);
    lc.dynamicSmemBytes = L::kSmem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    // the kernel waits for the work before it ahead of its first access
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, tmA, tmTile, tmB, tmC, p);
}

}  // namespace

cudaError_t launch_ragged(const CUtensorMap &tmA, const CUtensorMap &tmTile, const CUtensorMap &tmB,
                          const CUtensorMap &tmC, const RaggedParams &p, int bn, const LaunchCfg &cfg)
{
    return bn == 256 ? launch_ragged_t<256, 4, 128, 1>(tmA, tmTile, tmB, tmC, p, cfg)
                     : launch_ragged_t<128, 6, 64, 1>(tmA, tmTile, tmB, tmC, p, cfg);
}

}  // namespace w8a8
