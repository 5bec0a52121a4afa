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
// expert by binary search.  Tokens sit on the MMA's M side at every size:
//  - where experts have many rows this is the tiled kernel's work;
//  - where they have a few (decode), the weights bound the time: an expert's
//    block is read once, and only the 32-row boxes of A that hold valid rows
//    are loaded.  The MMA still runs 128 rows (the others hold whatever the
//    stage last held: a row of the product depends on its own row of A alone,
//    and those rows are neither promoted nor stored), which costs nothing:
//    per 32 KB of weights the MMA takes about a fifth of the SM's share of the
//    HBM time.  The ring runs across items, so the stream of weights does not
//    pause between experts.
// Where even that leaves most SMs without an item (a few rows of a few experts),
// the CTAs of a cluster share one: each takes a range of its K groups, leaves its
// fp32 partial rows in shared memory, and they are added in rank order through
// distributed shared memory.
//
// Roles per CTA, promotion and scale ring are those of the tiled kernel (see
// gemm_tiled.cu): warp 0 TMA producer, warps 1 and 3 MMA issuers, warp 2 scale
// loader, warps 4.. promotion and epilogue.
#include "epilogue.cuh"
#include "kernels.cuh"
#include "promote.cuh"
#include "ptx.cuh"

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

// The items of one CTA: blockIdx.x, blockIdx.x + gridDim.x, ... over (row
// tile, column tile), column tiles innermost, so that the CTAs running at one
// time share row tiles of A and an expert's weights in L2.  SPLIT: the one item
// of this CTA's cluster, of which it takes the K groups g0 .. g1-1.
template <bool SPLIT> __device__ __forceinline__ int first_item(const RaggedParams &p)
{
    return static_cast<int>(SPLIT ? blockIdx.x / p.split : blockIdx.x);
}
template <bool SPLIT>
__device__ __forceinline__ void group_range(const RaggedParams &p, int &g0, int &g1)
{
    g0 = 0;
    g1 = p.G;
    if (SPLIT) {
        const int r = static_cast<int>(blockIdx.x % p.split);
        g0 = p.G * r / p.split;
        g1 = p.G * (r + 1) / p.split;
    }
}
template <bool SPLIT> struct RaggedWalk {
    const int *row0, *tile0;      // [experts + 1] first row and first tile of each expert
    int item, items, num_n, experts;
    int e, m0, rows, nb;          // the current item: expert, first row, valid rows, column tile
    __device__ RaggedWalk(const RaggedParams &p, const int *r, const int *t)
        : row0(r), tile0(t), item(first_item<SPLIT>(p)), items(t[p.experts] * p.num_n_tiles),
          num_n(p.num_n_tiles), experts(p.experts)
    {
    }
    __device__ bool next()
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
        m0 = row0[lo] + (mt - tile0[lo]) * 128;
        rows = min(128, row0[lo + 1] - m0);
        item = SPLIT ? items : item + static_cast<int>(gridDim.x);
        return true;
    }
};

// A partial tile in shared memory: rows of 128 floats, padded so that neighbouring
// rows start in different banks.
constexpr int kPartialPitch = 132;

template <int BN, int STAGES, int CPW, int EB, bool SPLIT>
__global__ void __launch_bounds__(RaggedLayout<BN, STAGES, CPW, EB>::kThreads, 1)
    k_ragged(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmTile,
             const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmC,
             const RaggedParams p)
{
    using L = RaggedLayout<BN, STAGES, CPW, EB>;
    static_assert(!SPLIT || (BN == 128 && 128 * kPartialPitch * 4 <= L::kStageBytes),
                  "the partial tile takes the stages' place");
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

    // The tile list.  Offsets that decrease or leave [0, M] are bent into a
    // non-decreasing sequence in [0, M] (a running maximum), so that nothing
    // below leaves a buffer whatever they hold.
    {
        constexpr int kPerThread = (kRaggedMaxExperts + 1 + L::kThreads - 1) / L::kThreads;
        const int first = static_cast<int>(threadIdx.x) * kPerThread;
        auto max_op = [](int a, int b) { return max(a, b); };
        auto add_op = [](int a, int b) { return a + b; };
        int o[kPerThread], top = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            o[i] = first + i <= p.experts ? min(max(__ldg(p.offsets + first + i), 0), p.M) : 0;
            top = max(top, o[i]);
        }
        int run = block_prefix<L::kThreads>(top, 0, warp_part, max_op);
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
            tiles[i] = e < p.experts ? (row0[e + 1] - row0[e] + 127) / 128 : 0;
            sum += tiles[i];
        }
        int at = block_prefix<L::kThreads>(sum, 0, warp_part, add_op);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (first + i <= p.experts)
                tile0[first + i] = at;
            at += tiles[i];
        }
        __syncthreads();
    }

    int g0, g1;
    group_range<SPLIT>(p, g0, g1);

    if (warp < 4) {
        regs_dealloc<L::kRegsLow>();
        if (warp == 0) {
            // ---------------------------------------------------------- TMA producer
            // The whole warp walks the stages and an elected lane issues.
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            RaggedWalk<SPLIT> w(p, row0, tile0);
            while (ok && w.next()) {
                // All 128 rows at once, or the boxes of 32 that hold valid ones (an
                // issue takes the producer some hundred cycles: with four boxes for
                // a whole tile, 128-column tiles took 476 us instead of 412 for
                // 16384 rows of 64 experts, N = K = 4096).
                const bool whole = w.rows > 128 - kBoxRows;
                const CUtensorMap *const map_a = whole ? &tmTile : &tmA;
                const int loads = whole ? 1 : (w.rows + kBoxRows - 1) / kBoxRows;
                const uint32_t a_bytes = (whole ? 128 : loads * kBoxRows) * 128u;
                for (int g = g0; g < g1; ++g) {
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
            for (int item = first_item<SPLIT>(p); ok && item < items;
                 item = SPLIT ? items : item + static_cast<int>(gridDim.x)) {
                for (int g = g0; g < g1; ++g) {
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
            RaggedWalk<SPLIT> w(p, row0, tile0);
            while (ok && w.next()) {
                const size_t b_row0 = static_cast<size_t>(w.e) * p.NB;
                for (int g = g0; g < g1; ++g) {
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
        __syncwarp();
        if (SPLIT) {
            cluster_sync();       // the partial rows are in shared memory
            cluster_sync();       // and have been read
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
        RaggedWalk<SPLIT> w(p, row0, tile0);
        while (w.next()) {
            const int col0 = w.nb * BN + h * CPW;
            const int mine = min(32, w.rows - static_cast<int>(q * 32));   // rows of this warp
            const bool idle = mine <= 0 || col0 >= p.N;
            uint64_t acc[L::kPairs];
#pragma unroll
            for (int j = 0; j < L::kPairs; ++j)
                acc[j] = 0ull;
            bool ok = true;
            for (int g = g0; g < g1; ++g) {
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
            if (SPLIT) {
                // Every group's MMA has completed (its partial was read), so the
                // stages are free.
                float4 *part = reinterpret_cast<float4 *>(smem) + row * (kPartialPitch / 4) + h * (CPW / 4);
#pragma unroll
                for (int j = 0; j < CPW / 4; ++j) {
                    float4 v;
                    unpack2f(acc[2 * j], v.x, v.y);
                    unpack2f(acc[2 * j + 1], v.z, v.w);
                    if (!idle)
                        part[j] = v;
                }
            } else if (!idle && in_bounds(y >= 0 && y + mine <= p.M, p.status, SITE_BOUNDS_C)) {
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
        if (SPLIT) {
            cluster_sync();
            // Each CTA finishes its share of the tile's rows: 32 threads to a row,
            // four columns each.
            RaggedWalk<SPLIT> last(p, row0, tile0);
            const int S = p.split, rank = static_cast<int>(blockIdx.x % p.split);
            if (last.next()) {
                const int n = last.nb * BN + 4 * static_cast<int>(lane);
                const uint32_t at = smem_addr(smem) + 16u * lane;
                const int r1 = last.rows * (rank + 1) / S;
                for (int r = last.rows * rank / S + static_cast<int>(warp) - 4; r < r1 && n < p.N; r += 8) {
                    float4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)          // every load before the first addition
                        if (i < S)
                            v[i] = ld_cluster_f4(cluster_map(at + 4u * kPartialPitch * r,
                                                             static_cast<uint32_t>(i)));
#pragma unroll
                    for (int i = 1; i < 8; ++i)
                        if (i < S) {
                            v[0].x += v[i].x;
                            v[0].y += v[i].y;
                            v[0].z += v[i].z;
                            v[0].w += v[i].w;
                        }
                    const size_t to = static_cast<size_t>(last.m0 + r) * p.N + n;
                    if (!in_bounds(last.m0 + r < p.M && n + 4 <= p.N, p.status, SITE_BOUNDS_C))
                        continue;
                    if (fp32)
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + to) = v[0];
                    else
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + to) =
                            bf ? make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[0].z, v[0].w))
                               : make_uint2(pack_f16x2(v[0].x, v[0].y), pack_f16x2(v[0].z, v[0].w));
                }
            }
            cluster_sync();
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

template <int BN, int STAGES, int CPW, int EB, bool SPLIT>
cudaError_t launch_ragged_t(const CUtensorMap &tmA, const CUtensorMap &tmTile,
                            const CUtensorMap &tmB, const CUtensorMap &tmC, const RaggedParams &p,
                            const LaunchCfg &cfg, int *clusters = nullptr)
{
    using L = RaggedLayout<BN, STAGES, CPW, EB>;
    auto kernel = k_ragged<BN, STAGES, CPW, EB, SPLIT>;
    static volatile int smem_set[kMaxDeviceFlags] = {};
    cudaError_t e = ensure_smem_limit(kernel, smem_set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(clusters ? p.split : cfg.grid, 1, 1);
    lc.blockDim = dim3(L::kThreads, 1, 1);
    lc.dynamicSmemBytes = L::kSmem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[2];
    // the kernel waits for the work before it ahead of its first access
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = clusters ? 0 : 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(SPLIT ? p.split : 1);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = SPLIT ? 2 : 1;
    if (clusters)
        return cudaOccupancyMaxActiveClusters(clusters, kernel, &lc);
    return cudaLaunchKernelEx(&lc, kernel, tmA, tmTile, tmB, tmC, p);
}

}  // namespace

int ragged_clusters(int split)
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
    if (launch_ragged_t<128, 6, 64, 1, true>(none, none, none, none, p, LaunchCfg{}, &n) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cached[dev][split] = n;
    return n;
}

cudaError_t launch_ragged(const CUtensorMap &tmA, const CUtensorMap &tmTile, const CUtensorMap &tmB,
                          const CUtensorMap &tmC, const RaggedParams &p, int bn, const LaunchCfg &cfg)
{
    if (p.split > 1)
        return launch_ragged_t<128, 6, 64, 1, true>(tmA, tmTile, tmB, tmC, p, cfg);
    return bn == 256 ? launch_ragged_t<256, 4, 128, 1, false>(tmA, tmTile, tmB, tmC, p, cfg)
                     : launch_ragged_t<128, 6, 64, 1, false>(tmA, tmTile, tmB, tmC, p, cfg);
}

}  // namespace w8a8
