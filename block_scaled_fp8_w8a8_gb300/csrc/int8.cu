// INT8 matmul with one scale per token and per output channel on sm_103a:
//
//   C[m,n] = cast( a_s[m] * b_s[n] * sum_k A[m,k] B[n,k] )
//
// The sum is over whole numbers and exact (32 bits); it is converted to fp32
// once and multiplied by the two scales in fp32.
//
// This part's INT8 tensor rate is a small fraction of its fp16 rate, and the
// tcgen05 kinds of sm_103a have no INT8 form.  But every INT8 value is an fp16
// value, a product of two is at most 2^14, and a sum of up to 512 of them stays
// within 2^23, which the MMA's fp32 accumulator holds without rounding.  So the
// operands are widened to fp16, multiplied with tcgen05.mma kind::f16, and
// every 512 columns of K the accumulator is added to 32-bit integer registers:
// the INT8 product at the fp16 tensor rate, to the bit.
//
// Three forms, by how often a widened value is used:
//  - up to 32 tokens, k_int8_small widens in registers right after the load;
//  - some hundred tokens, k_int8_mid widens on the way to shared memory;
//  - beyond, k_int8_widen writes both operands as fp16 into the workspace (rows
//    padded with zeros to whole 128-column stages, so that any size, stride and
//    alignment of the INT8 operands is as good as another) and k_int8_mma
//    multiplies them.
#include <algorithm>

#include "epilogue.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

// An accumulator takes the products of 512 columns: this many steps of 64 (one
// 128-byte fp16 row each), or stages of 128.
constexpr int kChunkSteps = 8;
constexpr int kChunkStages = 4;

// ------------------------------------------------------------------ widening

// Four INT8 values of a word as fp16 pairs, exactly: byte b (offset by 128) in
// the low mantissa bits of 1024 is 1024 + b + 128; the constant goes off again.
__device__ __forceinline__ uint2 widen4(uint32_t w)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&hi), off);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// 16 INT8 values at columns c .. c+15 of a row (zeros past K).  ACCESS: bytes
// per load (16, 8 or 4 where the operands' addresses, strides and K are
// multiples of it, so that no load straddles the row's end; else 1).
template <int ACCESS>
__device__ __forceinline__ uint4 load16(const uint8_t *row, int c, int K)
{
    if constexpr (ACCESS == 16)
        return c < K ? __ldg(reinterpret_cast<const uint4 *>(row + c)) : make_uint4(0, 0, 0, 0);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = c + 4 * i;
        if constexpr (ACCESS == 8) {
            if (i & 1)
                continue;
            const uint2 v = k < K ? __ldg(reinterpret_cast<const uint2 *>(row + k)) : make_uint2(0, 0);
            w[i] = v.x;
            w[i + 1] = v.y;
        } else if constexpr (ACCESS == 4) {
            w[i] = k < K ? __ldg(reinterpret_cast<const uint32_t *>(row + k)) : 0u;
        } else {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j < K)
                    w[i] |= static_cast<uint32_t>(__ldg(row + k + j)) << (8 * j);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kWidenThreads = 256;
constexpr int kWidenUnroll = 4;

// rows x Kp fp16 from INT8 rows: units of 16 columns, dealt round robin to the
// grid's threads, kWidenUnroll loads of a thread in flight.
template <int ACCESS>
__device__ __forceinline__ void widen_rows(const uint8_t *src, long long ld, uint8_t *dst,
                                           long long rows, int K, int Kp, unsigned *status)
{
    const unsigned per_row = static_cast<unsigned>(Kp) / 16;
    const unsigned stride = gridDim.x * kWidenThreads;       // units; a row is at most 2^13 of them
    const unsigned step_r = stride / per_row, step_c = stride - step_r * per_row;
    const unsigned at = blockIdx.x * kWidenThreads + threadIdx.x;
    long long r = at / per_row;
    unsigned c = at % per_row;
    while (r < rows) {
        uint4 w[kWidenUnroll];
        uint8_t *to[kWidenUnroll];
#pragma unroll
        for (int i = 0; i < kWidenUnroll; ++i) {
            to[i] = nullptr;
            if (r < rows && in_bounds(c < per_row, status, SITE_BOUNDS_WORKSPACE)) {
                w[i] = load16<ACCESS>(src + r * ld, static_cast<int>(16 * c), K);
                to[i] = dst + (r * Kp + 16 * c) * 2;
            }
            r += step_r;
            c += step_c;
            if (c >= per_row) {
                c -= per_row;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kWidenUnroll; ++i) {
            if (!to[i])
                continue;
            const uint2 h0 = widen4(w[i].x), h1 = widen4(w[i].y), h2 = widen4(w[i].z),
                        h3 = widen4(w[i].w);
            const uint32_t out[8] = {h0.x, h0.y, h1.x, h1.y, h2.x, h2.y, h3.x, h3.y};
            st_global_v8(to[i], out);            // 32 bytes on a 32-byte boundary
        }
    }
}

// Both operands in one launch.  HBM- and L2-bound: of 16384 x 4096 and 4096 x 4096 it
// reads 84 MB and writes 168 in about 36 us (7 TB/s).
template <int ACCESS>
__global__ void __launch_bounds__(kWidenThreads) k_int8_widen(const Int8WidenParams p)
{
    grid_launch_dependents();
    grid_dependency_wait();
    widen_rows<ACCESS>(p.A, p.lda, p.A16, p.rows_a, p.K, p.Kp, p.status);
    widen_rows<ACCESS>(p.B, p.ldb, p.B16, p.rows_b, p.K, p.Kp, p.status);
}

// ------------------------------------------------------------------ few tokens

// Up to 32 tokens: the weights' bytes bound the time, and each is widened in
// registers right after its load (writing them as fp16 first would triple
// their traffic).  A warp multiplies 16 MT weight rows (the MMA's M side) with 8
// NT tokens on mma.sync fp16 tiles, whose operands a thread builds from plain
// 16-byte loads: the MMA sums over k in any order, so thread t of a quad takes
// bytes 16 t .. 16 t + 15 of every 64-byte run, for weights and tokens alike,
// and word j of them is its share of the run's j-th MMA.  (tcgen05 would want
// both operands in shared memory: at the HBM rate the widened weights' way
// through it takes more than its bandwidth.)
// The warps of a CTA, and the CTAs of a cluster, split K; whole sums meet in
// shared memory, where the order of integer additions does not matter.
// Bound by the latency of a launch and of the loads: two batches of loads a
// thread, 32 KB a CTA, stay in flight.  One token by 4096 x 4096: 4.05 us (4.1
// TB/s; at the lower clock that a long prefill leaves behind it 4.65; with a single
// batch 5.4), by 8192 x 16384: 28.0 us (4.8 TB/s).
// Batches of 4 steps gave 4.6 and 26.4 us where these took 4.25 and 28.7.  (The form of
// 17 to 32 tokens spills some 50 bytes at the 128 registers of two CTAs per SM, and with
// narrower loads 24 to 172.)
constexpr int kSmallWarps = 8, kSmallCtas = 2;       // CTAs per SM

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int j)
{
    return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// UN: 64-column steps whose loads are issued together; two such batches are held.
template <int NT, int MT, int UN, int ACCESS>
__global__ void __launch_bounds__(32 * kSmallWarps, kSmallCtas) k_int8_small(const Int8SmallParams p)
{
    constexpr int kRows = 16 * MT, kTokens = 8 * NT;
    // [token][row], of two tiles in turn; with 4 words of padding a warp's
    // additions fall into different banks
    constexpr int kPitch = kRows + 4, kSums = kPitch * kTokens;
    __shared__ int sums2[2][kSums];
    __shared__ float tok_s[kTokens], row_s[2][kRows];    // scales, fetched while the sums form
    const int lane = static_cast<int>(lane_index()), warp = static_cast<int>(warp_index());
    const int g = lane >> 2, t = lane & 3;
    for (int i = static_cast<int>(threadIdx.x); i < 2 * kSums; i += 32 * kSmallWarps)
        sums2[0][i] = 0;
    __syncthreads();
    grid_launch_dependents();
    grid_dependency_wait();

    const int m0 = static_cast<int>(blockIdx.z) * kTokens, tid = static_cast<int>(threadIdx.x);
    if (tid < kTokens)
        cp_async_4(smem_addr(tok_s + tid), p.a_s + min(m0 + tid, p.M - 1), 4u);
    // This warp's steps: the cluster's CTAs and their warps take equal shares.
    const int steps = (p.K + 63) / 64, shares = static_cast<int>(gridDim.y) * kSmallWarps;
    const int share = static_cast<int>(blockIdx.y) * kSmallWarps + warp;
    const int first = static_cast<int>(static_cast<long long>(steps) * share / shares);
    const int last = static_cast<int>(static_cast<long long>(steps) * (share + 1) / shares);
    // Rows past the ends repeat the last one; their sums are not stored.
    const uint8_t *wrow[2 * MT], *xrow[NT];
    auto rows_from = [&](int n0) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            wrow[i] = p.B + static_cast<long long>(min(n0 + 8 * i + g, p.N - 1)) * p.ldb;
    };
#pragma unroll
    for (int i = 0; i < NT; ++i)
        xrow[i] = p.A + static_cast<long long>(min(m0 + 8 * i + g, p.M - 1)) * p.lda;

    float acc[MT][NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[i][j][k] = 0.f;
    };
    // An accumulator's element: weight row g (+ 8), tokens 2 t and 2 t + 1.
    auto flush = [&](int *sums) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    atomicAdd(sums + (8 * j + 2 * t + (k & 1)) * kPitch + 16 * i + g + 8 * (k >> 1),
                              __float2int_rn(acc[i][j][k]));
    };
    struct Batch {
        uint4 w[UN][2 * MT], x[UN][NT];
    };
    auto load = [&](Batch &q, int s) {
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int c = (s + u) * 64 + 16 * t;
            const int end = s + u < last ? p.K : 0;          // nothing past this warp's steps
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                q.w[u][i] = load16<ACCESS>(wrow[i], c, end);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                q.x[u][i] = load16<ACCESS>(xrow[i], c, end);
        }
    };
    int since = 0;                                   // steps in the accumulators: at most 8
    auto multiply = [&](const Batch &q, int *sums) {
        if (since + UN > kChunkSteps) {
            flush(sums);
            clear();
            since = 0;
        }
        since += UN;
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[MT][4];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint2 lo = widen4(word_of(q.w[u][2 * i], j));
                    const uint2 hi = widen4(word_of(q.w[u][2 * i + 1], j));
                    a[i][0] = lo.x;
                    a[i][1] = hi.x;
                    a[i][2] = lo.y;
                    a[i][3] = hi.y;
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint2 b = widen4(word_of(q.x[u][i], j));
#pragma unroll
                    for (int k = 0; k < MT; ++k)
                        mma_16x8x16(acc[k][i], a[k], b.x, b.y);
                }
            }
    };
    // The CTA's tiles.  Two batches in turn: one's loads are in flight while the
    // other is multiplied, and the next tile's first while a tile is finished.
    const int S = static_cast<int>(gridDim.y);
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0;
    const int step_n = static_cast<int>(gridDim.x) * kRows;
    Batch q0, q1;
    int n0 = static_cast<int>(blockIdx.x) * kRows, turn = 0;
    rows_from(n0);
    load(q0, first);
    for (;; turn ^= 1) {
        int *sums = sums2[turn];
        const bool next = step_n < p.N - n0;         // this CTA has another tile
        if (tid < kRows)
            cp_async_4(smem_addr(row_s[turn] + tid), p.b_s + min(n0 + tid, p.N - 1), 4u);
        clear();
        since = 0;
        for (int s = first;; s += 2 * UN) {
            load(q1, s + UN);
            multiply(q0, sums);
            const bool half = s + UN < last, more = s + 2 * UN < last;
            if (!more && next)
                rows_from(n0 + step_n);
            if (more || next)
                load(q0, more ? s + 2 * UN : first);
            if (half)
                multiply(q1, sums);
            if (!more)
                break;
        }
        flush(sums);
        cp_async_wait_all();
        // The CTAs of a cluster hold partial sums of the same tile: each finishes
        // its share of it, reading the others' through distributed shared memory.
        if (S > 1)
            cluster_sync();
        else
            __syncthreads();
        constexpr int kAll = kRows * kTokens;
        const int hi = kAll * (static_cast<int>(rank) + 1) / S;
        for (int i = kAll * static_cast<int>(rank) / S + static_cast<int>(threadIdx.x); i < hi;
             i += 32 * kSmallWarps) {
            const int m = m0 + i / kRows, n = n0 + i % kRows;
            int *const at_sum = sums + i / kRows * kPitch + i % kRows;
            int sum = 0;
            if (S == 1) {
                sum = *at_sum;
                *at_sum = 0;         // for the tile after the next, a barrier away
            } else {
                for (int r = 0; r < S; ++r) {
                    int v;
                    asm volatile("ld.shared::cluster.s32 %0, [%1];"
                                 : "=r"(v)
                                 : "r"(cluster_map(smem_addr(at_sum), static_cast<uint32_t>(r)))
                                 : "memory");
                    sum += v;
                }
            }
            if (m >= p.M || n >= p.N)
                continue;
            const float v = __int2float_rn(sum) * tok_s[i / kRows] * row_s[turn][i % kRows];
            if (!in_bounds(m >= 0 && n >= 0, p.status, SITE_BOUNDS_C))
                continue;
            const long long at = m * p.ldc + n;
            if (p.out_kind == OUT_FP32)
                static_cast<float *>(p.C)[at] = v;
            else if (p.out_kind == OUT_BF16)
                static_cast<__nv_bfloat16 *>(p.C)[at] = __float2bfloat16_rn(v);
            else
                static_cast<__half *>(p.C)[at] = __float2half_rn(v);
        }
        if (!next)
            break;
        n0 += step_n;
    }
    if (S > 1)
        cluster_sync();              // no CTA leaves while another reads its sums
}

template <int NT, int MT, int UN>
cudaError_t launch_small_t(const Int8SmallParams &p, int access, int sm_count, cudaStream_t stream)
{
    auto kernel = access == 16  ? k_int8_small<NT, MT, UN, 16>
                  : access == 8 ? k_int8_small<NT, MT, UN, 8>
                  : access == 4 ? k_int8_small<NT, MT, UN, 4>
                                : k_int8_small<NT, MT, UN, 1>;
    const int tiles_n = (p.N + 16 * MT - 1) / (16 * MT), tiles_m = (p.M + 8 * NT - 1) / (8 * NT);
    // Split K over a cluster while that keeps the GPU within about two CTAs per
    // SM and leaves every warp a step.
    const long long tiles = static_cast<long long>(tiles_n) * tiles_m;
    const int steps = (p.K + 63) / 64;
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= static_cast<long long>(kSmallCtas) * sm_count &&
           steps >= 2 * splits * kSmallWarps)
        splits *= 2;
    // Without a split a CTA takes several tiles where there are more than stay
    // resident; a split has one tile a cluster.
    const int resident = (kSmallCtas * sm_count + tiles_m - 1) / tiles_m;
    const int each = (tiles_n + resident - 1) / resident;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(splits > 1 ? tiles_n : (tiles_n + each - 1) / each, splits, tiles_m);
    lc.blockDim = dim3(32 * kSmallWarps, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

// ------------------------------------------------------------------ some hundred tokens

// Between those and the sizes that repay widening in a launch of its own: the
// operands are widened on their way to shared memory.  One CTA owns 128 weight
// rows (the MMA's M side), up to 256 tokens (its N side) and a share of K; its
// eight warps load INT8 runs of 16 columns, several steps ahead, widen them and
// store them in the 128-byte-swizzled layout that the MMA reads; a ninth
// issues the MMAs.  Each 512 columns of K go to a tensor memory buffer of their
// own, so nothing is promoted before the end: the buffers' whole numbers are
// added up then, and the cluster's CTAs, which split K, add theirs through
// distributed shared memory.
// Bound by shared memory: a step's 24 KB (of 128 + 64 rows) to 48 KB (128 + 256)
// are written once and read once by the MMA; where CTAs have few steps, by the
// latency of launch, first loads and the cluster's sum.  256 tokens by 4096 x
// 4096: 20.7 us (the widening launch and k_int8_mma: 24.7), 512: 41.0 (26.2); 257 by
// 1537 x 1000, rows off 16-byte boundaries: 8.6.
constexpr int kMidGroup = 8;
constexpr int kMidGroups = 2;
constexpr int kMidWarps = kMidGroup * kMidGroups;
constexpr int kMidStages = 4;
constexpr int kMidSmem = 1024 + kMidStages * (128 + 256) * 128;     // the most: 256 tokens

struct MidBars {
    uint64_t full[kMidStages], empty[kMidStages], done;
    uint32_t tmem;
    int abort_word;
};

// CH: 16-column runs per thread and step, (rows of both operands) / 64 rounded
// up; AHEAD: steps whose loads are in flight.
template <int CH, int AHEAD, int ACCESS>
__global__ void __launch_bounds__(32 * kMidWarps + 32, 1) k_int8_mid(const Int8MidParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ MidBars bars;
    const uint32_t sW = smem_addr(smem);
    const int Nt = p.tile_tokens;                      // a multiple of 16, at most 256
    const uint32_t w_bytes = 128u * 128u, stage_bytes = w_bytes + static_cast<uint32_t>(Nt) * 128u;
    const uint32_t full0 = smem_addr(bars.full), empty0 = smem_addr(bars.empty);
    const uint32_t done = smem_addr(&bars.done);
    volatile int *abort_flag = &bars.abort_word;
    const int tid = static_cast<int>(threadIdx.x);
    const uint32_t warp = warp_uniform(warp_index()), lane = lane_index();
    const int buf_cols = (Nt + 31) / 32 * 32;          // columns of a tensor memory buffer

    if (tid == 0) {
        for (int s = 0; s < kMidStages; ++s) {
            mbar_init(full0 + 8u * s, kMidGroup);
            mbar_init(empty0 + 8u * s, 1);
        }
        mbar_init(done, 1);
        bars.abort_word = 0;
        mbar_fence_init();
    }
    if (warp == kMidWarps) {
        tmem_alloc(smem_addr(&bars.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = warp_uniform(bars.tmem);
    const WaitGuard guard{abort_flag, p.status, p.wait_limit};
    grid_launch_dependents();
    grid_dependency_wait();

    const int n0 = static_cast<int>(blockIdx.x) * 128, m0 = static_cast<int>(blockIdx.z) * Nt;
    const int S = static_cast<int>(gridDim.y);
    const int all = (p.K + 63) / 64;
    const int first = static_cast<int>(static_cast<long long>(all) * blockIdx.y / S);
    const int steps = static_cast<int>(static_cast<long long>(all) * (blockIdx.y + 1) / S) - first;

    if (warp < kMidWarps) {
        // ------------------------------------------------------------ widening
        // Run i of the group's thread gt: row (gt + 256 i) / 4 of the stage (weights,
        // then tokens), 16 columns from 16 (gt % 4).  Rows past the ends repeat the
        // last one: their results are not stored.
        const int gt = tid % (32 * kMidGroup), group = tid / (32 * kMidGroup);
        const int c0 = 16 * (gt & 3);
        const uint8_t *src[CH];
        uint32_t dst[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int r = (gt + 256 * i) >> 2;
            src[i] = r < 128 ? p.B + static_cast<long long>(min(n0 + r, p.N - 1)) * p.ldb
                             : p.A + static_cast<long long>(min(m0 + r - 128, p.M - 1)) * p.lda;
            dst[i] = sW + static_cast<uint32_t>(r) * 128u;       // tokens follow the weights
        }
        const uint32_t sw = static_cast<uint32_t>((gt >> 2) & 7);       // row % 8, the same for all i
        const uint32_t p0 = 16u * ((2u * (gt & 3)) ^ sw), p1 = 16u * ((2u * (gt & 3) + 1u) ^ sw);
        const int runs = (4 * (128 + Nt) - gt + 255) / 256;             // of the CH, those that exist
        auto load = [&](uint4(&x)[CH], int s) {
            const int c = (first + s) * 64 + c0, end = s < steps ? p.K : 0;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                x[i] = load16<ACCESS>(src[i], c, i < runs ? end : 0);
        };
        auto put = [&](const uint4(&x)[CH], int s) {
            const int stage = s % kMidStages;
            const uint32_t parity = static_cast<uint32_t>(s / kMidStages) & 1u;
            if (!__all_sync(0xffffffffu, wait_bounded(empty0 + 8u * stage, parity ^ 1u, guard,
                                                      SITE_TILED_PRODUCER)))
                return false;
            const uint32_t off = static_cast<uint32_t>(stage) * stage_bytes;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if (i < runs) {
                    const uint2 a = widen4(x[i].x), b = widen4(x[i].y), c = widen4(x[i].z),
                                d = widen4(x[i].w);
                    st_shared_v4(dst[i] + off + p0, a.x, a.y, b.x, b.y);
                    st_shared_v4(dst[i] + off + p1, c.x, c.y, d.x, d.y);
                }
            }
            fence_async_smem();              // the codes are read by the tensor cores
            __syncwarp();
            if (lane == 0 && s != p.debug_skip)
                mbar_arrive(full0 + 8u * stage);
            return true;
        };
        uint4 x[AHEAD][CH];
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            load(x[d], group + kMidGroups * d);
        bool ok = true;
        for (int s = group; ok && s < steps; s += kMidGroups * AHEAD) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int at = s + kMidGroups * d;
                ok = ok && (at >= steps || put(x[d], at));
                load(x[d], at + kMidGroups * AHEAD);
            }
        }
    } else {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_f16_f32(128, static_cast<uint32_t>(Nt));
        bool ready = false;
        for (int s = 0; s < steps; ++s) {
            const int stage = s % kMidStages;
            if (!__all_sync(0xffffffffu,
                            ready || wait_bounded(full0 + 8u * stage,
                                                  static_cast<uint32_t>(s / kMidStages) & 1u, guard,
                                                  SITE_TILED_MMA_FULL)))
                break;
            // the next step's probe answers while this one's MMAs are issued
            ready = mbar_test_wait(full0 + 8u * ((s + 1) % kMidStages),
                                   static_cast<uint32_t>((s + 1) / kMidStages) & 1u);
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(s / kChunkSteps * buf_cols);
            const uint64_t ad = sw128_kmajor_desc(sW + stage * stage_bytes);
            const uint64_t bd = sw128_kmajor_desc(sW + stage * stage_bytes + w_bytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f16_elect<false>(d, ad + 2u * kk, bd + 2u * kk, idesc,
                                     (s % kChunkSteps > 0 || kk > 0) ? 1u : 0u);
            mma_commit_elect<false>(empty0 + 8u * stage);
        }
        mma_commit_elect<false>(done);
    }
    __syncwarp();
    // All MMAs have read shared memory and written tensor memory (after a
    // timeout too, whose garbage the status word reports).
    wait_drain(done, 0, p.status, p.wait_limit, (SITE_DRAIN << 8) | 4u);
    tc_fence_after_sync();
    __syncthreads();                   // every warp is past its stores into the stages

    // ---------------------------------------------------------------- the sums, [token][weight row]
    int *sums = reinterpret_cast<int *>(smem);
    const int bufs = (steps + kChunkSteps - 1) / kChunkSteps;
    if (warp < kMidWarps) {
        const uint32_t q = warp & 3u;
        const int row = static_cast<int>(q * 32 + lane);
        for (int c = 32 * static_cast<int>(warp >> 2); c < Nt; c += 8 * kMidWarps) {
            int sum[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                sum[j] = 0;
            for (int b = 0; b < bufs; ++b) {
                float v[32];
                tmem_load_32cols(tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(b * buf_cols + c), v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    sum[j] += __float2int_rn(v[j]);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j < Nt)
                    sums[(c + j) * 128 + row] = sum[j];
        }
    }
    uint32_t rank = 0;
    if (S > 1) {
        rank = cluster_ctarank();
        cluster_sync();
    } else {
        __syncthreads();
    }
    // Each CTA of the cluster finishes its share of the tokens: 32 threads to a
    // token's row, four columns each.
    const int tokens = min(Nt, p.M - m0);
    const int t0 = tokens * static_cast<int>(rank) / S, t1 = tokens * (static_cast<int>(rank) + 1) / S;
    const int n = n0 + 4 * static_cast<int>(lane);
    if (warp < kMidWarps && n < p.N) {
        float bs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bs[j] = n + j < p.N ? __ldg(p.b_s + n + j) : 0.f;
        uint32_t base[8];                       // the cluster's tiles
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t own = smem_addr(sums + 4 * static_cast<int>(lane));
            base[r] = S > 1 ? cluster_map(own, static_cast<uint32_t>(min(r, S - 1))) : own;
        }
        for (int tk = t0 + static_cast<int>(warp); tk < t1; tk += kMidWarps) {
            const int m = m0 + tk;
            const float as = __ldg(p.a_s + m);
            int v[8][4], s[4] = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < 8; ++r)         // every load before the first addition
                if (r < S)
                    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[r][0]), "=r"(v[r][1]), "=r"(v[r][2]), "=r"(v[r][3])
                                 : "r"(base[r] + 512u * tk)
                                 : "memory");
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < S) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[j] += v[r][j];
                }
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __int2float_rn(s[j]) * as * bs[j];
            if (!in_bounds(m < p.M && n < p.N, p.status, SITE_BOUNDS_C))
                continue;
            const long long o = static_cast<long long>(m) * p.ldc + n;
            if (p.out_kind == OUT_FP32) {
                float *c = static_cast<float *>(p.C) + o;
                if (p.wide && n + 4 <= p.N)
                    *reinterpret_cast<float4 *>(c) = make_float4(f[0], f[1], f[2], f[3]);
                else
                    for (int j = 0; j < 4 && n + j < p.N; ++j)
                        c[j] = f[j];
            } else {
                uint16_t *c = static_cast<uint16_t *>(p.C) + o;
                const bool bf = p.out_kind == OUT_BF16;
                const uint32_t lo = bf ? pack_bf16x2(f[0], f[1]) : pack_f16x2(f[0], f[1]);
                const uint32_t hi = bf ? pack_bf16x2(f[2], f[3]) : pack_f16x2(f[2], f[3]);
                if (p.wide && n + 4 <= p.N)
                    *reinterpret_cast<uint2 *>(c) = make_uint2(lo, hi);
                else
                    for (int j = 0; j < 4 && n + j < p.N; ++j)
                        c[j] = static_cast<uint16_t>((j < 2 ? lo : hi) >> (16 * (j & 1)));
            }
        }
    }
    tc_fence_before_sync();
    if (S > 1)
        cluster_sync();                // no CTA leaves while another reads its sums
    else
        __syncthreads();
    if (warp == kMidWarps) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, 512);
    }
}

template <int CH, int AHEAD>
cudaError_t launch_mid_t(const Int8MidParams &p, int access, int splits, cudaStream_t stream)
{
    auto kernel = access == 16  ? k_int8_mid<CH, AHEAD, 16>
                  : access == 8 ? k_int8_mid<CH, AHEAD, 8>
                  : access == 4 ? k_int8_mid<CH, AHEAD, 4>
                                : k_int8_mid<CH, AHEAD, 1>;
    const size_t smem = 1024 + kMidStages * (128 * 128 + static_cast<size_t>(p.tile_tokens) * 128);
    static volatile int smem_set[4][kMaxDeviceFlags] = {};
    const int a = access == 16 ? 0 : access == 8 ? 1 : access == 4 ? 2 : 3;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDeviceFlags))
        e = cudaErrorInvalidDevice;
    if (e == cudaSuccess && !smem_set[a][dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMidSmem);
        smem_set[a][dev] = e == cudaSuccess;
    }
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((p.N + 127) / 128, splits, (p.M + p.tile_tokens - 1) / p.tile_tokens);
    lc.blockDim = dim3(32 * kMidWarps + 32, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

// ------------------------------------------------------------------ product

template <bool PAIR, int BN, int STAGES, int CPW, int EB> struct Int8Layout {
    static constexpr int kTileM = PAIR ? 256 : 128;
    static constexpr int kPromoWG = BN / CPW;
    static constexpr int kThreads = 128 + 128 * kPromoWG;
    // A stage: 128 columns of K, as two 64-column halves of this CTA's rows of A
    // (128) and of B.  (One wait and one commit for eight MMAs: the issuing warp
    // takes longer over four with theirs than the tensor core.)
    static constexpr uint32_t kAHalf = 128u * 128u;
    static constexpr uint32_t kBHalf = static_cast<uint32_t>(PAIR ? BN / 2 : BN) * 128u;
    static constexpr uint32_t kABytes = 2 * kAHalf, kBBytes = 2 * kBHalf;
    static constexpr int kBufs = 512 / BN;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr size_t kStageBytes = STAGES * (kABytes + kBBytes);
    static constexpr size_t kEpiBytes = 4 * kPromoWG * 2048 * EB;
    static constexpr size_t kScaleBytes = 4 * kPromoWG * CPW * 4;                // b_s, per warp
    static constexpr int kRegsLow = 56, kRegsHigh = 224;
    static_assert(kThreads == 384 && 128 * kRegsLow + 256 * kRegsHigh <= 384 * 168,
                  "register split exceeds the launch's registers");
    // full, empty per stage; tfull, tempty per buffer; drain
    static constexpr int kBars = 2 * STAGES + 2 * kBufs + 1;
    static constexpr size_t kSmem = 1024 + kStageBytes + kEpiBytes + kScaleBytes + kBars * 8 + 16;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

constexpr int kRaster = 8;           // M tiles per raster group

__device__ __forceinline__ void int8_tile_coords(int t, int num_m, int num_n, int &mb, int &nb)
{
    const int per_group = kRaster * num_n;
    const int gid = t / per_group;
    const int first_m = gid * kRaster;
    const int gm = min(num_m - first_m, kRaster);
    const int r = t - gid * per_group;
    mb = first_m + r % gm;
    nb = r / gm;
}

// One persistent CTA (PAIR: one CTA pair, sharing 256 x BN tiles through
// cta_group::2 MMAs) per SM (SM pair).  Roles, barriers and the pair's protocol
// are those of the FP8 kernels (gemm_tiled.cu, gemm_pair.cu) without their
// per-group scales: warp 0 TMA producer, warp 1 MMA issuer (the odd CTA's:
// forwarder of its landed stages), warps 4.. integer promotion and epilogue.
// Bound by the tensor cores under the power cap: 16384 x 4096 x 4096 with the
// widening launch takes 340 us, without it about 300, 1.83 PFLOP/s (one-CTA tiles: 433).
template <bool PAIR, int BN, int STAGES, int CPW, int EB>
__global__ void __launch_bounds__(Int8Layout<PAIR, BN, STAGES, CPW, EB>::kThreads, 1)
    k_int8_mma(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmC, const Int8Params p)
{
    using L = Int8Layout<PAIR, BN, STAGES, CPW, EB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sB = smem_addr(smem);
    const uint32_t sA = sB + STAGES * L::kBBytes;
    const uint32_t sEpi = sB + static_cast<uint32_t>(L::kStageBytes);
    float *scales = reinterpret_cast<float *>(smem + L::kStageBytes + L::kEpiBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kStageBytes + L::kEpiBytes +
                                                  L::kScaleBytes);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + L::kBufs + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * L::kBufs);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const uint32_t warp = warp_uniform(warp_index()), lane = lane_index();
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int first_tile = static_cast<int>(PAIR ? blockIdx.x >> 1 : blockIdx.x);
    const int tile_stride = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // rank 0 of a pair also counts its peer's landed stage
            mbar_init(full_bar(s), PAIR && rank == 0 ? 2 : 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < L::kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), (PAIR ? 2 : 1) * 4 * L::kPromoWG);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        tma_prefetch_map(&tmC);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), L::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(tmem_slot), L::kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    if constexpr (PAIR)
        cluster_sync();      // barriers of both CTAs initialised, TMEM allocated in both
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = warp_uniform(*tmem_slot);
    const WaitGuard guard{abort_flag, p.status, p.wait_limit};

    grid_launch_dependents();
    grid_dependency_wait();

    // A role that gives up also raises the peer's abort flag.
    auto abort_peer = [&]() {
        if constexpr (PAIR) {
            const uint32_t peer_flag =
                cluster_map(smem_addr(const_cast<int *>(abort_flag)), rank ^ 1u);
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_flag), "r"(1u) : "memory");
        }
    };

    if (warp < 4) {
        regs_dealloc<L::kRegsLow>();
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int t = first_tile; ok && t < p.num_tiles; t += tile_stride) {
                int mb, nb;
                int8_tile_coords(t, p.num_m_tiles, p.num_n_tiles, mb, nb);
                const int arow0 = mb * L::kTileM + 128 * static_cast<int>(rank);
                const int brow = nb * BN + (PAIR ? (BN / 2) * static_cast<int>(rank) : 0);
                for (int g = 0; g < p.steps; ++g) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, guard, SITE_TILED_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const int arow = arow0 + ((W8A8_DEBUG_BOUNDS && issued == 0 &&
                                               p.debug_skip_tma == kDebugBadFirstLoad)
                                                  ? (1 << 28)
                                                  : 0);
                    const bool in =
                        in_bounds(arow < p.num_m_tiles * L::kTileM, p.status, SITE_BOUNDS_A) &&
                        in_bounds(brow < p.num_n_tiles * BN, p.status, SITE_BOUNDS_B);
                    if (issued != p.debug_skip_tma && in) {
                        mbar_arrive_expect_tx(full_bar(stage), L::kABytes + L::kBBytes);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_load_2d(sA + stage * L::kABytes + h * L::kAHalf, &tmA, full_bar(stage),
                                        g * 256 + 128 * h, arow);
                            tma_load_2d(sB + stage * L::kBBytes + h * L::kBHalf, &tmB, full_bar(stage),
                                        g * 256 + 128 * h, brow);
                        }
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
                // Tail: every stage released by the MMA, so that no commit
                // arrives on this CTA after it has left.
                for (int s = 0; s < STAGES && ok; ++s) {
                    ok = wait_bounded(empty_bar(stage), phase ^ 1u, guard, SITE_TILED_PRODUCER);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                abort_peer();
                // Drain this CTA's own loads (the last issue into each stage).
                for (int s = 0; s < STAGES; ++s) {
                    const bool this_round = s < next_stage;
                    if (!this_round && issued < STAGES && s >= issued)
                        continue;
                    wait_drain(full_bar(s), this_round ? next_phase : (next_phase ^ 1u), p.status,
                               p.wait_limit, (SITE_DRAIN << 8) | 4u);
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ---------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_f16_f32(L::kTileM, BN);
            int stage = 0;
            uint32_t phase = 0;
            uint32_t it = 0;                 // accumulator uses
            bool ok = true, ready = false;
            for (int t = first_tile; ok && t < p.num_tiles; t += tile_stride) {
                for (int g = 0; g < p.steps; ++g) {
                    const uint32_t buf = it % L::kBufs;
                    const int in_chunk = g % kChunkStages;
                    ok = __all_sync(
                        0xffffffffu,
                        (in_chunk > 0 || wait_bounded(tempty_bar(buf), ((it / L::kBufs) & 1u) ^ 1u,
                                                      guard, SITE_TILED_MMA_TMEM)) &&
                            (ready || wait_bounded(full_bar(stage), phase, guard,
                                                   SITE_TILED_MMA_FULL)));
                    if (!ok)
                        break;
                    // the next stage's probe answers while this one's MMAs are issued
                    ready = mbar_test_wait(full_bar(stage + 1 < STAGES ? stage + 1 : 0),
                                           stage + 1 < STAGES ? phase : phase ^ 1u);
                    tc_fence_after_sync();
                    const uint32_t d = tmem_base + buf * BN;
                    const uint64_t ad = sw128_kmajor_desc(sA + stage * L::kABytes);
                    const uint64_t bd = sw128_kmajor_desc(sB + stage * L::kBBytes);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_f16_elect<PAIR>(d, ad + 2u * (kk % 4) + (kk / 4) * (L::kAHalf >> 4),
                                            bd + 2u * (kk % 4) + (kk / 4) * (L::kBHalf >> 4), idesc,
                                            (in_chunk > 0 || kk > 0) ? 1u : 0u);
                    const bool last = in_chunk == kChunkStages - 1 || g == p.steps - 1;
                    mma_commit_elect<PAIR>(empty_bar(stage));
                    if (last) {
                        mma_commit_elect<PAIR>(tfull_bar(buf));
                        ++it;
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && lane == 0)
                abort_peer();
            // Every MMA has finished reading shared memory and writing TMEM
            // before the CTA (pair) can pass its final barrier.
            mma_commit_elect<PAIR>(drain_bar, 1);
            wait_drain(drain_bar, 0, p.status, p.wait_limit, (SITE_DRAIN << 8) | 4u);
        } else if (PAIR && warp == 1 && lane == 0) {
            // ---------------------------------------------------------- forwarder (rank 1)
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first_tile; ok && t < p.num_tiles; t += tile_stride) {
                for (int g = 0; g < p.steps; ++g) {
                    if (!wait_bounded(full_bar(stage), phase, guard, SITE_PAIR_PEER)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote(cluster_map(full_bar(stage), 0));
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok)
                abort_peer();
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------- promotion + epilogue
        regs_alloc<L::kRegsHigh>();
        const uint32_t w = warp_index();       // (the uniform copy costs more spills; these are 28 bytes)
        const int h = static_cast<int>(w / 4) - 1;
        const uint32_t q = w & 3u;
        const uint32_t epi_buf = sEpi + (w - 4u) * 2048u * EB;
        float *my_bs = scales + (w - 4u) * CPW;
        const bool fp32 = p.out_kind == OUT_FP32, bf = p.out_kind == OUT_BF16;
        uint32_t it = 0;
        bool ok = true;
        for (int t = first_tile; t < p.num_tiles; t += tile_stride) {
            int mb, nb;
            int8_tile_coords(t, p.num_m_tiles, p.num_n_tiles, mb, nb);
            const int col0 = nb * BN + h * CPW;
            const int y = mb * L::kTileM + 128 * static_cast<int>(rank) + static_cast<int>(q * 32);
            const int rows = min(32, p.M - y);
            // This warp's column scales, and the lane's row scale.
            __syncwarp();
            for (int c = static_cast<int>(lane); c < CPW; c += 32)
                my_bs[c] = col0 + c < p.N ? __ldg(p.b_s + col0 + c) : 0.f;
            const float as = static_cast<int>(lane) < rows ? __ldg(p.a_s + y + lane) : 0.f;
            __syncwarp();
            int acc[CPW];
#pragma unroll
            for (int j = 0; j < CPW; ++j)
                acc[j] = 0;
            for (int g = 0; g < p.steps; g += kChunkStages) {
                const uint32_t buf = it % L::kBufs;
                ok = __all_sync(0xffffffffu, wait_bounded(tfull_bar(buf), (it / L::kBufs) & 1u,
                                                          guard, SITE_TILED_PROMOTE));
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t taddr = tmem_base + ((q * 32u) << 16) + buf * BN + h * CPW;
#pragma unroll
                for (int c = 0; c < CPW / 32; ++c) {
                    float v[32];
                    tmem_load_32cols(taddr + 32u * c, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        acc[32 * c + j] += __float2int_rn(v[j]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        mbar_arrive_remote(cluster_map(tempty_bar(buf), 0));
                    else
                        mbar_arrive(tempty_bar(buf));
                }
                ++it;
            }
            if (!ok)
                break;
            if (rows > 0 && col0 < p.N &&
                in_bounds(y + rows <= p.M && y >= 0, p.status, SITE_BOUNDS_C)) {
                auto pack = [&](int k, int j) {
                    if (fp32) {
                        const int c = (16 * k + 4 * j) % CPW;
                        const float4 s = *reinterpret_cast<const float4 *>(my_bs + c);
                        return make_uint4(__float_as_uint(__int2float_rn(acc[c]) * as * s.x),
                                          __float_as_uint(__int2float_rn(acc[c + 1]) * as * s.y),
                                          __float_as_uint(__int2float_rn(acc[c + 2]) * as * s.z),
                                          __float_as_uint(__int2float_rn(acc[c + 3]) * as * s.w));
                    }
                    const int c = (32 * k + 8 * j) % CPW;
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 s = *reinterpret_cast<const float2 *>(my_bs + c + 2 * i);
                        const float lo = __int2float_rn(acc[c + 2 * i]) * as * s.x;
                        const float hi = __int2float_rn(acc[c + 2 * i + 1]) * as * s.y;
                        w[i] = bf ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                    }
                    return make_uint4(w[0], w[1], w[2], w[3]);
                };
                store_warp_rows<CPW, EB>(pack, &tmC, epi_buf, lane, col0, y, p.N, fp32, p.tma_store,
                                         false, rows, p.C, p.ldc);
            }
        }
        if (!ok && lane == 0)
            abort_peer();
        if (lane == 0)
            tma_store_wait_read();
    }

    tc_fence_before_sync();
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem_base, L::kTmemCols);
        else
            tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

template <bool PAIR, int BN, int STAGES, int CPW, int EB>
cudaError_t launch_mma(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmC,
                       const Int8Params &p, const LaunchCfg &cfg, int *clusters)
{
    using L = Int8Layout<PAIR, BN, STAGES, CPW, EB>;
    auto kernel = k_int8_mma<PAIR, BN, STAGES, CPW, EB>;
    static volatile int smem_set[kMaxDeviceFlags] = {};
    cudaError_t e = ensure_smem_limit(kernel, smem_set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(clusters ? 2 : cfg.grid, 1, 1);
    lc.blockDim = dim3(L::kThreads, 1, 1);
    lc.dynamicSmemBytes = L::kSmem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (PAIR) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    lc.attrs = attr;
    if (clusters) {
        lc.numAttrs = n;
        return cudaOccupancyMaxActiveClusters(clusters, kernel, &lc);
    }
    // Behind the widening launch it always overlaps that one's tail: it waits
    // for it before its first access.
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    lc.numAttrs = n + 1;
    return cudaLaunchKernelEx(&lc, kernel, tmA, tmB, tmC, p);
}

}  // namespace

cudaError_t launch_int8_small(const Int8SmallParams &p, int access, int sm_count, cudaStream_t stream)
{
    if (p.M <= 8)
        return launch_small_t<1, 1, 2>(p, access, sm_count, stream);
    if (p.M <= 16)
        return launch_small_t<2, 1, 2>(p, access, sm_count, stream);
    return launch_small_t<4, 2, 1>(p, access, sm_count, stream);
}

namespace {

// CTAs of k_int8_mid that run at once when they come in clusters of s (1, 2, 4, 8):
// one to an SM, and clusters do not cross the GPU's processing clusters, so that
// those of 8 leave some SMs idle.
int mid_at_once(int s, int sm_count)
{
    static volatile int cached[kMaxDeviceFlags][9] = {};
    int dev = 0, n = 0;
    if (s == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDeviceFlags)
        return sm_count;
    if (cached[dev][s])
        return cached[dev][s];
    auto kernel = k_int8_mid<6, 2, 16>;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(1, s, 1);
    lc.blockDim = dim3(32 * kMidWarps + 32, 1, 1);
    lc.dynamicSmemBytes = kMidSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = static_cast<unsigned>(s);
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMidSmem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &lc) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = std::max(1, sm_count / s / 2);
    }
    cached[dev][s] = n * s;
    return n * s;
}

// Estimated microseconds of k_int8_mid with token tiles of nt and K split by s:
// per wave of CTAs a fixed part, its steps, and adding up and storing the tile.
// (Fitted on a GB300 for N x K from 512 x 512 to 8192 x 4096 and M from 48 to 1024;
// a step's 740 to 1330 cycles are the MMA issue for few tokens and the shared
// memory's bandwidth for many.)
float mid_cost(int blocks, int tiles, int nt, int s, int steps, int sm_count)
{
    const int at_once = mid_at_once(s, sm_count);
    const float waves = static_cast<float>((blocks * static_cast<long long>(tiles) * s + at_once - 1) / at_once);
    const float cycles = 5500.f + static_cast<float>((steps + s - 1) / s) * (700.f + 2.45f * nt) +
                         (s > 1 ? 50.f : 30.f) * nt;
    return 1.f + waves * cycles / 1900.f;
}

}  // namespace

float int8_mid_plan(int M, int N, int K, int sm_count, int *tile_tokens, int *splits)
{
    const int steps = (K + 63) / 64, blocks = (N + 127) / 128;
    const int fixed_nt = *tile_tokens, fixed_s = *splits;
    float best = -1.f;
    const int fewest = fixed_nt ? (M + fixed_nt - 1) / fixed_nt : (M + 255) / 256;
    const int most = fixed_nt ? fewest : std::min(fewest + 7, (M + 15) / 16);
    for (int tiles = fewest; tiles <= most; ++tiles) {
        const int nt = fixed_nt ? fixed_nt : ((M + tiles - 1) / tiles + 15) / 16 * 16;
        // The 512 columns of tensor memory hold 512 / nt buffers of 8 steps.
        const int room = 512 / ((nt + 31) / 32 * 32) * kChunkSteps;
        for (int s = fixed_s ? fixed_s : 1; s <= (fixed_s ? fixed_s : 8); s *= 2) {
            if ((steps + s - 1) / s > room || (!fixed_s && s > 1 && s > steps) || tiles > 65535)
                continue;
            const float c = mid_cost(blocks, (M + nt - 1) / nt, nt, s, steps, sm_count);
            if (best < 0.f || c < best) {
                best = c;
                *tile_tokens = nt;
                *splits = s;
            }
        }
    }
    return best;
}

// The same for widening in a launch of its own and multiplying 128 x 128 tiles or
// a CTA pair's 256 x 256: both launches, the widened elements (mostly in L2), and
// per wave a tile's stages of 128 columns and its stores.
float int8_tiled_cost(int M, int N, int K, int sm_count, int pair)
{
    const long long tile = pair ? 256 : 128, at_once = pair ? sm_count / 2 : sm_count;
    const long long tiles = (M + tile - 1) / tile * ((N + tile - 1) / tile);
    const float stages = static_cast<float>((K + 127) / 128);
    return 6.f + (static_cast<float>(M) + static_cast<float>(N)) * static_cast<float>(K) / 5.2e6f +
           static_cast<float>((tiles + at_once - 1) / at_once) *
               (pair ? 3.f + 0.64f * stages : 0.4f + 0.46f * stages);
}

cudaError_t launch_int8_mid(const Int8MidParams &p, int access, int splits, cudaStream_t stream)
{
    const int ch = (4 * (128 + p.tile_tokens) + 255) / 256;
    return ch <= 3 ? launch_mid_t<3, 3>(p, access, splits, stream)
                   : ch <= 4 ? launch_mid_t<4, 2>(p, access, splits, stream)
                             : launch_mid_t<6, 2>(p, access, splits, stream);
}

cudaError_t launch_int8_widen(const Int8WidenParams &p, int access, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid, 1, 1);
    lc.blockDim = dim3(kWidenThreads, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, access == 16  ? k_int8_widen<16>
                                   : access == 8 ? k_int8_widen<8>
                                   : access == 4 ? k_int8_widen<4>
                                                 : k_int8_widen<1>,
                              p);
}

cudaError_t launch_int8_mma(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmC,
                            const Int8Params &p, int pair, const LaunchCfg &cfg)
{
    return pair ? launch_mma<true, 256, 3, 128, 1>(tmA, tmB, tmC, p, cfg, nullptr)
                : launch_mma<false, 128, 3, 64, 1>(tmA, tmB, tmC, p, cfg, nullptr);
}

int int8_max_pairs()
{
    static volatile int cached[kMaxDeviceFlags] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDeviceFlags)
        return -1;
    if (cached[dev] > 0)
        return cached[dev];
    const CUtensorMap none = {};
    if (launch_mma<true, 256, 3, 128, 1>(none, none, none, Int8Params{}, LaunchCfg{}, &n) !=
            cudaSuccess ||
        n <= 0)
        return -1;
    cached[dev] = n;
    return n;
}

}  // namespace w8a8
