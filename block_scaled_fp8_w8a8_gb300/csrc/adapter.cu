// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scales[l] * (x[t] A[l]^T) B[l]^T,   l the adapter of row t
//
// with rows sorted by adapter (group_rows): adapter l's are order[offsets[l]] ..
// order[offsets[l+1] - 1]; rows behind offsets[L] have none and are base's.
//
// A cluster of CTAs takes up to 8 NT rows of one adapter.  First each CTA multiplies
// its share of K: h^T = A[l] x^T by mma.sync, A's rows on the M side, tokens on the
// N side, operands straight from global memory in 16-byte pieces (a permutation of K
// that both operands share).  Partial h go to every CTA of the cluster through
// distributed shared memory and are added in rank order, so that all have the same
// bits.  Then each CTA takes its share of N: out^T = base^T + B[l] h^T.
//
// h is kept to fp32: an MMA takes 16-bit operands, so h is split into a sum of two or
// three of them, each the rounding of what the ones before leave.  bf16: two leave an
// error of 2^-18 (16-bit output, whose rounding is 2^-9), three one of 2^-27 (fp32
// output).  fp16: two leave 2^-24; h is first scaled by a power of two per row so that
// its largest element is near 2^14, because fp16's range is narrow.
#include <algorithm>
#include <cstdio>

#include "../../include/w8a8_block_fp8.h"
#include "adapter.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {
w8a8_status record_error(w8a8_status st, const char *message);

namespace {

using namespace lora;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 64;          // rows of A whose sums a warp holds at once
constexpr int kMaxCluster = 8;

// Eight elements of a row at k, zeros past its end (row null: zeros).
__device__ __forceinline__ uint4 load8(const uint16_t *row, int k, int K, bool vec)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!row || k >= K)
        return v;
    if (vec)
        return *reinterpret_cast<const uint4 *>(row + k);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
        w[i] = hi << 16 | lo;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 load4(const uint16_t *row, int k, int K, bool vec)
{
    if (!row || k >= K)
        return make_uint2(0, 0);
    if (vec)
        return *reinterpret_cast<const uint2 *>(row + k);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
        w[i] = hi << 16 | lo;
    }
    return make_uint2(w[0], w[1]);
}

// D (16 x 8) += A (16 x 16) B (16 x 8), fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int OUT> __device__ __forceinline__ float load_out(const void *p, long long i)
{
    if constexpr (OUT == W8A8_OUT_FP32)
        return static_cast<const float *>(p)[i];
    else if constexpr (OUT == W8A8_OUT_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else
        return __half2float(static_cast<const __half *>(p)[i]);
}
template <int OUT> __device__ __forceinline__ void store_out(void *p, long long i, float v)
{
    if constexpr (OUT == W8A8_OUT_FP32)
        static_cast<float *>(p)[i] = v;
    else if constexpr (OUT == W8A8_OUT_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// Shared memory: partial sums of the warps (later h's parts as MMA operands), every
// CTA's partial h, h itself.
template <int NT> struct FewSmem {
    static constexpr int kRows = 8 * NT;
    static __host__ __device__ size_t part(int terms, int r_pad)
    {
        const size_t sums = sizeof(float) * kWarps * kChunk * kRows, frags = sizeof(uint2) * 32 * (r_pad / 16) * NT * terms;
        return sums > frags ? sums : frags;
    }
    static __host__ __device__ size_t received(int r_pad, int cluster) { return sizeof(float) * r_pad * kRows * cluster; }
    static __host__ __device__ size_t bytes(int terms, int r_pad, int cluster)
    {
        return part(terms, r_pad) + received(r_pad, cluster) + sizeof(float) * r_pad * kRows;
    }
};

template <bool BF16, int OUT, int NT> __global__ void __launch_bounds__(kThreads) k_adapter_few(const AdapterParams p)
{
    constexpr int kRows = 8 * NT, kTerms = BF16 && OUT == W8A8_OUT_FP32 ? 3 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[16];
    __shared__ int rows[kRows];
    __shared__ float factor[kRows];         // what a row's sums are multiplied by (fp16)
    uint32_t ctas, cluster;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
    const uint32_t me = cluster_ctarank();
    float *const part = reinterpret_cast<float *>(smem);
    float *const received = reinterpret_cast<float *>(smem + FewSmem<NT>::part(kTerms, p.r_pad));
    float *const h = received + p.r_pad * kRows * ctas;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const Item item = find_item<kThreads>(p, static_cast<int>(cluster), kRows, p.out == p.base ? p.L : p.L + 1, scratch);
    if (item.rows == 0)
        return;                             // the whole cluster
    if (threadIdx.x < kRows) {
        int row = threadIdx.x < item.rows ? p.order[item.first + threadIdx.x] : -1;
        rows[threadIdx.x] = static_cast<unsigned>(row) < static_cast<unsigned>(p.T) ? row : -1;
    }
    __syncthreads();
    const int n_tiles = (p.N + 15) / 16;
    const int tile_lo = static_cast<int>(static_cast<long long>(n_tiles) * me / ctas);
    const int tile_hi = static_cast<int>(static_cast<long long>(n_tiles) * (me + 1) / ctas);
    if (item.adapter == p.L) {
        const int from = tile_lo * 16, to = min(tile_hi * 16, p.N);
        constexpr int kElement = OUT == W8A8_OUT_FP32 ? 4 : 2;
        if (p.vec_n)
            copy_rows<uint4, kThreads>(p, rows, item.rows, from, to, kElement);
        else if constexpr (kElement == 4)
            copy_rows<uint32_t, kThreads>(p, rows, item.rows, from, to, kElement);
        else
            copy_rows<uint16_t, kThreads>(p, rows, item.rows, from, to, kElement);
        return;
    }
    const uint16_t *const A = p.A + static_cast<long long>(item.adapter) * p.r * p.K;
    const uint16_t *const B = p.B + static_cast<long long>(item.adapter) * p.N * p.r;

    if (ctas > 1)                           // peers write here once every CTA has started
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    // h^T, this CTA's share of K
    const int blocks = (p.K + 63) / 64;
    const int lo = static_cast<int>(static_cast<long long>(blocks) * me / ctas);
    const int hi = static_cast<int>(static_cast<long long>(blocks) * (me + 1) / ctas);
    const uint16_t *token[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = rows[8 * t + g];
        token[t] = row >= 0 ? p.x + row * p.ld_x : nullptr;
    }
    for (int r0 = 0; r0 < p.r_pad; r0 += kChunk) {
        float acc[4][NT][4] = {};
        const int m_tiles = min(4, (p.r_pad - r0) / 16);
        for (int b = lo + warp; b < hi; b += kWarps) {
            const int k = b * 64 + 8 * c;
            uint4 xv[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    xv[t][s] = load8(token[t], k + 32 * s, p.K, p.vec_k);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m >= m_tiles)
                    continue;
                const int r_lo = r0 + 16 * m + g, r_hi = r_lo + 8;
                const uint16_t *const a_lo = r_lo < p.r ? A + static_cast<long long>(r_lo) * p.K : nullptr;
                const uint16_t *const a_hi = r_hi < p.r ? A + static_cast<long long>(r_hi) * p.K : nullptr;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint4 u = load8(a_lo, k + 32 * s, p.K, p.vec_k), v = load8(a_hi, k + 32 * s, p.K, p.vec_k);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma<BF16>(acc[m][t], u.x, v.x, u.y, v.y, xv[t][s].x, xv[t][s].y);
                        mma<BF16>(acc[m][t], u.z, v.z, u.w, v.w, xv[t][s].z, xv[t][s].w);
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2 *>(part + ((warp * kChunk + 16 * m + g + 8 * i) * kRows + 8 * t + 2 * c)) =
                        make_float2(acc[m][t][2 * i], acc[m][t][2 * i + 1]);
        __syncthreads();
        if (ctas > 1 && r0 == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        for (int i = threadIdx.x; i < 16 * m_tiles * kRows; i += kThreads) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += part[w * kChunk * kRows + i];
            const uint32_t at = smem_addr(received + me * p.r_pad * kRows + r0 * kRows + i);
            for (uint32_t q = 0; q < ctas; ++q)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(at, q)), "f"(sum) : "memory");
        }
        __syncthreads();
    }
    if (ctas > 1) {
        if (p.r_pad == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        cluster_sync();
    }
    const float scale = p.scales ? p.scales[item.adapter] : 1.f;
    for (int i = threadIdx.x; i < p.r_pad * kRows; i += kThreads) {
        float sum = 0.f;
        for (uint32_t q = 0; q < ctas; ++q)
            sum += received[q * p.r_pad * kRows + i];
        h[i] = sum * scale;
    }
    __syncthreads();
    if constexpr (!BF16) {
        for (int t = warp; t < kRows; t += kWarps) {
            float top = 0.f;
            for (int i = lane; i < p.r_pad; i += 32)
                top = fmaxf(top, fabsf(h[i * kRows + t]));
#pragma unroll
            for (int d = 16; d; d /= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            float shrink, back;
            power_of(top, &shrink, &back);
            for (int i = lane; i < p.r_pad; i += 32)
                h[i * kRows + t] *= shrink;
            if (lane == 0)
                factor[t] = back;
        }
        __syncthreads();
    }
    // h's parts as B operands: lane (g, c) of step s has elements 16 s + 4 c .. + 3 of token g
    const int steps = p.r_pad / 16;
    uint2 *const frags = reinterpret_cast<uint2 *>(part);
    for (int i = threadIdx.x; i < steps * NT * 32; i += kThreads) {
        const int ln = i & 31, t = (i >> 5) % NT, s = (i >> 5) / NT;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = h[(16 * s + 4 * (ln & 3) + j) * kRows + 8 * t + (ln >> 2)];
#pragma unroll
        for (int q = 0; q < kTerms; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = take_part<BF16>(v[j]);
            frags[((s * NT + t) * kTerms + q) * 32 + ln] = make_uint2(w[1] << 16 | w[0], w[3] << 16 | w[2]);
        }
    }
    __syncthreads();
    // out^T, this CTA's share of N
    for (int tile = tile_lo + warp; tile < tile_hi; tile += kWarps) {
        const int n_lo = tile * 16 + g, n_hi = n_lo + 8;
        const uint16_t *const b_lo = n_lo < p.N ? B + static_cast<long long>(n_lo) * p.r : nullptr;
        const uint16_t *const b_hi = n_hi < p.N ? B + static_cast<long long>(n_hi) * p.r : nullptr;
        float acc[NT][4] = {};
#pragma unroll 4
        for (int s = 0; s < steps; ++s) {
            const uint2 u = load4(b_lo, 16 * s + 4 * c, p.r, p.vec_r), v = load4(b_hi, 16 * s + 4 * c, p.r, p.vec_r);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int q = 0; q < kTerms; ++q) {
                    const uint2 f = frags[((s * NT + t) * kTerms + q) * 32 + lane];
                    mma<BF16>(acc[t], u.x, v.x, u.y, v.y, f.x, f.y);
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = i < 2 ? n_lo : n_hi, slot = 8 * t + 2 * c + (i & 1), row = rows[slot];
                if (n < p.N && row >= 0) {
                    const float f = BF16 ? 1.f : factor[slot];
                    store_out<OUT>(p.out, row * p.ld_out + n, fmaf(acc[t][i], f, load_out<OUT>(p.base, row * p.ld_base + n)));
                }
            }
    }
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool BF16, int OUT, int NT>
cudaError_t launch_few(const AdapterParams &p, long long items, const DeviceView &dev, cudaStream_t stream)
{
    constexpr int kTerms = BF16 && OUT == W8A8_OUT_FP32 ? 3 : 2;
    constexpr size_t kRoom = 200 * 1024;
    auto kernel = k_adapter_few<BF16, OUT, NT>;
    // As many CTAs share an item as fill the SMs twice, with 128 columns of K for each.
    int cluster = 1;
    while (cluster < kMaxCluster && items * cluster * 2 <= 2ll * dev.sm_count && cluster * 2 * 128 <= p.K &&
           FewSmem<NT>::bytes(kTerms, p.r_pad, cluster * 2) <= kRoom)
        cluster *= 2;
    const size_t smem = FewSmem<NT>::bytes(kTerms, p.r_pad, cluster);
    static volatile int flags[kMaxDeviceFlags] = {};
    if (const cudaError_t e = allow_smem(kernel, kRoom, flags); e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(items * cluster), 1, 1);
    lc.blockDim = dim3(kThreads, 1, 1);
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

template <bool BF16, int OUT> cudaError_t launch_adapter(const AdapterParams &p, const DeviceView &dev, cudaStream_t s)
{
    const long long groups = p.out == p.base ? p.L : p.L + 1;
    if (groups == 0)
        return cudaSuccess;
    if (p.T <= 4 * p.L)
        return launch_few<BF16, OUT, 1>(p, most_items(p.T, groups, 8), dev, s);
    return launch_few<BF16, OUT, 2>(p, most_items(p.T, groups, 16), dev, s);
}

// Whether a problem's sizes are for the tiles of 128 rows (adapter_tile.cu): where adapters
// have many rows on average.
bool tiled(const AdapterParams &p) { return p.L > 0 && p.T >= 32 * p.L && p.r >= 8 && p.K >= 64; }

size_t workspace_bytes(const AdapterParams &p)
{
    return tiled(p) ? sizeof(float) * tile_splits(p) * p.T * p.r_pad : 0;
}

}  // namespace
}  // namespace w8a8

extern "C" size_t w8a8_adapter_workspace_size(int64_t T, int64_t L, int64_t r, int64_t K)
{
    using namespace w8a8;
    if (T <= 0 || L <= 0 || r <= 0 || K <= 0 || L > W8A8_GROUPS_MAX || r > W8A8_ADAPTER_MAX_R || T >= (1ll << 28) ||
        K > (1ll << 24))
        return 0;
    AdapterParams p = {};
    p.T = static_cast<int>(T);
    p.L = static_cast<int>(L);
    p.r = static_cast<int>(r);
    p.K = static_cast<int>(K);
    p.r_pad = static_cast<int>((r + 15) / 16 * 16);
    return workspace_bytes(p);
}

extern "C" w8a8_status w8a8_adapter_matmul(const void *x_dev, w8a8_in_dtype dtype, int64_t ld_x, const void *A_dev,
                                           const void *B_dev, const int32_t *order_dev, const int32_t *offsets_dev,
                                           const float *scales_dev, const void *base_dev, int64_t ld_base,
                                           void *out_dev, w8a8_out_dtype out_dtype, int64_t ld_out, int64_t T,
                                           int64_t L, int64_t r, int64_t K, int64_t N, void *workspace_dev,
                                           size_t workspace_bytes, w8a8_stream_t stream)
{
    using namespace w8a8;
    if (T < 0 || L < 0 || r < 0 || K < 0 || N < 0)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size");
    if (dtype < W8A8_IN_BF16 || dtype > W8A8_IN_FP32 || out_dtype < W8A8_OUT_BF16 || out_dtype > W8A8_OUT_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown dtype");
    if (dtype == W8A8_IN_FP32)
        return record_error(W8A8_ERR_UNSUPPORTED, "x, A and B must be bf16 or fp16");
    if (out_dtype != W8A8_OUT_FP32 && static_cast<int>(out_dtype) != static_cast<int>(dtype))
        return record_error(W8A8_ERR_UNSUPPORTED, "base and out must have x's type or fp32");
    ld_x = ld_x ? ld_x : K;
    ld_base = ld_base ? ld_base : N;
    ld_out = ld_out ? ld_out : N;
    if (ld_x < K || ld_base < N || ld_out < N)
        return record_error(W8A8_ERR_INVALID_ARG, "a row stride is shorter than its row");
    if (base_dev == out_dev && ld_base != ld_out)
        return record_error(W8A8_ERR_INVALID_ARG, "out in base's place with another row stride");
    if (T == 0 || N == 0)
        return W8A8_OK;
    if (!base_dev || !out_dev || !order_dev || !offsets_dev)
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (L > 0 && r > 0 && K > 0 && (!x_dev || !A_dev || !B_dev))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (L > W8A8_GROUPS_MAX || r > W8A8_ADAPTER_MAX_R || T >= (1ll << 28) || K > (1ll << 24) || N > (1ll << 24))
        return record_error(W8A8_ERR_UNSUPPORTED, "L above W8A8_GROUPS_MAX, r above W8A8_ADAPTER_MAX_R, T of 2^28 or "
                                                  "more, or K or N above 2^24");
    const int ob = out_dtype == W8A8_OUT_FP32 ? 4 : 2;
    if (!on(x_dev, 2) || !on(A_dev, 2) || !on(B_dev, 2) || !on(order_dev, 4) || !on(offsets_dev, 4) ||
        !on(scales_dev, 4) || !on(base_dev, ob) || !on(out_dev, ob))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    AdapterParams p = {};
    p.x = static_cast<const uint16_t *>(x_dev);
    p.A = static_cast<const uint16_t *>(A_dev);
    p.B = static_cast<const uint16_t *>(B_dev);
    p.order = order_dev;
    p.offsets = offsets_dev;
    p.scales = scales_dev;
    p.base = base_dev;
    p.out = out_dev;
    p.ld_x = ld_x;
    p.ld_base = ld_base;
    p.ld_out = ld_out;
    p.T = static_cast<int>(T);
    p.L = static_cast<int>(L);
    p.r = static_cast<int>(r);
    p.K = static_cast<int>(K);
    p.N = static_cast<int>(N);
    p.r_pad = static_cast<int>((r + 15) / 16 * 16);
    p.vec_k = K % 8 == 0 && ld_x % 8 == 0 && on(x_dev, 16) && on(A_dev, 16);
    p.vec_r = r % 4 == 0 && on(B_dev, 8);
    const int each = 16 / ob;
    p.vec_n = N % each == 0 && ld_base % each == 0 && ld_out % each == 0 && on(base_dev, 16) && on(out_dev, 16);
    const bool tiles = tiled(p) && tile_takes(p);
    if (const size_t need = tiles ? w8a8::workspace_bytes(p) : 0;
        need && (!workspace_dev || workspace_bytes < need || !on(workspace_dev, 16))) {
        char msg[160];
        snprintf(msg, sizeof(msg), "workspace of %zu bytes at %p: need %zu bytes, 16-byte aligned", workspace_bytes,
                 workspace_dev, need);
        return record_error(W8A8_ERR_WORKSPACE, msg);
    }
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (tiles)
        e = launch_tile(p, dtype, out_dtype, static_cast<float *>(workspace_dev), dev, s);
    else if (dtype == W8A8_IN_BF16)
        e = out_dtype == W8A8_OUT_FP32 ? launch_adapter<true, W8A8_OUT_FP32>(p, dev, s)
                                       : launch_adapter<true, W8A8_OUT_BF16>(p, dev, s);
    else
        e = out_dtype == W8A8_OUT_FP32 ? launch_adapter<false, W8A8_OUT_FP32>(p, dev, s)
                                       : launch_adapter<false, W8A8_OUT_FP16>(p, dev, s);
    if (e == cudaSuccess)
        return W8A8_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "kernel launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return record_error(W8A8_ERR_CUDA, msg);
}
