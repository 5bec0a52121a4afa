// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scales[l] * (x[t] A[l]^T) B[l]^T,   l the adapter of row t
//
// with rows sorted by adapter (group_rows): adapter l's are order[offsets[l]] ..
// order[offsets[l+1] - 1]; rows behind offsets[L] have none and are base's.
//
// A cluster of CTAs takes up to 16 rows of one adapter.  First each CTA multiplies
// its share of K: h = x A[l]^T by mma.sync, tokens on the M side, A's rows on the N side,
// operands straight from global memory in 16-byte pieces (a permutation of K that both
// operands share).  Partial h go to every CTA of the cluster through distributed shared
// memory and are added in rank order, so that all have the same bits.  Then each CTA takes
// its share of N: out = base + h B[l]^T, by warps of 32 columns, whose order in the MMAs is
// such that a lane ends with eight neighbouring ones.  B's and base's share are fetched into
// L2 while x A^T is computed.
//
// h is made in fp32: an MMA takes 16-bit operands, so h is split into a sum of two or
// three of them, each the rounding of what the ones before leave (a rounding of p bits
// leaves at most 2^-p, and what it leaves begins one bit lower).  bf16: two leave an error of
// 2^-17 (16-bit output, whose rounding is 2^-8: 0.2 % of 16384 x 4096 outputs fall to the other side of
// one than with all of h, and the error against 64 bits is the same), three one of 2^-26 (fp32
// output; three for both would cost the tiles their second CTA on an SM).  fp16:
// two leave 2^-23, a step of fp32; h is first scaled by a power of two per row so that its
// largest element is near 2^14, because fp16's range is narrow.
//
// Latency bounds it (the SMs hold 16 warps each by registers): one row of rank 16, 4096x4096, 6.5
// us; 64 rows of 32 adapters of rank 64 12.5 us, of which the weights' 24 MB are 3.6; 257 rows of
// rank 24, 1000x1537 in fp16, 11.5 us (9.0 with 1536 columns, on 16-byte boundaries); 2048 rows of 16
// adapters of rank 32, 1024x8192 into fp32, 40.6 us, 3.5 TB/s.
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
constexpr int kRows = 16;           // of an item
constexpr int kMaxCluster = 16;     // CTAs (more than 8 where that is allowed, see launch_few)

// Eight elements of a row of `of` at k, zeros past its end (row null: zeros).
__device__ __forceinline__ uint4 load8(const Buffer &of, const uint16_t *row, int k, int K, bool vec)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!row || k >= K)
        return v;
    if (!of.holds(row + k, 2 * (vec ? 8 : min(8, K - k))))
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

// Shared memory of floats: the warps' partial sums (later h's parts as MMA operands), every
// CTA's partial h, h itself.
template <int TERMS> struct FewSmem {
    static constexpr int kPitch = kChunk + 4;           // of a row of partial sums: spreads banks
    static __host__ __device__ int padded(int r_pad) { return (r_pad + 31) / 32 * 32; }
    static __host__ __device__ size_t part(int r_pad)
    {
        const size_t sums = sizeof(float) * kWarps * kRows * kPitch;
        const size_t frags = sizeof(uint4) * 32 * (padded(r_pad) / 16) * TERMS;
        return sums > frags ? sums : frags;
    }
    static __host__ __device__ size_t received(int r_pad, int cluster) { return sizeof(float) * r_pad * kRows * cluster; }
    static __host__ __device__ size_t bytes(int r_pad, int cluster)
    {
        return part(r_pad) + received(r_pad, cluster) + sizeof(float) * padded(r_pad) * kRows;
    }
};

// Starts fetching into L2 (16-byte boundaries; of long ranges the first megabyte).
__device__ __forceinline__ void prefetch_l2(const Buffer &of, const void *p, size_t bytes)
{
    const uint32_t n = static_cast<uint32_t>(min(bytes, static_cast<size_t>(1) << 20));
    if (of.holds(p, bytes))
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}

// Eight neighbouring elements of a row of base or out, as fp32.
template <int OUT> struct Eight {
    uint4 w[OUT == W8A8_OUT_FP32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, long long i)
    {
        const uint4 *const p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + i * (OUT == W8A8_OUT_FP32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(w) / 16); ++j)
            w[j] = p[j];
    }
    __device__ __forceinline__ float at(int i) const
    {
        const uint32_t *const u = reinterpret_cast<const uint32_t *>(w);
        if constexpr (OUT == W8A8_OUT_FP32)
            return __uint_as_float(u[i]);
        else if constexpr (OUT == W8A8_OUT_BF16)
            return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
        else
            return __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? u[i >> 1] >> 16 : u[i >> 1])));
    }
    __device__ __forceinline__ void store(void *out, long long i, const float (&v)[8])
    {
        uint32_t u[sizeof(w) / 4];
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(w) / 4); ++j)
            u[j] = OUT == W8A8_OUT_FP32   ? __float_as_uint(v[j])
                   : OUT == W8A8_OUT_BF16 ? pack_bf16x2(v[2 * j % 8], v[(2 * j + 1) % 8])
                                          : pack_f16x2(v[2 * j % 8], v[(2 * j + 1) % 8]);
        uint4 *const p = reinterpret_cast<uint4 *>(static_cast<char *>(out) + i * (OUT == W8A8_OUT_FP32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(w) / 16); ++j)
            p[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
    }
};

template <bool BF16, int OUT>
__global__ void __launch_bounds__(kThreads, 2) k_adapter_few(const AdapterParams p)
{
    constexpr int kTerms = BF16 && OUT == W8A8_OUT_FP32 ? 3 : 2;
    using S = FewSmem<kTerms>;
    constexpr int kElement = OUT == W8A8_OUT_FP32 ? 4 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int scratch[16];
    __shared__ int rows[kRows];
    __shared__ float factor[kRows];         // what a row's sums are multiplied by (fp16)
    uint32_t ctas, cluster;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
    const uint32_t me = cluster_ctarank();
    float *const part = reinterpret_cast<float *>(smem);
    float *const received = reinterpret_cast<float *>(smem + S::part(p.r_pad));
    float *const h = received + p.r_pad * kRows * ctas;
    const int r32 = S::padded(p.r_pad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const Item item = find_item<kThreads>(p, static_cast<int>(cluster), kRows, p.out == p.base ? p.L : p.L + 1, scratch);
    if (item.rows == 0 || !in_bounds(item.first >= 0 && item.first + item.rows <= p.T && item.adapter <= p.L, p.status,
                                     SITE_BOUNDS_A))
        return;                             // the whole cluster
    auto row_at = [&](int i) { return i < item.rows ? row_in_place(p, item.first + i) : -1; };
    const Buffer x_all = x_of(p), a_all = a_of(p), b_all = b_of(p), base_all = base_of(p, kElement), out_all = out_of(p, kElement);
    const int n_blocks = (p.N + 31) / 32;
    const int block_lo = static_cast<int>(static_cast<long long>(n_blocks) * me / ctas);
    const int block_hi = static_cast<int>(static_cast<long long>(n_blocks) * (me + 1) / ctas);
    const int n_lo = block_lo * 32, n_hi = min(block_hi * 32, p.N);
    // (the last warp has the least to do at first)
    const int slot = static_cast<int>(threadIdx.x) - (kThreads - 32);
    if (slot >= 0 && slot < kRows)
        rows[slot] = row_at(slot);
    if (item.adapter == p.L) {
        __syncthreads();
        if (p.vec_n)
            copy_rows<uint4, kThreads>(p, rows, item.rows, n_lo, n_hi, kElement);
        else if constexpr (kElement == 4)
            copy_rows<uint32_t, kThreads>(p, rows, item.rows, n_lo, n_hi, kElement);
        else
            copy_rows<uint16_t, kThreads>(p, rows, item.rows, n_lo, n_hi, kElement);
        return;
    }
    __syncwarp();
    if (ctas > 1)                           // peers write here once every CTA has started
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const uint16_t *const A = p.A + static_cast<long long>(item.adapter) * p.r * p.K;
    const uint16_t *const B = p.B + static_cast<long long>(item.adapter) * p.N * p.r;
    if (slot == kRows && p.vec_r && n_hi > n_lo && p.r)
        prefetch_l2(b_all, B + static_cast<long long>(n_lo) * p.r, static_cast<size_t>(n_hi - n_lo) * p.r * 2);
    if (slot >= 0 && slot < kRows && p.vec_n && n_hi > n_lo)
        if (const int row = rows[slot]; row >= 0)
            prefetch_l2(base_all, static_cast<const char *>(p.base) + (row * p.ld_base + n_lo) * kElement,
                        static_cast<size_t>(n_hi - n_lo) * kElement);
    __syncwarp();

    // h, this CTA's share of K
    const int blocks = (p.K + 63) / 64;
    const int lo = static_cast<int>(static_cast<long long>(blocks) * me / ctas);
    const int hi = static_cast<int>(static_cast<long long>(blocks) * (me + 1) / ctas);
    const uint16_t *token[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = row_at(8 * i + g);
        token[i] = row >= 0 ? p.x + row * p.ld_x : nullptr;
    }
    for (int r0 = 0; r0 < p.r_pad; r0 += kChunk) {
        float acc[8][4] = {};
        const int tiles = min(8, (p.r_pad - r0) / 8);
        for (int b = lo + warp; b < hi; b += kWarps) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = b * 64 + 32 * s + 8 * c;
                uint4 a[8], xv[2];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = r0 + 8 * j + g;
                    if (j < tiles)
                        a[j] = load8(a_all, r < p.r ? A + static_cast<long long>(r) * p.K : nullptr, k, p.K, p.vec_k);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    xv[i] = load8(x_all, token[i], k, p.K, p.vec_k);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < tiles) {
                        mma<BF16>(acc[j], xv[0].x, xv[1].x, xv[0].y, xv[1].y, a[j].x, a[j].y);
                        mma<BF16>(acc[j], xv[0].z, xv[1].z, xv[0].w, xv[1].w, a[j].z, a[j].w);
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (j < tiles)
                    *reinterpret_cast<float2 *>(part + ((warp * kRows + g + 8 * i) * S::kPitch + 8 * j + 2 * c)) =
                        make_float2(acc[j][2 * i], acc[j][2 * i + 1]);
        __syncthreads();
        if (ctas > 1 && r0 == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        for (int i = threadIdx.x; i < item.rows * 2 * tiles; i += kThreads) {
            const int row = i / (2 * tiles), r = (i - row * 2 * tiles) * 4;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 v = *reinterpret_cast<const float4 *>(part + (w * kRows + row) * S::kPitch + r);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const uint32_t at = smem_addr(received + (me * kRows + row) * p.r_pad + r0 + r);
            for (uint32_t q = 0; q < ctas; ++q)
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_map(at, q)), "f"(sum.x),
                             "f"(sum.y), "f"(sum.z), "f"(sum.w)
                             : "memory");
        }
        __syncthreads();
    }
    if (ctas > 1) {
        if (p.r_pad == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        cluster_sync();
    }
    const float scale = scale_of(p, item.adapter);
    for (int i = threadIdx.x; i < item.rows * (r32 / 4); i += kThreads) {
        const int row = i / (r32 / 4), r = (i - row * (r32 / 4)) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < p.r_pad)
#pragma unroll 8
            for (uint32_t q = 0; q < ctas; ++q) {
                const float4 v = *reinterpret_cast<const float4 *>(received + (q * kRows + row) * p.r_pad + r);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
        *reinterpret_cast<float4 *>(h + row * r32 + r) =
            make_float4(sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale);
    }
    __syncthreads();
    if constexpr (!BF16) {
        for (int t = warp; t < item.rows; t += kWarps) {
            float top = 0.f;
            for (int i = lane; i < p.r_pad; i += 32)
                top = fmaxf(top, fabsf(h[t * r32 + i]));
#pragma unroll
            for (int d = 16; d; d /= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            float shrink, back;
            power_of(top, &shrink, &back);
            for (int i = lane; i < p.r_pad; i += 32)
                h[t * r32 + i] *= shrink;
            if (lane == 0)
                factor[t] = back;
        }
        __syncthreads();
    }
    // h's parts as A operands: for step s of 16 columns lane (g, c) has the elements
    // 32 (s / 2) + 8 c + 4 (s % 2) .. + 3 of rows g and g + 8 (what lies past the item's
    // rows stays in its own rows of the product)
    const int steps = r32 / 16;
    uint4 *const frags = reinterpret_cast<uint4 *>(part);
    for (int i = threadIdx.x; i < steps * 32; i += kThreads) {
        const int ln = i & 31, s = i >> 5;
        const int k = 32 * (s / 2) + 8 * (ln & 3) + 4 * (s & 1), row = ln >> 2;
        const float4 u = *reinterpret_cast<const float4 *>(h + row * r32 + k);
        const float4 w = *reinterpret_cast<const float4 *>(h + (row + 8) * r32 + k);
        float a[4] = {u.x, u.y, u.z, u.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < kTerms; ++q) {
            uint32_t x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = take_part<BF16>(a[j]);
                y[j] = take_part<BF16>(b[j]);
            }
            frags[(s * kTerms + q) * 32 + ln] =
                make_uint4(x[1] << 16 | x[0], y[1] << 16 | y[0], x[3] << 16 | x[2], y[3] << 16 | y[2]);
        }
    }
    __syncthreads();
    // out, this CTA's share of N: in tile j of 8, the MMA's column i is column
    // 8 (i / 2) + 2 j + i % 2 of the block (a lane's 2 c and 2 c + 1 of four tiles are 8 c ..
    // 8 c + 7), or 8 j + i where rows of base or out do not lie on 16 bytes
    for (int block = block_lo + warp; block < block_hi; block += kWarps) {
        const int n0 = block * 32;
        int to[2];
        Eight<OUT> old[2];
        const bool whole = p.vec_n && n0 + 8 * c < p.N;         // (vec_n: eight columns are in or out of N)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            to[i] = rows[8 * i + g];
            if (whole && to[i] >= 0 &&
                base_all.holds(static_cast<const char *>(p.base) + (to[i] * p.ld_base + n0 + 8 * c) * kElement, 8 * kElement))
                old[i].load(p.base, to[i] * p.ld_base + n0 + 8 * c);
        }
        const uint16_t *b_row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + (p.vec_n ? 8 * (g >> 1) + 2 * j + (g & 1) : 8 * j + g);
            b_row[j] = n < p.N ? B + static_cast<long long>(n) * p.r : nullptr;
        }
        float acc[4][4] = {};
#pragma unroll 2
        for (int s = 0; s < steps; s += 2) {
            uint4 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = load8(b_all, b_row[j], 16 * s + 8 * c, p.r, p.vec_r);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int q = 0; q < kTerms; ++q) {
                    const uint4 f = frags[((s + half) * kTerms + q) * 32 + lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma<BF16>(acc[j], f.x, f.y, f.z, f.w, half ? b[j].z : b[j].x, half ? b[j].w : b[j].y);
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (to[i] < 0)
                continue;
            const float f = BF16 ? 1.f : factor[8 * i + g];
            const long long at_out = to[i] * p.ld_out + n0, at_base = to[i] * p.ld_base + n0;
            if (p.vec_n) {
                if (!whole)
                    continue;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = fmaf(acc[j >> 1][2 * i + (j & 1)], f, old[i].at(j));
                if (out_all.holds(static_cast<const char *>(p.out) + (at_out + 8 * c) * kElement, 8 * kElement))
                    old[i].store(p.out, at_out + 8 * c, v);
            } else {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int n = 8 * (j >> 1) + 2 * c + (j & 1);
                    const bool in = n0 + n < p.N &&
                                    base_all.holds(static_cast<const char *>(p.base) + (at_base + n) * kElement, kElement);
                    v[j] = in ? load_out<OUT>(p.base, at_base + n) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int n = 8 * (j >> 1) + 2 * c + (j & 1);
                    if (n0 + n < p.N && out_all.holds(static_cast<const char *>(p.out) + (at_out + n) * kElement, kElement))
                        store_out<OUT>(p.out, at_out + n, fmaf(acc[j >> 1][2 * i + (j & 1)], f, v[j]));
                }
            }
        }
    }
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool BF16, int OUT>
cudaError_t launch_few(const AdapterParams &p, long long items, const DeviceView &dev, cudaStream_t stream)
{
    constexpr int kTerms = BF16 && OUT == W8A8_OUT_FP32 ? 3 : 2;
    using S = FewSmem<kTerms>;
    constexpr size_t kRoom = 200 * 1024;
    auto kernel = k_adapter_few<BF16, OUT>;
    // As many CTAs share an item as fill the SMs twice, 16 as fill them once, with 128
    // columns of K for each (one row, rank 16, 4096x4096: 4 CTAs 8.9 us, 8 6.7, 16 6.2; 64
    // rows of 32 adapters of rank 64: 2 23 us, 4 14.7, 8 11.4).
    int cluster = 1;
    while (cluster < kMaxCluster && items * cluster * 2 <= (cluster < 8 ? 2ll : 1ll) * dev.sm_count &&
           cluster * 2 * 128 <= std::max(p.K, p.N) && S::bytes(p.r_pad, cluster * 2) <= kRoom)
        cluster *= 2;
    const size_t smem = S::bytes(p.r_pad, cluster);
    static volatile int flags[kMaxDeviceFlags] = {};
    if (const cudaError_t e = allow_smem(kernel, kRoom, flags, true); e != cudaSuccess)
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
    return launch_few<BF16, OUT>(p, most_items(p.T, groups, kRows), dev, s);
}

// Whether a problem's sizes are for the tiles of 128 rows (adapter_tile.cu), which take two
// launches and some 10 to 20 us for them, then stream: where there is much to read, and many rows
// to an adapter.  The clusters of 16 rows take a time that grows with T (K + N + 640) and with r,
// the tiles one that hardly depends on r.  Clusters / tiles in us, T of L adapters, KxN, bf16 into
// bf16:
//   r 16   1600 of 24 1024x1024 9.4 / 13.6, 2048 of 4 4096x4096 21.1 / 16.5, 4096 of 8 1024x1024
//          13.5 / 12.4, 16384 256x256 23 / 11.6; 1536 256x4096 into fp32 20.7 / 19.3
//   r 32   2200 of 8 4096x4096 24.0 / 35.3, 4200 of 8 2048x2048 22.9 / 36.6, into fp32 29.0 / 46.2
//   r 64   4096 of 8 2048x2048 31.3 / 36.7, 8192 of 8 1024x1024 35.5 / 27.2, 16384 512x512 42.7 / 22.2;
//          2048 of 16 4096x4096 33.2 / 38.8, into fp32 40.6 / 51.5
//   r 128  3200 of 8 4096x4096 103 / 68, 16384 512x512 68 / 36; 4096 of 16 1024x8192 into fp32 138 / 148
// One line for every output type and every shape of the widths: over 760 problems of the range that it
// decides (1 to 64 adapters, K and N 64 to 8192, r 8 to 128, runs of 1 to 2000 rows; 304 of them into fp32,
// 456 into bf16) it takes 4.8 % longer than the faster form of each on average, more than 10 % longer
// for 121, 1.9 times at worst.  It is too high for many rows of narrow layers (r 64: 12000 of 4 512x512
// 32.3 / 21.2, 7400 of 8 1024x1024 35.3 / 26.7) and for a narrow K beside a wide N (r 32, 2048 of 16
// 1024x8192 27.5 / 24.2, into fp32 39.6 / 38.8), too low for rank 8 and 16 (4500 of 4 512x512 9.1 / 13.6).
bool many_rows(const AdapterParams &p) { return p.L > 0 && p.T >= 1536 && p.T / 64 >= p.L && p.r >= 8 && p.K >= 64; }
bool tiled(const AdapterParams &p)
{
    const long long work = static_cast<long long>(p.T) * (static_cast<long long>(p.K) + p.N + 640);
    return many_rows(p) && work >= (p.r <= 16 ? 6500000 : p.r <= 64 ? 21000000 : 25000000);
}

// Asked for wherever some N makes tiles of the rows.
size_t workspace_bytes(const AdapterParams &p, int variant)
{
    const bool tiles = variant == W8A8_VARIANT_TILED || (variant == W8A8_VARIANT_AUTO && many_rows(p));
    return tiles ? sizeof(float) * tile_splits(p) * p.T * p.r_pad : 0;
}

}  // namespace
}  // namespace w8a8

extern "C" size_t w8a8_adapter_workspace_size(int64_t T, int64_t L, int64_t r, int64_t K, int variant)
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
    return workspace_bytes(p, variant);
}

extern "C" w8a8_status w8a8_adapter_matmul(const void *x_dev, w8a8_in_dtype dtype, int64_t ld_x, const void *A_dev,
                                           const void *B_dev, const int32_t *order_dev, const int32_t *offsets_dev,
                                           const float *scales_dev, const void *base_dev, int64_t ld_base,
                                           void *out_dev, w8a8_out_dtype out_dtype, int64_t ld_out, int64_t T,
                                           int64_t L, int64_t r, int64_t K, int64_t N, int variant,
                                           void *workspace_dev, size_t workspace_bytes, w8a8_stream_t stream)
{
    using namespace w8a8;
    if (T < 0 || L < 0 || r < 0 || K < 0 || N < 0)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size");
    if (dtype < W8A8_IN_BF16 || dtype > W8A8_IN_FP32 || out_dtype < W8A8_OUT_BF16 || out_dtype > W8A8_OUT_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown dtype");
    if (variant < W8A8_VARIANT_AUTO || variant > W8A8_VARIANT_GENERIC)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown variant");
    if (variant != W8A8_VARIANT_AUTO && variant != W8A8_VARIANT_SMALLM && variant != W8A8_VARIANT_TILED)
        return record_error(W8A8_ERR_UNSUPPORTED, "variant must be AUTO, SMALLM or TILED");
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
    // (B does not depend on K, and is read where x and A have no columns too)
    if (L > 0 && r > 0 && (!B_dev || (K > 0 && (!x_dev || !A_dev))))
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
    p.vec_r = r % 8 == 0 && on(B_dev, 16);
    const int each = 16 / ob;
    p.vec_n = N % 8 == 0 && ld_base % each == 0 && ld_out % each == 0 && on(base_dev, 16) && on(out_dev, 16);
    const bool fits = L > 0 && tile_takes(p);
    if (variant == W8A8_VARIANT_TILED && !fits)
        return record_error(W8A8_ERR_UNSUPPORTED, "TILED needs an adapter, r % 8 == 0 from 8 to 128, K % 8 == 0 from 64 on, "
                                                  "N % 8 == 0 and rows on 16-byte boundaries");
    const bool tiles = fits && (variant == W8A8_VARIANT_TILED || (variant == W8A8_VARIANT_AUTO && tiled(p)));
    if (const size_t need = fits ? w8a8::workspace_bytes(p, variant) : 0;
        need && (!workspace_dev || workspace_bytes < need || !on(workspace_dev, 16))) {
        char msg[160];
        snprintf(msg, sizeof(msg), "workspace of %zu bytes at %p: need %zu bytes, 16-byte aligned", workspace_bytes,
                 workspace_dev, need);
        return record_error(W8A8_ERR_WORKSPACE, msg);
    }
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    p.status = dev.status;
    p.wait_limit = dev.wait_limit;
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
