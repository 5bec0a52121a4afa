// The weighted sum of the experts' rows back to tokens:
//
//   out[t] = sum_j weights[t, j] * Y[rows[t, j]] + add[t]
//
// with Y's rows in the experts' order and rows as the router gives them; a row outside
// [0, M) (-1: no expert) is left out.  Sums in fp32 in the order of j, then add, one rounding.
//
// HBM-bound: every row of Y is read once, wherever it lies.  A thread holds eight
// neighbouring columns of one token and has up to eight rows' loads in flight (16384 tokens of 8
// rows of 4096 in bf16 and an addend 208 us, 6.5 TB/s; one token 1.9 us).
#include <algorithm>
#include <cstdio>

#include "../../include/w8a8_block_fp8.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace w8a8 {
w8a8_status record_error(w8a8_status st, const char *message);

namespace {

struct CombineParams {
    const void *Y;              // [M, ld_y]
    const int *rows;            // [T, k]
    const float *weights;       // [T, k]
    const void *add;            // [T, ld_add] of out's type, or null
    void *out;                  // [T, ld_out]
    long long M, ld_y, ld_add, ld_out;
    int k, D;
    int chunks;                 // CTAs of a token
};

constexpr int kThreads = 128;
constexpr int kFlight = 8;
constexpr int kVec = 8;             // columns a thread, on 16-byte boundaries

template <int KIND> struct Raw {
    static constexpr int kPieces = KIND == W8A8_IN_FP32 ? 2 : 1;
    uint32_t w[4 * kPieces];
    __device__ __forceinline__ void load(const void *base, long long element)
    {
        const uint4 *const p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + element * 2 * kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            *reinterpret_cast<uint4 *>(&w[4 * i]) = p[i];
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (KIND == W8A8_IN_FP32)
            return __uint_as_float(w[i]);
        else if constexpr (KIND == W8A8_IN_BF16)
            return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else
            return __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1])));
    }
    __device__ __forceinline__ void set(const float (&v)[kVec])
    {
#pragma unroll
        for (int i = 0; i < 4 * kPieces; ++i)
            w[i] = KIND == W8A8_IN_FP32   ? __float_as_uint(v[i])
                   : KIND == W8A8_IN_BF16 ? pack_bf16x2(v[2 * i % kVec], v[(2 * i + 1) % kVec])
                                          : pack_f16x2(v[2 * i % kVec], v[(2 * i + 1) % kVec]);
    }
    __device__ __forceinline__ void store(void *base, long long element) const
    {
        uint4 *const p = reinterpret_cast<uint4 *>(static_cast<char *>(base) + element * 2 * kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            p[i] = *reinterpret_cast<const uint4 *>(&w[4 * i]);
    }
};

template <int KIND, int OUT> __global__ void __launch_bounds__(kThreads) k_combine(const CombineParams p)
{
    const long long t = blockIdx.x / p.chunks;
    const int col = (static_cast<int>(blockIdx.x % p.chunks) * kThreads + threadIdx.x) * kVec;
    grid_dependency_wait();
    grid_launch_dependents();
    if (col >= p.D)
        return;
    float acc[kVec] = {};
    Raw<OUT> plus;
    if (p.add)
        plus.load(p.add, t * p.ld_add + col);
    const int *rows = p.rows + t * p.k;
    const float *weights = p.weights + t * p.k;
    for (int j0 = 0; j0 < p.k; j0 += kFlight) {
        Raw<KIND> y[kFlight];
        float w[kFlight];
        bool in[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const long long row = j0 + j < p.k ? rows[j0 + j] : -1;
            in[j] = row >= 0 && row < p.M;
            w[j] = in[j] ? weights[j0 + j] : 0.f;
            if (in[j])
                y[j].load(p.Y, row * p.ld_y + col);
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (in[j]) {
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    acc[i] = fmaf(w[j], y[j].at(i), acc[i]);
            }
    }
    if (p.add) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            acc[i] += plus.at(i);
    }
    Raw<OUT> o;
    o.set(acc);
    o.store(p.out, t * p.ld_out + col);
}

// Rows off 16-byte boundaries.  A thread takes the columns of 16 bytes of a row; of each row
// it loads the two aligned pieces that hold them and shifts them into place (the same shift for
// the whole row), without a branch before the loads (but where a piece would not lie wholly in
// Y).  Results go through shared memory, so
// that neighbouring threads store neighbouring elements: 1013 tokens of 6 rows of 1537 in fp16
// 10.7 us (an element at a time 15.4).  What remains over the bytes' 3.7 us is the picking of
// elements: the same rows of 1536 columns, on boundaries, take 5.1.
constexpr int kShiftThreads = 64, kShiftFlight = 4;         // as many CTAs on an SM as registers allow

template <int KIND> struct Shifted {        // of bf16 or fp16
    static constexpr int kBytes = 2, kEach = 8;
    uint4 w0, w1;
    // acc += weight * the elements from p on (shift: p's place in its piece)
    __device__ __forceinline__ void add_to(float (&acc)[kEach], float weight, int shift) const
    {
        uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 6; ++i)
            w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i)
            w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = __funnelshift_r(w[i], w[i + 1], 8 * (shift & 2));
            float lo, hi;
            if constexpr (KIND == W8A8_IN_BF16) {
                lo = __uint_as_float(u << 16), hi = __uint_as_float(u & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
                lo = f.x, hi = f.y;
            }
            acc[2 * i] = fmaf(weight, lo, acc[2 * i]);
            acc[2 * i + 1] = fmaf(weight, hi, acc[2 * i + 1]);
        }
    }
};

template <int OUT> __device__ __forceinline__ float element(const void *p, long long i)
{
    if constexpr (OUT == W8A8_IN_FP32)
        return static_cast<const float *>(p)[i];
    else if constexpr (OUT == W8A8_IN_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else
        return __half2float(static_cast<const __half *>(p)[i]);
}

template <int KIND, int OUT> __global__ void __launch_bounds__(kShiftThreads, 14) k_combine_shift(const CombineParams p)
{
    using In = Shifted<KIND>;
    constexpr int kEach = In::kEach;
    __shared__ float sums[kShiftThreads * kEach];
    const long long t = blockIdx.x / p.chunks;
    // an even share of the row's pieces
    const int pieces = (p.D + kEach - 1) / kEach, part = static_cast<int>(blockIdx.x % p.chunks);
    const int first = static_cast<int>(static_cast<long long>(pieces) * part / p.chunks) * kEach;
    const int last = min(p.D, static_cast<int>(static_cast<long long>(pieces) * (part + 1) / p.chunks) * kEach);
    const int col = first + static_cast<int>(threadIdx.x) * kEach;
    grid_dependency_wait();
    grid_launch_dependents();
    // what is added, as it is stored: neighbouring elements by neighbouring threads
    float plus[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int c = first + static_cast<int>(threadIdx.x) + i * kShiftThreads;
        plus[i] = p.add && c < last ? element<OUT>(p.add, t * p.ld_add + c) : 0.f;
    }
    const char *const begin = static_cast<const char *>(p.Y);
    const char *const end = begin + ((p.M - 1) * p.ld_y + p.D) * In::kBytes;
    const int need = min(kEach, last - col) * In::kBytes;
    const int *rows = p.rows + t * p.k;
    const float *weights = p.weights + t * p.k;
    float acc[kEach] = {};
    if (need > 0)
        for (int j0 = 0; j0 < p.k; j0 += kShiftFlight) {
            const char *at[kShiftFlight];
            float w[kShiftFlight];
            bool edge = false;          // a piece is not wholly within Y
#pragma unroll
            for (int j = 0; j < kShiftFlight; ++j) {
                const long long row = j0 + j < p.k ? rows[j0 + j] : -1;
                const bool in = row >= 0 && row < p.M;
                at[j] = in ? begin + (row * p.ld_y + col) * In::kBytes : nullptr;
                w[j] = in ? weights[j0 + j] : 0.f;
                const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(at[j]) & 15);
                edge = edge || (in && (at[j] - shift < begin || at[j] - shift + (shift + need > 16 ? 32 : 16) > end));
            }
            if (!edge) {
                In y[kShiftFlight];
#pragma unroll
                for (int j = 0; j < kShiftFlight; ++j) {
                    y[j].w0 = y[j].w1 = make_uint4(0, 0, 0, 0);
                    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(at[j]) & 15);
                    const uint4 *const piece = reinterpret_cast<const uint4 *>(at[j] - shift);
                    if (at[j])
                        y[j].w0 = piece[0];
                    if (at[j] && shift + need > 16)
                        y[j].w1 = piece[1];
                }
#pragma unroll
                for (int j = 0; j < kShiftFlight; ++j)
                    if (at[j])
                        y[j].add_to(acc, w[j], static_cast<int>(reinterpret_cast<uintptr_t>(at[j]) & 15));
            } else {
#pragma unroll 1
                for (int j = j0; j < min(p.k, j0 + kShiftFlight); ++j) {
                    const long long row = rows[j];
                    if (row < 0 || row >= p.M)
                        continue;
                    const float weight = weights[j];
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (col + i < p.D)
                            acc[i] = fmaf(weight, element<KIND>(p.Y, row * p.ld_y + col + i), acc[i]);
                }
            }
        }
    // [element of a thread][thread]: no two lanes of a warp in one bank
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        sums[i * kShiftThreads + threadIdx.x] = acc[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int n = static_cast<int>(threadIdx.x) + i * kShiftThreads;
        if (first + n >= last)
            continue;
        const float v = sums[(n % kEach) * kShiftThreads + n / kEach] + plus[i];
        const long long at = t * p.ld_out + first + n;
        if constexpr (OUT == W8A8_IN_FP32)
            static_cast<float *>(p.out)[at] = v;
        else if constexpr (OUT == W8A8_IN_BF16)
            static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
        else
            static_cast<__half *>(p.out)[at] = __float2half_rn(v);
    }
}

// fp32 rows off 16-byte boundaries: whole elements, eight columns a thread, 64 apart, so that the
// rows' places and weights are loaded once for eight: 1013 tokens of 6 rows of 1537 10.8 us (one
// column a thread 23, shifted as above 17.7).
__global__ void __launch_bounds__(kShiftThreads, 14) k_combine_columns(const CombineParams p)
{
    constexpr int kEach = 8;
    const long long t = blockIdx.x / p.chunks;
    const int first = static_cast<int>(static_cast<long long>(p.D) * (blockIdx.x % p.chunks) / p.chunks);
    const int last = static_cast<int>(static_cast<long long>(p.D) * (blockIdx.x % p.chunks + 1) / p.chunks);
    const int col = first + static_cast<int>(threadIdx.x);
    grid_dependency_wait();
    grid_launch_dependents();
    const float *const Y = static_cast<const float *>(p.Y), *const add = static_cast<const float *>(p.add);
    const int *rows = p.rows + t * p.k;
    const float *weights = p.weights + t * p.k;
    float acc[kEach] = {}, plus[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        plus[i] = add && col + i * kShiftThreads < last ? add[t * p.ld_add + col + i * kShiftThreads] : 0.f;
    for (int j0 = 0; j0 < p.k; j0 += kShiftFlight) {
        float y[kShiftFlight][kEach], w[kShiftFlight];
        bool in[kShiftFlight];
#pragma unroll
        for (int j = 0; j < kShiftFlight; ++j) {
            const long long row = j0 + j < p.k ? rows[j0 + j] : -1;
            in[j] = row >= 0 && row < p.M;
            w[j] = in[j] ? weights[j0 + j] : 0.f;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (in[j] && col + i * kShiftThreads < last)
                    y[j][i] = Y[row * p.ld_y + col + i * kShiftThreads];
        }
#pragma unroll
        for (int j = 0; j < kShiftFlight; ++j)
            if (in[j]) {
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    acc[i] = fmaf(w[j], y[j][i], acc[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (col + i * kShiftThreads < last)
            static_cast<float *>(p.out)[t * p.ld_out + col + i * kShiftThreads] = acc[i] + plus[i];
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

cudaError_t launch_chunks(void (*kernel)(CombineParams), const CombineParams &p, long long T, int threads,
                          cudaStream_t stream)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(T * p.chunks), 1, 1);
    lc.blockDim = dim3(threads, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

template <int KIND, int OUT> cudaError_t launch(const CombineParams &p, long long T, cudaStream_t stream)
{
    // Eight columns a thread where every row of every tensor allows it.
    constexpr int kY = KIND == W8A8_IN_FP32 ? 4 : 2, kO = OUT == W8A8_IN_FP32 ? 4 : 2;
    if (p.D % 8 == 0 && on(p.Y, 16) && on(p.add, 16) && on(p.out, 16) && p.ld_y * kY % 16 == 0 &&
        (!p.add || p.ld_add * kO % 16 == 0) && p.ld_out * kO % 16 == 0) {
        CombineParams q = p;
        q.chunks = (p.D + kThreads * kVec - 1) / (kThreads * kVec);
        return launch_chunks(k_combine<KIND, OUT>, q, T, kThreads, stream);
    }
    CombineParams q = p;
    q.chunks = (p.D + kShiftThreads * 8 - 1) / (kShiftThreads * 8);
    if constexpr (KIND == W8A8_IN_FP32)
        return launch_chunks(k_combine_columns, q, T, kShiftThreads, stream);
    else
        return launch_chunks(k_combine_shift<KIND, OUT>, q, T, kShiftThreads, stream);
}

}  // namespace
}  // namespace w8a8

extern "C" w8a8_status w8a8_combine_experts(const void *Y_dev, w8a8_in_dtype y_dtype, int64_t ld_y, int64_t M,
                                            const int32_t *rows_dev, const float *weights_dev, const void *add_dev,
                                            int64_t ld_add, void *out_dev, w8a8_in_dtype out_dtype, int64_t ld_out,
                                            int64_t T, int64_t k, int64_t D, w8a8_stream_t stream)
{
    using namespace w8a8;
    if (T < 0 || k < 0 || D < 0 || M < 0)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size");
    if (y_dtype < W8A8_IN_BF16 || y_dtype > W8A8_IN_FP32 || out_dtype < W8A8_IN_BF16 || out_dtype > W8A8_IN_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown dtype");
    if (out_dtype != y_dtype && out_dtype != W8A8_IN_FP32)
        return record_error(W8A8_ERR_UNSUPPORTED, "out must have Y's type or fp32");
    ld_y = ld_y ? ld_y : D;
    ld_add = ld_add ? ld_add : D;
    ld_out = ld_out ? ld_out : D;
    if (ld_y < D || ld_add < D || ld_out < D)
        return record_error(W8A8_ERR_INVALID_ARG, "a row stride is shorter than its row");
    if (T == 0 || D == 0)
        return W8A8_OK;
    if (!out_dev || (k > 0 && (!rows_dev || !weights_dev)) || (k > 0 && M > 0 && !Y_dev))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (D > (1ll << 24) || k > (1ll << 20) || T > ((1ll << 31) - 1) / ((D + kThreads - 1) / kThreads))
        return record_error(W8A8_ERR_UNSUPPORTED, "D above 2^24, k above 2^20, or T * ceil(D / 128) of 2^31 or more");
    const int yb = y_dtype == W8A8_IN_FP32 ? 4 : 2, ob = out_dtype == W8A8_IN_FP32 ? 4 : 2;
    if (!on(Y_dev, yb) || !on(rows_dev, 4) || !on(weights_dev, 4) || !on(add_dev, ob) || !on(out_dev, ob))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    CombineParams p = {};
    p.Y = Y_dev;
    p.rows = rows_dev;
    p.weights = weights_dev;
    p.add = add_dev;
    p.out = out_dev;
    p.M = M;
    p.ld_y = ld_y;
    p.ld_add = ld_add;
    p.ld_out = ld_out;
    p.k = static_cast<int>(k);
    p.D = static_cast<int>(D);
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (y_dtype == W8A8_IN_FP32)
        e = launch<W8A8_IN_FP32, W8A8_IN_FP32>(p, T, s);
    else if (y_dtype == W8A8_IN_BF16)
        e = out_dtype == W8A8_IN_FP32 ? launch<W8A8_IN_BF16, W8A8_IN_FP32>(p, T, s)
                                      : launch<W8A8_IN_BF16, W8A8_IN_BF16>(p, T, s);
    else
        e = out_dtype == W8A8_IN_FP32 ? launch<W8A8_IN_FP16, W8A8_IN_FP32>(p, T, s)
                                      : launch<W8A8_IN_FP16, W8A8_IN_FP16>(p, T, s);
    if (e == cudaSuccess)
        return W8A8_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "kernel launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return record_error(W8A8_ERR_CUDA, msg);
}
