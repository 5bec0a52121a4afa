// The weighted sum of the experts' rows back to tokens:
//
//   out[t] = add[t] + sum_j weights[t, j] * Y[rows[t, j]]
//
// with Y's rows in the experts' order and rows as the router gives them; a row outside
// [0, M) (-1: no expert) is left out.  Sums in fp32 in the order of j, one rounding.
//
// HBM-bound: every row of Y is read once, wherever it lies.  A thread holds VEC
// neighbouring columns of one token and has up to eight rows' loads in flight.
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

template <int KIND, int VEC> struct Raw {
    static constexpr int kBytes = (KIND == W8A8_IN_FP32 ? 4 : 2) * VEC;
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void *base, long long element)
    {
        const char *p = static_cast<const char *>(base) + element * (KIND == W8A8_IN_FP32 ? 4 : 2);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                *reinterpret_cast<uint4 *>(&w[4 * i]) = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
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
    __device__ __forceinline__ void set(const float (&v)[VEC])
    {
        if constexpr (KIND == W8A8_IN_FP32) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float hi = i + 1 < VEC ? v[i + 1] : 0.f;
                w[i >> 1] = KIND == W8A8_IN_BF16 ? pack_bf16x2(v[i], hi) : pack_f16x2(v[i], hi);
            }
        }
    }
    __device__ __forceinline__ void store(void *base, long long element) const
    {
        char *p = static_cast<char *>(base) + element * (KIND == W8A8_IN_FP32 ? 4 : 2);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = *reinterpret_cast<const uint4 *>(&w[4 * i]);
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(w);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
        }
    }
};

template <int KIND, int OUT, int VEC> __global__ void __launch_bounds__(kThreads) k_combine(const CombineParams p)
{
    const long long t = blockIdx.x / p.chunks;
    const int col = (static_cast<int>(blockIdx.x % p.chunks) * kThreads + threadIdx.x) * VEC;
    grid_dependency_wait();
    grid_launch_dependents();
    if (col >= p.D)
        return;
    float acc[VEC] = {};
    if (p.add) {
        Raw<OUT, VEC> a;
        a.load(p.add, t * p.ld_add + col);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            acc[i] = a.at(i);
    }
    const int *rows = p.rows + t * p.k;
    const float *weights = p.weights + t * p.k;
    for (int j0 = 0; j0 < p.k; j0 += kFlight) {
        Raw<KIND, VEC> y[kFlight];
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
                for (int i = 0; i < VEC; ++i)
                    acc[i] = fmaf(w[j], y[j].at(i), acc[i]);
            }
    }
    Raw<OUT, VEC> o;
    o.set(acc);
    o.store(p.out, t * p.ld_out + col);
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int KIND, int OUT, int VEC> cudaError_t launch(CombineParams p, long long T, cudaStream_t stream)
{
    p.chunks = (p.D + kThreads * VEC - 1) / (kThreads * VEC);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(T * p.chunks), 1, 1);
    lc.blockDim = dim3(kThreads, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, k_combine<KIND, OUT, VEC>, p);
}

template <int KIND, int OUT> cudaError_t launch(const CombineParams &p, long long T, cudaStream_t stream)
{
    // Eight, two or one column a thread, as every row of every tensor allows.
    constexpr int kY = KIND == W8A8_IN_FP32 ? 4 : 2, kO = OUT == W8A8_IN_FP32 ? 4 : 2;
    auto wide = [&](int vec) {
        const int y = std::min(16, kY * vec), o = std::min(16, kO * vec);
        return p.D % vec == 0 && on(p.Y, y) && on(p.add, o) && on(p.out, o) && p.ld_y * kY % y == 0 &&
               (!p.add || p.ld_add * kO % o == 0) && p.ld_out * kO % o == 0;
    };
    return wide(8)   ? launch<KIND, OUT, 8>(p, T, stream)
           : wide(2) ? launch<KIND, OUT, 2>(p, T, stream)
                     : launch<KIND, OUT, 1>(p, T, stream);
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
