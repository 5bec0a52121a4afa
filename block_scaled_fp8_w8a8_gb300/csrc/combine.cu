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
    int chunks;                 // pieces of a token's row
    long long pieces;           // of all
    long long T;
    unsigned *status;
};

// (debug-bounds build: whether an access lies in its buffer)
__device__ __forceinline__ bool is_choice(const CombineParams &p, long long t, int j)
{
    return in_bounds(t >= 0 && t < p.T && j >= 0 && j < p.k, p.status, SITE_BOUNDS_SCALES);
}
template <int KIND> __device__ __forceinline__ bool is_y(const CombineParams &p, const void *at, int bytes)
{
    return in_bounds(inside(at, bytes, p.Y, span(p.M, p.ld_y, p.D, KIND == W8A8_IN_FP32 ? 4 : 2)), p.status, SITE_BOUNDS_A);
}
template <int OUT> __device__ __forceinline__ bool is_add(const CombineParams &p, long long element, int count)
{
    constexpr int kBytes = OUT == W8A8_IN_FP32 ? 4 : 2;
    return in_bounds(inside(static_cast<const char *>(p.add) + element * kBytes, count * kBytes, p.add,
                            span(p.T, p.ld_add, p.D, kBytes)), p.status, SITE_BOUNDS_B);
}
template <int OUT> __device__ __forceinline__ bool is_out(const CombineParams &p, long long element, int count)
{
    constexpr int kBytes = OUT == W8A8_IN_FP32 ? 4 : 2;
    return in_bounds(inside(static_cast<const char *>(p.out) + element * kBytes, count * kBytes, p.out,
                            span(p.T, p.ld_out, p.D, kBytes)), p.status, SITE_BOUNDS_C);
}

constexpr int kThreads = 128;
constexpr int kVec = 8;                     // columns of a thread

// A CTA, or for narrow rows each of its warps, takes UNITS pieces of a token, of kVec columns a
// thread, one after the other whatever the tokens that they lie in: with few rows to a token as
// many loads are in flight as with many (4767 of one row of 1936 in bf16 and an addend 23.0 us by
// one piece, 14.4), and narrow rows leave few threads idle (15012 tokens of 6 rows of 160 in
// fp16 18.0 us by a CTA's pieces, 12.9 by a warp's).  Wide rows are a CTA's: tokens that
// come from the block's number alone cost less (16384 tokens of 8 rows of 4096 by a warp's pieces 222
// us, not 208).
struct Piece {
    long long t;
    int col;                    // the thread's or warp's first
    bool in;
};
template <bool WARPS, int UNITS> __device__ __forceinline__ void find_pieces(const CombineParams &p, Piece (&at)[UNITS])
{
    constexpr int kWarps = kThreads / 32, columns = (WARPS ? 32 : kThreads) * kVec;
    const long long first =
        UNITS * (WARPS ? static_cast<long long>(blockIdx.x) * kWarps + warp_uniform(warp_index()) : static_cast<long long>(blockIdx.x));
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const long long n = first + u;
        at[u].in = n < p.pieces;
        if (n >> 32) {
            at[u].t = n / p.chunks;
            at[u].col = static_cast<int>(n - at[u].t * p.chunks) * columns;
        } else {
            const uint32_t t = static_cast<uint32_t>(n) / static_cast<uint32_t>(p.chunks);
            at[u].t = t;
            at[u].col = static_cast<int>(static_cast<uint32_t>(n) - t * p.chunks) * columns;
        }
    }
}

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

template <int KIND, int OUT, bool WARPS, int UNITS>
__global__ void __launch_bounds__(kThreads) k_combine(const CombineParams p)
{
    constexpr int kDeep = 8 / UNITS, kBytes = KIND == W8A8_IN_FP32 ? 4 : 2;
    Piece at[UNITS];
    find_pieces<WARPS>(p, at);
    bool mine[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        at[u].col += static_cast<int>(WARPS ? lane_index() : threadIdx.x) * kVec;
        mine[u] = at[u].in && at[u].col < p.D;
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (UNITS == 1 && !mine[0])
        return;
    float acc[UNITS][kVec] = {};
    Raw<OUT> plus[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        if (p.add && mine[u] && is_add<OUT>(p, at[u].t * p.ld_add + at[u].col, kVec))
            plus[u].load(p.add, at[u].t * p.ld_add + at[u].col);
    for (int j0 = 0; j0 < p.k; j0 += kDeep) {
        Raw<KIND> y[UNITS][kDeep];
        float w[UNITS][kDeep];
        bool in[UNITS][kDeep];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int *const rows = p.rows + at[u].t * p.k + j0;
            const float *const weights = p.weights + at[u].t * p.k + j0;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                const long long row = mine[u] && j0 + j < p.k && is_choice(p, at[u].t, j0 + j) ? rows[j] : -1;
                in[u][j] = row >= 0 && row < p.M &&
                           is_y<KIND>(p, static_cast<const char *>(p.Y) + (row * p.ld_y + at[u].col) * kBytes, kVec * kBytes);
                w[u][j] = in[u][j] ? weights[j] : 0.f;
                if (in[u][j])
                    y[u][j].load(p.Y, row * p.ld_y + at[u].col);
            }
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int j = 0; j < kDeep; ++j)
                if (in[u][j]) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        acc[u][i] = fmaf(w[u][j], y[u][j].at(i), acc[u][i]);
                }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        if (!mine[u])
            continue;
        if (p.add) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                acc[u][i] += plus[u].at(i);
        }
        Raw<OUT> o;
        o.set(acc[u]);
        if (is_out<OUT>(p, at[u].t * p.ld_out + at[u].col, kVec))
            o.store(p.out, at[u].t * p.ld_out + at[u].col);
    }
}

// Rows off 16-byte boundaries, by words of 4 bytes: neighbouring threads have neighbouring words.
// A row of 16-bit elements that begins within a word is one element off: then a thread
// also loads the word after its own and takes the halves that it needs from the two, which is
// one instruction; the first and last row of Y, whose outer words may not lie wholly in Y, are
// loaded by elements.  Instructions and latency bound it: 1013 tokens of 6 rows of 1537 in fp16
// 6.8 us, with columns in whole pieces (1536) 4.8 as above (by elements 15.4; by aligned pieces
// of 16 bytes shifted into place 10.7, of 200 instructions a piece and row).  The CTAs that an
// SM holds hide more than rows in flight do: 16384 tokens 96 us with eight CTAs of four rows,
// 104 with seven, 146 with three or four of eight rows (in fp32, 1013 tokens, 10.4 with seven, 11.3
// with eight).
template <int KIND> struct Words {
    static constexpr bool kFp32 = KIND == W8A8_IN_FP32;
    static constexpr int kEach = kFp32 ? 8 : 4;         // a thread's words
    // a thread's i-th column in its warp's piece
    static __device__ __forceinline__ int column(int i)
    {
        const int lane = static_cast<int>(lane_index());
        return kFp32 ? 32 * i + lane : 64 * (i / 2) + 2 * lane + i % 2;
    }
    uint32_t w[kEach], next[kFp32 ? 1 : kEach];
    uint32_t shift;                                     // in bits
    // columns from p on, of which `left` are in the row (FULL: all); whole: words may be loaded
    // that reach an element out of it
    template <bool FULL> __device__ __forceinline__ void load(const CombineParams &c, const char *p, int left, bool whole)
    {
        shift = 0;
        if constexpr (kFp32) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if ((FULL || column(i) < left) && is_y<KIND>(c, p + 128 * i + 4 * lane_index(), 4))
                    w[i] = *reinterpret_cast<const uint32_t *>(p + 128 * i + 4 * lane_index());
        } else if (whole) {
            shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2) * 8;
            const uint32_t *const word = reinterpret_cast<const uint32_t *>(p - shift / 8) + lane_index();
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if ((FULL || column(2 * i) < left) && is_y<KIND>(c, word + 32 * i, 4))
                    w[i] = word[32 * i];
                if (shift && (FULL || column(2 * i + 1) < left) && is_y<KIND>(c, word + 32 * i + 1, 4))
                    next[i] = word[32 * i + 1];
            }
        } else {
            const uint16_t *const half = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                w[i] = (FULL || column(2 * i) < left) && is_y<KIND>(c, half + column(2 * i), 2) ? half[column(2 * i)] : 0;
                if ((FULL || column(2 * i + 1) < left) && is_y<KIND>(c, half + column(2 * i + 1), 2))
                    w[i] |= static_cast<uint32_t>(half[column(2 * i + 1)]) << 16;
            }
        }
    }
    __device__ __forceinline__ void add_to(float (&acc)[kVec], float weight) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if constexpr (kFp32) {
                acc[i] = fmaf(weight, __uint_as_float(w[i]), acc[i]);
            } else {
                const uint32_t u = __funnelshift_r(w[i], next[i], shift);
                float2 f;
                if constexpr (KIND == W8A8_IN_BF16)
                    f = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
                else
                    f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
                acc[2 * i] = fmaf(weight, f.x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(weight, f.y, acc[2 * i + 1]);
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

template <bool FULL, int KIND, int OUT, int UNITS>
__device__ __forceinline__ void sum_words(const CombineParams &p, const Piece (&at)[UNITS])
{
    using In = Words<KIND>;
    constexpr int kDeep = 4 / UNITS, kBytes = In::kFp32 ? 4 : 2;
    float acc[UNITS][kVec] = {}, plus[UNITS][kVec];
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int col = at[u].col + In::column(i);
            plus[u][i] = p.add && (FULL || (at[u].in && col < p.D)) && is_add<OUT>(p, at[u].t * p.ld_add + col, 1)
                             ? element<OUT>(p.add, at[u].t * p.ld_add + col) : 0.f;
        }
    for (int j0 = 0; j0 < p.k; j0 += kDeep) {
        In y[UNITS][kDeep];
        float w[UNITS][kDeep];
        bool in[UNITS][kDeep];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int *const rows = p.rows + at[u].t * p.k + j0;
            const float *const weights = p.weights + at[u].t * p.k + j0;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                const long long row = (FULL || at[u].in) && j0 + j < p.k && is_choice(p, at[u].t, j0 + j) ? rows[j] : -1;
                in[u][j] = row >= 0 && row < p.M;
                w[u][j] = in[u][j] ? weights[j] : 0.f;
                if (in[u][j])
                    y[u][j].template load<FULL>(p, static_cast<const char *>(p.Y) + (row * p.ld_y + at[u].col) * kBytes, p.D - at[u].col,
                                 row > 0 && row < p.M - 1);
            }
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int j = 0; j < kDeep; ++j)
                if (in[u][j])
                    y[u][j].add_to(acc[u], w[u][j]);
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int col = at[u].col + In::column(i);
            if (!FULL && (!at[u].in || col >= p.D))
                continue;
            const long long n = at[u].t * p.ld_out + col;
            const float v = acc[u][i] + plus[u][i];
            if (!is_out<OUT>(p, n, 1))
                continue;
            if constexpr (OUT == W8A8_IN_FP32)
                static_cast<float *>(p.out)[n] = v;
            else if constexpr (OUT == W8A8_IN_BF16)
                static_cast<__nv_bfloat16 *>(p.out)[n] = __float2bfloat16_rn(v);
            else
                static_cast<__half *>(p.out)[n] = __float2half_rn(v);
        }
}

template <int KIND, int OUT, int UNITS>
__global__ void __launch_bounds__(kThreads, UNITS == 4 ? 3 : UNITS == 2 ? 5 : Words<KIND>::kFp32 ? 7 : 8)
k_combine_words(const CombineParams p)
{
    Piece at[UNITS];
    find_pieces<true>(p, at);
    bool full = true;
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        full = full && at[u].in && at[u].col + 32 * kVec <= p.D;
    grid_dependency_wait();
    grid_launch_dependents();
    if (full)
        sum_words<true, KIND, OUT>(p, at);
    else
        sum_words<false, KIND, OUT>(p, at);
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

cudaError_t launch_pieces(void (*kernel)(CombineParams), const CombineParams &p, long long each, cudaStream_t stream)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>((p.pieces + each - 1) / each), 1, 1);
    lc.blockDim = dim3(kThreads, 1, 1);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

template <int KIND, int OUT> cudaError_t launch(CombineParams p, long long T, int sms, cudaStream_t stream)
{
    constexpr int kY = KIND == W8A8_IN_FP32 ? 4 : 2, kO = OUT == W8A8_IN_FP32 ? 4 : 2;
    const bool wide = p.D % 8 == 0 && on(p.Y, 16) && on(p.add, 16) && on(p.out, 16) && p.ld_y * kY % 16 == 0 &&
                      (!p.add || p.ld_add * kO % 16 == 0) && p.ld_out * kO % 16 == 0;
    // pieces of a CTA where they leave at most an eighth of its threads idle
    constexpr int kWarps = kThreads / 32;
    auto chunks = [&](int threads) { return (p.D + threads * kVec - 1) / (threads * kVec); };
    const bool warps = !wide || static_cast<long long>(chunks(kThreads)) * kThreads * kVec - p.D > p.D / 8;
    p.chunks = chunks(warps ? 32 : kThreads);
    p.pieces = T * p.chunks;
    // more of them with few rows to a token, where that leaves every SM 16 warps
    const int flight = wide ? 8 : 4;
    int units = p.k <= flight / 4 ? 4 : p.k <= flight / 2 ? 2 : 1;
    while (units > 1 && p.pieces * (warps ? 1 : kWarps) < 16ll * sms * units)
        units /= 2;
    const int each = units * (warps ? kWarps : 1);
    auto pick = [&](auto one, auto two, auto four) { return launch_pieces(units == 4 ? four : units == 2 ? two : one, p, each, stream); };
    if (wide && !warps)
        return pick(k_combine<KIND, OUT, false, 1>, k_combine<KIND, OUT, false, 2>, k_combine<KIND, OUT, false, 4>);
    if (wide)
        return pick(k_combine<KIND, OUT, true, 1>, k_combine<KIND, OUT, true, 2>, k_combine<KIND, OUT, true, 4>);
    return pick(k_combine_words<KIND, OUT, 1>, k_combine_words<KIND, OUT, 2>, k_combine_words<KIND, OUT, 4>);
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
    if (add_dev && add_dev == out_dev && ld_add != ld_out && T > 1)
        return record_error(W8A8_ERR_INVALID_ARG, "out in add's place with another row stride");
    if (T == 0 || D == 0)
        return W8A8_OK;
    if (!out_dev || (k > 0 && (!rows_dev || !weights_dev)) || (k > 0 && M > 0 && !Y_dev))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (D > (1ll << 24) || k > (1ll << 20) || T > ((1ll << 31) - 1) / ((D + 127) / 128))
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
    p.T = T;
    p.k = static_cast<int>(k);
    p.D = static_cast<int>(D);
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    p.status = dev.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (y_dtype == W8A8_IN_FP32)
        e = launch<W8A8_IN_FP32, W8A8_IN_FP32>(p, T, dev.sm_count, s);
    else if (y_dtype == W8A8_IN_BF16)
        e = out_dtype == W8A8_IN_FP32 ? launch<W8A8_IN_BF16, W8A8_IN_FP32>(p, T, dev.sm_count, s)
                                      : launch<W8A8_IN_BF16, W8A8_IN_BF16>(p, T, dev.sm_count, s);
    else
        e = out_dtype == W8A8_IN_FP32 ? launch<W8A8_IN_FP16, W8A8_IN_FP32>(p, T, dev.sm_count, s)
                                      : launch<W8A8_IN_FP16, W8A8_IN_FP16>(p, T, dev.sm_count, s);
    if (e == cudaSuccess)
        return W8A8_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "kernel launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return record_error(W8A8_ERR_CUDA, msg);
}
