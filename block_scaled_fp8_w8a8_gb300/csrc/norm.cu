// The norms around a transformer block, fused with its gate and its residual,
// and the per-token INT8 quantiser: the kernels that make the 8-bit operands
// of the matmuls from whole rows.
//
// Sandwich norm, for each row m (all arithmetic in fp32, one rounding per output):
//   u = h[m] / sqrt(mean(h[m]^2) + eps) * w_post      (w_post null: u = h[m])
//   r = res_scale * x[m] + gate[m / gate_rows] * u    (gate null: 1)
//   y = r / sqrt(mean(r^2) + eps) * w_pre             (w_pre null: y = r)
// x_out = r in x's type; y in h's type, or quantised as the matmuls take it:
// E4M3 codes with one scale per 128 columns, or INT8 codes with one per row.
// y is computed from the fp32 r, not from the rounded x_out.
//
// INT8 quantiser: a_s[m] = max_k |X[m,k]| / 127 (fp32 quotient; 1 where it is
// 0), A[m,k] = round_half_even(X[m,k] / a_s[m]) (fp32 quotient), in -127..127.
// A row with a NaN (an infinity) gets NaN (infinity) for a_s and zeros for A.
//
// HBM-bound: every input is read once and every output written once.  A row
// is held in registers by the threads of one CTA (or one warp, for short
// rows) between its two reductions; rows too long for that are held in shared
// memory.
#include <algorithm>
#include <cstdio>

#include "../../include/w8a8_block_fp8.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace w8a8 {
w8a8_status record_error(w8a8_status st, const char *message);

namespace {

constexpr int kPer = 16;                 // elements of a row that a thread holds in registers
constexpr int kMaxThreads = 1024;
constexpr int kRegRow = kPer * kMaxThreads;

template <int KIND> struct Elem;
template <> struct Elem<W8A8_IN_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float load(const T *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void store(T *p, float v) { *p = __float2bfloat16_rn(v); }
};
template <> struct Elem<W8A8_IN_FP16> {
    using T = __half;
    static __device__ __forceinline__ float load(const T *p) { return __half2float(*p); }
    static __device__ __forceinline__ void store(T *p, float v) { *p = __float2half_rn(v); }
};
template <> struct Elem<W8A8_IN_FP32> {
    using T = float;
    static __device__ __forceinline__ float load(const T *p) { return *p; }
    static __device__ __forceinline__ void store(T *p, float v) { *p = v; }
};

// VEC (8 or 1) consecutive elements at element index `i` of a row.  Eight are
// one or two 16-byte accesses; the row starts on a 16-byte boundary then.
template <int KIND, int VEC>
__device__ __forceinline__ void load_vec(const void *row, int i, float (&v)[VEC])
{
    using E = Elem<KIND>;
    const typename E::T *p = static_cast<const typename E::T *>(row) + i;
    if constexpr (VEC == 1) {
        v[0] = E::load(p);
    } else if constexpr (KIND == W8A8_IN_FP32) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = quant::element<KIND>(w, j);
    }
}

template <int KIND, int VEC>
__device__ __forceinline__ void store_vec(void *row, int i, const float (&v)[VEC])
{
    using E = Elem<KIND>;
    typename E::T *p = static_cast<typename E::T *>(row) + i;
    if constexpr (VEC == 1) {
        E::store(p, v[0]);
    } else if constexpr (KIND == W8A8_IN_FP32) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 a;
        if constexpr (KIND == W8A8_IN_BF16)
            a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        else
            a = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]),
                           pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
        *reinterpret_cast<uint4 *>(p) = a;
    }
}

// Sum (or maximum) of v over the threads of one row: the CTA, or a warp where
// the CTA's warps each have a row of their own.  Every thread gets the result;
// the order of the additions is fixed.  `part` is used once per launch.
struct Add {
    static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct Max {
    // NaN where either is one, so that a row with a NaN gets a NaN for its scale
    static __device__ __forceinline__ float op(float a, float b)
    {
        float m;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
        return m;
    }
};
// The same of a, |b| and |c| in one instruction.
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return m;
}
template <int N> __device__ __forceinline__ float max_abs(float a, const float (&v)[N])
{
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2)
        a = max_abs(a, v[j], v[j + 1]);
    return N % 2 ? Max::op(a, fabsf(v[N - 1])) : a;
}
template <typename Op>
__device__ __forceinline__ float row_reduce(float v, float *part, bool warp_rows)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = Op::op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (warp_rows)
        return v;
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int l = static_cast<int>(threadIdx.x & 31);
    v = part[l < warps ? l : 0];          // every warp reduces the partials alike
    if (l >= warps)
        v = 0.f;                          // neutral: the maxima are of magnitudes
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = Op::op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A row's scale for INT8 codes from its absolute maximum.
__device__ __forceinline__ float int8_scale(float amax)
{
    const float s = __fdiv_rn(amax, 127.f);
    return s == 0.f ? 1.f : s;            // an all-zero row, or a maximum that underflows
}

__device__ __forceinline__ uint32_t int8_code(float q)
{
    // |q| <= 127 (1 + 2^-23) but where a subnormal scale lost precision, or NaN
    // (a scale that is not finite), which is converted to 0
    return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(q)))) & 0xffu;
}

// Four codes of two quotient pairs.  FAST (a normal scale): |q| < 127.5, and
// adding 3 * 2^22 rounds a quotient half-to-even to its units, which are then
// the sum's low byte.
template <bool FAST>
__device__ __forceinline__ uint32_t int8_codes4(float a, float b, float c, float d, float s,
                                                uint64_t ns2, uint64_t y2)
{
    if constexpr (FAST) {
        const uint64_t one = pack2f(1.f, 1.f), magic = pack2f(12582912.f, 12582912.f);
        const uint64_t p = fma2_rn(quant::div_by_scale2(pack2f(a, b), ns2, y2), one, magic);
        const uint64_t q = fma2_rn(quant::div_by_scale2(pack2f(c, d), ns2, y2), one, magic);
        return __byte_perm(__byte_perm(static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32), 0x0040),
                           __byte_perm(static_cast<uint32_t>(q), static_cast<uint32_t>(q >> 32), 0x0040),
                           0x5410);
    } else {
        return int8_code(__fdiv_rn(a, s)) | int8_code(__fdiv_rn(b, s)) << 8 |
               int8_code(__fdiv_rn(c, s)) << 16 | int8_code(__fdiv_rn(d, s)) << 24;
    }
}

template <int VEC>
__device__ __forceinline__ void store_int8(uint8_t *p, const float (&v)[VEC], float s)
{
    const bool fast = s >= 0x1p-64f && s <= 0x1p64f;
    const float y = __frcp_rn(s);
    const uint64_t ns2 = pack2f(-s, -s), y2 = pack2f(y, y);
    if constexpr (VEC == 1) {
        *p = static_cast<uint8_t>(fast ? int8_codes4<true>(v[0], 0.f, 0.f, 0.f, s, ns2, y2)
                                       : int8_codes4<false>(v[0], 0.f, 0.f, 0.f, s, ns2, y2));
    } else {
        uint32_t w[VEC / 4];
        if (fast) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
                w[j / 4] = int8_codes4<true>(v[j], v[j + 1], v[j + 2], v[j + 3], s, ns2, y2);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
                w[j / 4] = int8_codes4<false>(v[j], v[j + 1], v[j + 2], v[j + 3], s, ns2, y2);
        }
#pragma unroll
        for (int j = 0; j < VEC / 8; ++j)
            reinterpret_cast<uint2 *>(p)[j] = make_uint2(w[2 * j], w[2 * j + 1]);
    }
}

struct NormParams {
    const void *h, *x, *w_post, *gate, *w_pre;
    void *x_out, *y;
    float *scales;
    long long M;
    int D;
    long long ld_h, ld_x, ld_xo, ld_y;     // elements per row
    long long gate_rows;
    float res_scale, eps;
    int y_kind;                            // w8a8_norm_out
    int row_threads;                       // 32: a warp per row, else the CTA
    unsigned *status;
};

// The E4M3 codes of eight columns e .. e+7 of row m and their group's scale.
// Sixteen neighbouring lanes hold one 128-column group; every lane of the warp
// calls it (`in`: the columns exist).
__device__ __forceinline__ void store_fp8(const NormParams &p, long long m, uint8_t *row, int e,
                                          bool in, const float (&v)[8], float amax)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = quant::group_scale(amax);
    if (!in)
        return;
    const bool fast = s >= 0x1p-64f && s <= 0x1p64f;
    const float rc = __frcp_rn(s);
    const uint64_t ns2 = pack2f(-s, -s), y2 = pack2f(rc, rc);
    uint32_t raw[8], c[2];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        raw[j] = __float_as_uint(v[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        c[j] = fast ? quant::encode4<W8A8_IN_FP32, true>(raw, j, s, ns2, y2)
                    : quant::encode4<W8A8_IN_FP32, false>(raw, j, s, ns2, y2);
    *reinterpret_cast<uint2 *>(row + e) = make_uint2(c[0], c[1]);
    if ((lane_index() & 15) == 0)
        p.scales[m * ((p.D + 127) / 128) + e / 128] = s;
}

// One row per CTA (per warp where row_threads is 32).  HELD: the row stays in
// the threads' registers; otherwise in dynamic shared memory (D floats).  EARLY:
// at most kEarlyThreads, whose registers also hold the weights and the gate,
// loaded along with the row.
// Bound by the latency of the loads and of two reductions over the CTA: one row of
// 4096 in bf16 2.6 us (back to back), 64 rows to FP8 or INT8 3.5 us.  (Beyond 8192
// columns, at 64 registers a thread, single elements (VEC 1) spill some 320 bytes.)
constexpr int kEarlyThreads = 512;
template <int HK, int XK, int VEC, bool HELD, bool EARLY>
__global__ void __launch_bounds__(EARLY ? kEarlyThreads : kMaxThreads)
    k_sandwich_norm(const NormParams p)
{
    extern __shared__ float held[];
    __shared__ float part[3][32];
    constexpr int kN = HELD ? kPer / VEC : 1;
    constexpr int kHB = HK == W8A8_IN_FP32 ? 4 : 2, kXB = XK == W8A8_IN_FP32 ? 4 : 2;
    grid_launch_dependents();
    grid_dependency_wait();          // the inputs come from the work before this launch
    const bool warp_rows = p.row_threads == 32;
    const int T = warp_rows ? 32 : static_cast<int>(blockDim.x);
    const int tid = warp_rows ? static_cast<int>(lane_index()) : static_cast<int>(threadIdx.x);
    const long long m = warp_rows
                            ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp_index()
                            : static_cast<long long>(blockIdx.x);
    if (m >= p.M || !in_bounds(m >= 0 && p.D > 0, p.status, SITE_BOUNDS_A))
        return;                      // whole warps (or the CTA): nothing waits for them
    const int D = p.D;
    const uint8_t *hrow = static_cast<const uint8_t *>(p.h) + m * p.ld_h * kHB;
    const uint8_t *xrow = static_cast<const uint8_t *>(p.x) + m * p.ld_x * kXB;
    uint8_t *orow = static_cast<uint8_t *>(p.x_out) + m * p.ld_xo * kXB;
    const uint8_t *grow =
        p.gate ? static_cast<const uint8_t *>(p.gate) + (m / p.gate_rows) * D * kHB : nullptr;
    const int steps = HELD ? kN : (D + T * VEC - 1) / (T * VEC);

    float v[kN][VEC], xv[kN][VEC], early[EARLY ? 3 : 1][kN][VEC];
    // Chunk i of this thread: VEC elements from (i T + tid) VEC; D % VEC == 0.
    auto at = [&](int i) { return (i * T + tid) * VEC; };

    // (the unrolled form of every pass indexes registers; the other walks the row)
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = at(i);
        float(&w)[VEC] = v[HELD ? i : 0];
        if (HELD && e < D) {
            load_vec<HK, VEC>(hrow, e, w);
            load_vec<XK, VEC>(xrow, e, xv[HELD ? i : 0]);
            if constexpr (EARLY) {
                if (p.w_post)
                    load_vec<HK, VEC>(p.w_post, e, early[0][i]);
                if (grow)
                    load_vec<HK, VEC>(grow, e, early[1][i]);
                if (p.w_pre)
                    load_vec<HK, VEC>(p.w_pre, e, early[2][i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = at(i);
        float(&w)[VEC] = v[HELD ? i : 0];
        if (e < D) {
            if (!HELD)
                load_vec<HK, VEC>(hrow, e, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                ss = fmaf(w[j], w[j], ss);
                if (!HELD)
                    held[e + j] = w[j];
            }
        }
    }
    float inv = 1.f;
    if (p.w_post)
        inv = rsqrtf(row_reduce<Add>(ss, part[0], warp_rows) / static_cast<float>(D) + p.eps);

    ss = 0.f;
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = at(i);
        float(&w)[VEC] = v[HELD ? i : 0];
        float(&xw)[VEC] = xv[HELD ? i : 0];
        if (e < D) {
            float wp_[VEC], g_[VEC];
            float(&wp)[VEC] = EARLY ? early[0][HELD ? i : 0] : wp_;
            float(&g)[VEC] = EARLY ? early[EARLY ? 1 : 0][HELD ? i : 0] : g_;
            if (!EARLY && p.w_post)
                load_vec<HK, VEC>(p.w_post, e, wp);
            if (!EARLY && grow)
                load_vec<HK, VEC>(grow, e, g);
            if (!HELD)
                load_vec<XK, VEC>(xrow, e, xw);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float u = HELD ? w[j] : held[e + j];
                if (p.w_post)
                    u = u * inv * wp[j];
                if (grow)
                    u *= g[j];
                const float r = fmaf(p.res_scale, xw[j], u);
                ss = fmaf(r, r, ss);
                w[j] = r;
                if (!HELD)
                    held[e + j] = r;
            }
            if (p.x_out)
                store_vec<XK, VEC>(orow, e, w);
        }
    }
    inv = 1.f;
    if (p.w_pre)
        inv = rsqrtf(row_reduce<Add>(ss, part[1], warp_rows) / static_cast<float>(D) + p.eps);

    // y, and its absolute maximum where one scale covers the row
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = at(i);
        float(&w)[VEC] = v[HELD ? i : 0];
        const bool in = e < D;
        if (in) {
            float wp_[VEC];
            float(&wp)[VEC] = EARLY ? early[EARLY ? 2 : 0][HELD ? i : 0] : wp_;
            if (!EARLY && p.w_pre)
                load_vec<HK, VEC>(p.w_pre, e, wp);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float y = HELD ? w[j] : held[e + j];
                if (p.w_pre)
                    y = y * inv * wp[j];
                w[j] = y;
                if (!HELD && p.y_kind == W8A8_NORM_INT8)
                    held[e + j] = y;
            }
            if (p.y_kind == W8A8_NORM_INT8) {
                amax = max_abs(amax, w);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    amax = fmaxf(amax, fabsf(w[j]));
            }
        }
        if (p.y_kind == W8A8_NORM_SAME) {
            if (in)
                store_vec<HK, VEC>(static_cast<uint8_t *>(p.y) + m * p.ld_y * kHB, e, w);
        } else if (VEC == 8 && p.y_kind == W8A8_NORM_FP8) {
            const int warp_first = at(i) - static_cast<int>(lane_index()) * VEC;
            if (warp_first < D) {            // the same for the whole warp
                float w8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w8[j] = w[VEC == 8 ? j : 0];
                store_fp8(p, m, static_cast<uint8_t *>(p.y) + m * p.ld_y, e, in, w8,
                          in ? amax : 0.f);
            }
            amax = 0.f;
        }
    }
    if (p.y_kind == W8A8_NORM_INT8) {
        const float s = int8_scale(row_reduce<Max>(amax, part[2], warp_rows));
        uint8_t *row = static_cast<uint8_t *>(p.y) + m * p.ld_y;
#pragma unroll
        for (int i = 0; i < (HELD ? kN : steps); ++i) {
            const int e = at(i);
            if (e < D) {
                float w[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    w[j] = HELD ? v[HELD ? i : 0][j] : held[e + j];
                store_int8<VEC>(row + e, w, s);
            }
        }
        if (tid == 0)
            p.scales[m] = s;
    }
}

// ------------------------------------------------------------------ many rows

// The same for many rows of at most 8192 columns, as a stream: persistent CTAs
// walk the rows, each thread on the same 16 columns of every row, so that the
// norms' weights stay in its registers in fp32 (the post-norm's times the gate,
// while the gate's row lasts).  The rows of h and x come through a ring of
// shared-memory stages filled by bulk copies, so that the next rows' loads are in
// flight through a row's two reductions.
// HBM-bound: 16384 x 4096 in bf16 with FP8 codes 79.7 us (5.9 TB/s), with INT8 codes 84.2
// us (5.6 TB/s; a third reduction per row), with bf16 94.0 us (5.7 TB/s).
constexpr int kRingMaxStages = 4;
constexpr int kRingThreads = 512;

struct RingParams {
    NormParams n;
    int stages;
    uint32_t h_bytes, x_bytes;             // of one row
    float inv_d;                           // 1 / D
    unsigned long long wait_limit;
};

// A persistent CTA's rows.  Round robin, so that the CTAs read one neighbourhood
// of memory at a time (16384 rows of 3943: 120 against 140 us for a run of rows
// each); but neighbours where the gate's row changes among them, as it then
// changes seldom.  (g_rest counts rows since the gate's last change: with one row
// of the gate for all it never reaches gate_rows.)
struct RowWalk {
    int first, step, last;             // M < 2^31, and so is every m + step
    __device__ explicit RowWalk(const NormParams &p)
    {
        if (p.gate && p.gate_rows < p.M) {
            first = static_cast<int>(p.M * blockIdx.x / gridDim.x);
            step = 1;
            last = static_cast<int>(p.M * (blockIdx.x + 1) / gridDim.x);
        } else {
            first = static_cast<int>(blockIdx.x);
            step = static_cast<int>(gridDim.x);
            last = static_cast<int>(p.M);
        }
    }
};

// Eight elements as four fp32 pairs, from shared or global memory.
template <int KIND>
__device__ __forceinline__ void pairs_of(const uint32_t (&w)[KIND == W8A8_IN_FP32 ? 8 : 4],
                                         uint64_t *v)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = pack2f(quant::element<KIND>(w, 2 * j), quant::element<KIND>(w, 2 * j + 1));
}
template <int KIND> __device__ __forceinline__ void shared_pairs(uint32_t addr, uint64_t *v)
{
    uint32_t w[KIND == W8A8_IN_FP32 ? 8 : 4];
#pragma unroll
    for (int i = 0; i < (KIND == W8A8_IN_FP32 ? 2 : 1); ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(addr + 16u * i));
    pairs_of<KIND>(w, v);
}
template <int KIND> __device__ __forceinline__ void global_pairs(const void *row, int e, uint64_t *v)
{
    uint32_t w[KIND == W8A8_IN_FP32 ? 8 : 4];
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) +
                                                     e * (KIND == W8A8_IN_FP32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (KIND == W8A8_IN_FP32 ? 2 : 1); ++i) {
        const uint4 a = __ldg(p + i);
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
    pairs_of<KIND>(w, v);
}

// A thread's 16 columns from e.  WIDE: all exist and the row lies on 32-byte
// boundaries; whole 32-byte sectors leave in one store each (two 16-byte stores
// to a sector cost the L2 two requests: 37 against 31 us for 4864 x 4096).
template <int KIND, bool WIDE>
__device__ __forceinline__ void store_pairs(uint8_t *row, int e, bool in0, bool in1,
                                            const uint64_t (&v)[8])
{
    float f[16];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        unpack2f(v[j], f[2 * j], f[2 * j + 1]);
    if constexpr (!WIDE) {
        if (in0)
            store_vec<KIND, 8>(row, e, reinterpret_cast<const float(&)[8]>(f[0]));
        if (in1)
            store_vec<KIND, 8>(row, e + 8, reinterpret_cast<const float(&)[8]>(f[8]));
    } else if constexpr (KIND == W8A8_IN_FP32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = __float_as_uint(f[8 * h + j]);
            st_global_v8(row + 4 * e + 32 * h, w);
        }
    } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = KIND == W8A8_IN_BF16 ? pack_bf16x2(f[2 * j], f[2 * j + 1])
                                        : pack_f16x2(f[2 * j], f[2 * j + 1]);
        st_global_v8(row + 2 * e, w);
    }
}

// Sum over the CTA of at most THREADS threads, the same bits for every thread:
// warps by shuffles, then every thread adds the warps' partials in order (zeros
// past the last warp).
template <int THREADS> __device__ __forceinline__ float cta_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane_index() == 0)
        part[warp_index()] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < (THREADS + 127) / 128; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(part)[i];
        v += (f.x + f.y) + (f.z + f.w);
    }
    return v;
}

// E4M3 codes of a thread's 16 columns (values as fp32 pairs) and their group's
// scale; eight neighbouring lanes hold a group.
__device__ __forceinline__ void store_fp8_16(float *scale_row, uint8_t *row, int e, bool in0,
                                             bool in1, const uint64_t (&v)[8])
{
    uint32_t raw[16];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float a, b;
        unpack2f(v[j], a, b);
        raw[2 * j] = __float_as_uint(a);
        raw[2 * j + 1] = __float_as_uint(b);
        amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = quant::group_scale(amax);
    const uint4 q = quant::encode16<W8A8_IN_FP32>(raw, s);
    if (in0)
        *reinterpret_cast<uint2 *>(row + e) = make_uint2(q.x, q.y);
    if (in1)
        *reinterpret_cast<uint2 *>(row + e + 8) = make_uint2(q.z, q.w);
    if (in0 && (lane_index() & 7) == 0)
        scale_row[e >> 7] = s;
}

// FULL: the threads' columns cover the row exactly (D = 16 x the CTA's threads)
// and the outputs' rows lie on 32-byte boundaries.
template <int HK, int XK, int THREADS, int PER_SM, bool FULL>
__global__ void __launch_bounds__(THREADS, PER_SM) k_sandwich_ring(const RingParams rp)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) float part[2][2][16];
    __shared__ float part_max[2][32];
    __shared__ __align__(8) uint64_t bars[kRingMaxStages];
    __shared__ int abort_word;
    constexpr int kHB = HK == W8A8_IN_FP32 ? 4 : 2, kXB = XK == W8A8_IN_FP32 ? 4 : 2;
    const NormParams &p = rp.n;
    volatile int *abort_flag = &abort_word;
    const int tid = static_cast<int>(threadIdx.x), D = p.D;
    const int e0 = 16 * tid, e1 = e0 + 8;             // the thread's two chunks
    const bool in0 = FULL || e0 < D, in1 = FULL || e1 < D;
    const uint32_t ring0 = smem_addr(ring), bar0 = smem_addr(bars);
    const uint32_t stage_bytes = rp.h_bytes + rp.x_bytes;
    for (int i = tid; i < 64; i += static_cast<int>(blockDim.x))
        (&part[0][0][0])[i] = 0.f;
    if (tid == 0) {
        for (int s = 0; s < rp.stages; ++s)
            mbar_init(bar0 + 8u * s, 1);
        abort_word = 0;
        mbar_fence_init();
    }
    __syncthreads();
    const WaitGuard guard{abort_flag, p.status, rp.wait_limit};
    grid_launch_dependents();
    grid_dependency_wait();
    const RowWalk walk(p);
    const int first = walk.first, step = walk.step, last = walk.last;
    // (thread 0; after a timeout nothing more is copied)
    uint32_t filled = 0, last_phase = 0;   // stages filled at all, and their last fills' parities
    auto fill = [&](long long m, int s) {
        if (*abort_flag || !in_bounds(m >= 0 && m < p.M, p.status, SITE_BOUNDS_A))
            return;
        last_phase = filled >> s & 1u ? last_phase ^ (1u << s) : last_phase;
        filled |= 1u << s;
        const uint32_t bar = bar0 + 8u * s, dst = ring0 + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        bulk_load(dst, static_cast<const uint8_t *>(p.h) + m * p.ld_h * kHB, rp.h_bytes, bar);
        bulk_load(dst + rp.h_bytes, static_cast<const uint8_t *>(p.x) + m * p.ld_x * kXB, rp.x_bytes,
                  bar);
    };
    if (tid == 0)
        for (int s = 0; s < rp.stages && first + s * step < last; ++s)
            fill(first + s * step, s);

    const uint64_t one2 = pack2f(1.f, 1.f), scale2 = pack2f(p.res_scale, p.res_scale);
    uint64_t wpost[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        wpost[j] = one2;
    // The pre-norm's weights of this thread's columns wait in shared memory
    // (16 more registers a thread would cost the third CTA per SM), four
    // 16-byte words a thread, neighbouring threads' side by side.
    const uint32_t pre0 = ring0 + rp.stages * stage_bytes + 16u * tid;
    const uint32_t pre_step = 16u * blockDim.x;
    if (p.w_pre) {
        uint64_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = one2;
        if (in0)
            global_pairs<HK>(p.w_pre, e0, w);
        if (in1)
            global_pairs<HK>(p.w_pre, e1, w + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(pre0 + j * pre_step),
                         "l"(w[2 * j]), "l"(w[2 * j + 1])
                         : "memory");
    }
    // w_post times the gate's row
    auto load_post = [&](long long g) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int e = c ? e1 : e0;
            if (e < D) {
                if (p.w_post)
                    global_pairs<HK>(p.w_post, e, wpost + 4 * c);
                if (p.gate) {
                    uint64_t w[4];
                    global_pairs<HK>(static_cast<const uint8_t *>(p.gate) + g * D * kHB, e, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        wpost[4 * c + j] = p.w_post ? mul2_rn(wpost[4 * c + j], w[j]) : w[j];
                }
            }
        }
    };
    int g = 0, g_rest = 0;             // the gate's row, and rows since it began
    if (p.gate) {
        g = static_cast<int>(first / p.gate_rows);
        g_rest = static_cast<int>(first - g * p.gate_rows);
    }
    load_post(g);

    uint8_t *orow = static_cast<uint8_t *>(p.x_out) + static_cast<long long>(first) * p.ld_xo * kXB;
    const int yb = p.y_kind == W8A8_NORM_SAME ? kHB : 1;
    const int per_row = p.y_kind == W8A8_NORM_FP8 ? (D + 127) / 128 : 1;      // scales
    uint8_t *yrow = static_cast<uint8_t *>(p.y) + static_cast<long long>(first) * p.ld_y * yb;
    const long long o_step = step * p.ld_xo * kXB, y_step = step * p.ld_y * yb, s_step = static_cast<long long>(step) * per_row;
    float *srow = p.scales + static_cast<long long>(first) * per_row;
    int stage = 0, odd = 0;
    uint32_t phase = 0;
    for (int m = first; m < last; m += step, odd ^= 1, orow += o_step, yrow += y_step,
                   srow += s_step) {
        // A wait that runs out leaves garbage in the row, an entry in the
        // status word and the abort flag, which ends every later wait at once.
        wait_bounded(bar0 + 8u * stage, phase, guard, SITE_NORM_ROWS);
        const uint32_t src = ring0 + stage * stage_bytes;
        uint64_t v[8], ss2 = 0;
        if (!FULL) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = 0;
        }
        if (in0)
            shared_pairs<HK>(src + e0 * kHB, v);
        if (in1)
            shared_pairs<HK>(src + e1 * kHB, v + 4);
        float inv = 1.f, a, b;
        if (p.w_post) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                fma2(ss2, v[j], v[j]);
            unpack2f(ss2, a, b);
            inv = rsqrtf(fmaf(cta_sum<THREADS>(a + b, part[odd][0]), rp.inv_d, p.eps));
        }
        ss2 = 0;
        const uint64_t inv2 = pack2f(inv, inv);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint64_t x[4];
            if (!FULL)
                x[0] = x[1] = x[2] = x[3] = 0;
            if (c ? in1 : in0)
                shared_pairs<XK>(src + rp.h_bytes + (c ? e1 : e0) * kXB, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t &w = v[4 * c + j];
                w = fma2_rn(scale2, x[j], mul2_rn(mul2_rn(w, inv2), wpost[4 * c + j]));
                fma2(ss2, w, w);
            }
        }
        inv = 1.f;
        if (p.w_pre) {
            unpack2f(ss2, a, b);
            inv = rsqrtf(fmaf(cta_sum<THREADS>(a + b, part[odd][1]), rp.inv_d, p.eps));
        } else {
            __syncthreads();
        }
        // Every thread has read its part of the stage: refill it.
        if (tid == 0 && m + rp.stages * step < last)
            fill(m + rp.stages * step, stage);
        if (++stage == rp.stages) {
            stage = 0;
            phase ^= 1u;
        }
        if (p.x_out)
            store_pairs<XK, FULL>(orow, e0, in0, in1, v);
        if (p.w_pre) {
            const uint64_t pre2 = pack2f(inv, inv);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t a2, b2;
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                             : "=l"(a2), "=l"(b2)
                             : "r"(pre0 + j * pre_step));
                v[2 * j] = mul2_rn(mul2_rn(v[2 * j], pre2), a2);
                v[2 * j + 1] = mul2_rn(mul2_rn(v[2 * j + 1], pre2), b2);
            }
        }
        if (p.y_kind == W8A8_NORM_SAME) {
            store_pairs<HK, FULL>(yrow, e0, in0, in1, v);
        } else if (p.y_kind == W8A8_NORM_FP8) {
            store_fp8_16(srow, yrow, e0, in0, in1, v);
        } else {
            float amax = 0.f, f[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                unpack2f(v[j], f[2 * j], f[2 * j + 1]);
                amax = max_abs(amax, f[2 * j], f[2 * j + 1]);
            }
            const float s = int8_scale(row_reduce<Max>(amax, part_max[odd], false));
            if (in1)
                store_int8<16>(yrow + e0, f, s);
            else if (in0)
                store_int8<8>(yrow + e0, reinterpret_cast<const float(&)[8]>(f[0]), s);
            if (tid == 0)
                *srow = s;
        }
        if (p.gate && ++g_rest == p.gate_rows && m + step < last) {
            g_rest = 0;
            load_post(++g);
        }
    }
    // After a timeout the copies still in flight land before the CTA leaves.
    if (tid == 0 && *abort_flag)
        for (int s = 0; s < rp.stages; ++s)
            if (filled >> s & 1u)
                wait_drain(bar0 + 8u * s, last_phase >> s & 1u, p.status, rp.wait_limit,
                           (SITE_DRAIN << 8) | 4u);
}

// ------------------------------------------------------------------ rows of any width

// Rows of a width that leaves them off 16-byte boundaries (so not for FP8 codes).
// All tensors are dense, so row m starts at element m D of each; a thread takes 16
// elements from an element index that is a multiple of 8, which every tensor loads
// and stores in whole 16-byte words (the words at a row's two ends hold elements of
// its neighbours: masked on the way in, stored one by one on the way out).  Column 16 t + k of a norm's
// weights lies at [k][t] in shared memory, so that a row shifted by s of 8
// elements reads them without bank conflicts.  The next row's words wait in
// registers while this one's reductions run.
// Bound by instruction issue and the two reductions per row: 8192 rows of 1537 in
// fp16 25.5 us (3.9 TB/s), 16384 of 3943 in bf16 104 us (5.0 TB/s).  (1024 threads, at 64
// registers each, spill 170 to 290 bytes.)
struct FlatParams {
    NormParams n;
    float inv_d;
};

template <int KIND> struct Raw16 {
    static constexpr int kWords = KIND == W8A8_IN_FP32 ? 16 : 8;
    uint32_t w[kWords];
    // 16 elements at element index f, those before `total`
    __device__ __forceinline__ void load(const void *base, long long f, long long total)
    {
        constexpr int kB = KIND == W8A8_IN_FP32 ? 4 : 2;
        const uint8_t *p = static_cast<const uint8_t *>(base) + f * kB;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t *d = w + c * (kWords / 2);
            if (f + 8 * c + 8 <= total) {
                const uint4 *q = reinterpret_cast<const uint4 *>(p + 8 * c * kB);
#pragma unroll
                for (int i = 0; i < kWords / 8; ++i) {
                    const uint4 v = q[i];
                    d[4 * i] = v.x, d[4 * i + 1] = v.y, d[4 * i + 2] = v.z, d[4 * i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kWords / 2; ++i)
                    d[i] = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (f + 8 * c + j >= total)
                        continue;
                    if constexpr (KIND == W8A8_IN_FP32)
                        d[j] = reinterpret_cast<const uint32_t *>(p)[8 * c + j];
                    else
                        d[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[8 * c + j])
                                    << (16 * (j & 1));
                }
            }
        }
    }
    __device__ __forceinline__ float operator[](int j) const { return quant::element<KIND>(w, j); }
};

// The elements of v that lie in columns 0 .. D-1, v's first one being column c0.
template <int KIND>
__device__ __forceinline__ void store_flat(uint8_t *row, int c0, int D, const float (&v)[16])
{
    constexpr int kB = KIND == W8A8_IN_FP32 ? 4 : 2;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int at = c0 + 8 * c;
        if (at >= 0 && at + 8 <= D) {
            store_vec<KIND, 8>(row + static_cast<long long>(at) * kB, 0,
                               reinterpret_cast<const float(&)[8]>(v[8 * c]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at + j >= 0 && at + j < D)
                    Elem<KIND>::store(reinterpret_cast<typename Elem<KIND>::T *>(row) + at + j,
                                      v[8 * c + j]);
        }
    }
}

template <int HK, int XK, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) k_sandwich_flat(const FlatParams fp)
{
    // post [16][kPitch], pre [16][kPitch], thread t's columns at t + 1 (at 0 zeros, for
    // the elements before a row's first); the pitch keeps the columns of a coalesced
    // load, 16 words of a row apart, in different banks
    extern __shared__ float weights[];
    constexpr int kPitch = THREADS + 2;
    __shared__ __align__(16) float part[2][2][THREADS < 128 ? 4 : THREADS / 32];
    __shared__ float part_max[2][32];
    constexpr int kHB = HK == W8A8_IN_FP32 ? 4 : 2, kXB = XK == W8A8_IN_FP32 ? 4 : 2;
    const NormParams &p = fp.n;
    const int tid = static_cast<int>(threadIdx.x), D = p.D;
    const long long total = p.M * D;
    const RowWalk walk(p);
    const int first = walk.first, step = walk.step, last = walk.last;
    for (int i = tid; i < static_cast<int>(sizeof(part) / 4); i += static_cast<int>(blockDim.x))
        (&part[0][0][0])[i] = 0.f;
    if (tid < 32)
        weights[tid * kPitch] = 0.f;
    grid_launch_dependents();
    grid_dependency_wait();
    const bool has_post = p.w_post || p.gate;
    using HE = Elem<HK>;
    Raw16<HK> hn;
    Raw16<XK> xn;
    auto fetch = [&](long long row) {
        const long long f = (row * D & ~7ll) + 16 * tid;
        if (f < (row + 1) * D && in_bounds(row < p.M, p.status, SITE_BOUNDS_A)) {
            hn.load(p.h, f, total);
            xn.load(p.x, f, total);
        }
    };
    fetch(first);
    // Columns tid + i blockDim.x of a vector for eight i from h, 0 past D: every load
    // before any use.
    auto columns = [&](const void *w, int h, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = tid + (h + i) * static_cast<int>(blockDim.x);
            v[i] = c < D ? HE::load(static_cast<const typename HE::T *>(w) + c) : 0.f;
        }
    };
    auto put = [&](float *dst, int h, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = tid + (h + i) * static_cast<int>(blockDim.x);
            dst[(c & 15) * kPitch + (c >> 4) + 1] = v[i];
        }
    };
    auto load_post = [&](long long g) {
        for (int h = 0; h < 16; h += 8) {
            float w[8], u[8];
            if (p.gate)
                columns(static_cast<const typename HE::T *>(p.gate) + g * D, h, u);
            if (p.w_post)
                columns(p.w_post, h, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = !p.gate ? w[i] : p.w_post ? w[i] * u[i] : u[i];
            put(weights, h, w);
        }
    };
    int g = 0, g_rest = 0;             // the gate's row, and rows since it began
    if (p.gate) {
        g = static_cast<int>(first / p.gate_rows);
        g_rest = static_cast<int>(first - g * p.gate_rows);
    }
    if (has_post)
        load_post(g);
    if (p.w_pre)
        for (int h = 0; h < 16; h += 8) {
            float w[8];
            columns(p.w_pre, h, w);
            put(weights + 16 * kPitch, h, w);
        }
    __syncthreads();

    const uint32_t w0 = smem_addr(weights) + 4u * (tid + 1);
    int odd = 0;
    for (int m = first; m < last; m += step, odd ^= 1) {
        const long long m0 = static_cast<long long>(m) * D;        // the row's first element
        const int s = static_cast<int>(m0 & 7);
        const int c0 = 16 * tid - s;                   // column of v[0]
        const bool any = c0 < D, all = c0 >= 0 && c0 + 16 <= D;
        float v[16], x[16];
        if (all) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                v[j] = hn[j];
                x[j] = xn[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const bool in = c0 + j >= 0 && c0 + j < D;
                v[j] = in ? hn[j] : 0.f;
                x[j] = in ? xn[j] : 0.f;
            }
        }
        if (m + step < last)
            fetch(m + step);
        // weight of v[j]: [j - s][tid], or [j - s + 16][tid - 1]
        const uint32_t wa = w0 - 4u * s * kPitch;
        auto weight = [&](int j, int pre) {
            const uint32_t at = (j < 8 && j < s ? wa + 4u * (16 * kPitch - 1) : wa) +
                                4u * (j + 16 * pre) * kPitch;
            float w;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(at));
            return w;
        };
        float ss = 0.f, inv = 1.f;
        if (p.w_post) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                ss = fmaf(v[j], v[j], ss);
            inv = rsqrtf(fmaf(cta_sum<THREADS>(ss, part[odd][0]), fp.inv_d, p.eps));
        }
        ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float u = v[j];
            if (has_post)
                u = u * inv * weight(j, 0);
            v[j] = fmaf(p.res_scale, x[j], u);
            ss = fmaf(v[j], v[j], ss);
        }
        if (p.x_out && any)
            store_flat<XK>(static_cast<uint8_t *>(p.x_out) + m0 * kXB, c0, D, v);
        if (p.w_pre) {
            inv = rsqrtf(fmaf(cta_sum<THREADS>(ss, part[odd][1]), fp.inv_d, p.eps));
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = v[j] * inv * weight(j, 1);
        }
        if (p.y_kind == W8A8_NORM_SAME) {
            if (any)
                store_flat<HK>(static_cast<uint8_t *>(p.y) + m0 * kHB, c0, D, v);
        } else {
            const float sc = int8_scale(row_reduce<Max>(max_abs(0.f, v), part_max[odd], false));
            uint8_t *row = static_cast<uint8_t *>(p.y) + m0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int at = c0 + 8 * c;
                if (at >= 0 && at + 8 <= D) {
                    store_int8<8>(row + at, reinterpret_cast<const float(&)[8]>(v[8 * c]), sc);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (at + j >= 0 && at + j < D)
                            store_int8<1>(row + at + j, reinterpret_cast<const float(&)[1]>(v[8 * c + j]),
                                          sc);
                }
            }
            if (tid == 0)
                p.scales[m] = sc;
        }
        if (p.gate && ++g_rest == p.gate_rows && m + step < last) {
            g_rest = 0;
            __syncthreads();                       // this row's weights have been read
            load_post(++g);
            __syncthreads();
        }
    }
}

struct QuantParams {
    const void *X;
    uint8_t *A;
    float *a_s;
    long long M;
    int K;
    long long ld_x, ld_a;
    int row_threads;
    unsigned *status;
};

// HELD: the row stays in registers; otherwise it is read twice.
// 16384 x 4096 in bf16: 43.3 us (4.6 TB/s), with 60 % of the issue slots taken, most by
// the correctly rounded quotients.
template <int KIND, int VEC, bool HELD>
__global__ void __launch_bounds__(kMaxThreads) k_quant_int8(const QuantParams p)
{
    __shared__ float part[32];
    constexpr int kN = HELD ? kPer / VEC : 1;
    constexpr int kB = KIND == W8A8_IN_FP32 ? 4 : 2;
    grid_launch_dependents();
    grid_dependency_wait();
    const bool warp_rows = p.row_threads == 32;
    const int T = warp_rows ? 32 : static_cast<int>(blockDim.x);
    const int tid = warp_rows ? static_cast<int>(lane_index()) : static_cast<int>(threadIdx.x);
    const long long m = warp_rows
                            ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp_index()
                            : static_cast<long long>(blockIdx.x);
    if (m >= p.M || !in_bounds(m >= 0 && p.K > 0, p.status, SITE_BOUNDS_A))
        return;
    const uint8_t *row = static_cast<const uint8_t *>(p.X) + m * p.ld_x * kB;
    const int steps = HELD ? kN : (p.K + T * VEC - 1) / (T * VEC);
    float v[kN][VEC];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = (i * T + tid) * VEC;
        if (e < p.K) {
            load_vec<KIND, VEC>(row, e, v[HELD ? i : 0]);
            amax = max_abs(amax, v[HELD ? i : 0]);
        }
    }
    const float s = int8_scale(row_reduce<Max>(amax, part, warp_rows));
#pragma unroll
    for (int i = 0; i < (HELD ? kN : steps); ++i) {
        const int e = (i * T + tid) * VEC;
        if (e < p.K) {
            if (!HELD)
                load_vec<KIND, VEC>(row, e, v[0]);
            store_int8<VEC>(p.A + m * p.ld_a + e, v[HELD ? i : 0], s);
        }
    }
    if (tid == 0)
        p.a_s[m] = s;
}

// Threads of a row's CTA: enough for kPer elements each, whole warps.
int row_threads(long long n)
{
    const long long t = (n + kPer - 1) / kPer;
    return static_cast<int>(std::min<long long>(kMaxThreads, (t + 31) / 32 * 32));
}

w8a8_status cuda_error(const char *what, cudaError_t e)
{
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return record_error(W8A8_ERR_CUDA, msg);
}

template <typename Params>
cudaError_t launch_rows(void (*kernel)(Params), const Params &p, long long rows, int T, size_t smem,
                        cudaStream_t stream)
{
    const int per_cta = T == 32 ? 4 : 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta), 1, 1);
    lc.blockDim = dim3(T == 32 ? 128 : T, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

bool on(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int HK, int XK, int VEC>
cudaError_t launch_norm(NormParams p, cudaStream_t stream)
{
    if (p.D <= kRegRow) {
        p.row_threads = row_threads(p.D);
        return launch_rows(p.row_threads <= kEarlyThreads ? k_sandwich_norm<HK, XK, VEC, true, true>
                                                          : k_sandwich_norm<HK, XK, VEC, true, false>,
                           p, p.M, p.row_threads, 0, stream);
    }
    static volatile int smem_set[kMaxDeviceFlags] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDeviceFlags))
        e = cudaErrorInvalidDevice;
    if (e == cudaSuccess && !smem_set[dev]) {
        e = cudaFuncSetAttribute(k_sandwich_norm<HK, XK, VEC, false, false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, W8A8_NORM_MAX_D * 4);
        smem_set[dev] = e == cudaSuccess;
    }
    if (e != cudaSuccess)
        return e;
    p.row_threads = kMaxThreads;
    return launch_rows(k_sandwich_norm<HK, XK, VEC, false, false>, p, p.M, kMaxThreads,
                       static_cast<size_t>(p.D) * 4, stream);
}

// Long rows in number: the ring.  Threads of a CTA take 16 columns each; as many
// CTAs per SM as their registers allow (three of 256 threads: 80 registers
// each), and stages that fill the SM's shared memory between them.
template <int HK, int XK, int THREADS, int PER_SM, bool FULL>
cudaError_t launch_ring_t(RingParams &r, const DeviceView &dev, cudaStream_t stream)
{
    constexpr int kRoom = 220 * 1024;
    auto kernel = k_sandwich_ring<HK, XK, THREADS, PER_SM, FULL>;
    const int T = row_threads(r.n.D);
    const int per_sm = std::min(24, std::max(1, PER_SM * THREADS / T));
    r.h_bytes = static_cast<uint32_t>(r.n.D) * (HK == W8A8_IN_FP32 ? 4 : 2);
    r.x_bytes = static_cast<uint32_t>(r.n.D) * (XK == W8A8_IN_FP32 ? 4 : 2);
    const size_t stage = r.h_bytes + r.x_bytes, weights = r.n.w_pre ? 64 * T : 0;
    const size_t room = kRoom / per_sm - 2048 - weights;
    r.stages = static_cast<int>(std::min<size_t>(kRingMaxStages, room / stage));
    static volatile int smem_set[kMaxDeviceFlags] = {};
    int id = 0;
    cudaError_t e = cudaGetDevice(&id);
    if (e == cudaSuccess && !smem_set[id]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
        smem_set[id] = e == cudaSuccess;
    }
    if (e != cudaSuccess)
        return e;
    const long long ctas = std::min<long long>(r.n.M, static_cast<long long>(per_sm) * dev.sm_count);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    lc.blockDim = dim3(T, 1, 1);
    lc.dynamicSmemBytes = r.stages * stage + weights;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, r);
}

template <int HK, int XK, int THREADS, int PER_SM>
cudaError_t launch_flat_t(const NormParams &p, const DeviceView &dev, cudaStream_t stream)
{
    auto kernel = k_sandwich_flat<HK, XK, THREADS, PER_SM>;
    constexpr int kWeights = 2 * 16 * (THREADS + 2) * 4;
    static volatile int smem_set[kMaxDeviceFlags] = {};
    int id = 0;
    cudaError_t e = cudaGetDevice(&id);
    if (e == cudaSuccess && (id < 0 || id >= kMaxDeviceFlags))
        e = cudaErrorInvalidDevice;
    if (e == cudaSuccess && !smem_set[id]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWeights);
        smem_set[id] = e == cudaSuccess;
    }
    if (e != cudaSuccess)
        return e;
    const int T = row_threads(p.D + 7);     // a row's shift takes up to seven elements more
    FlatParams f = {};
    f.n = p;
    f.inv_d = 1.f / static_cast<float>(p.D);
    const int per_sm = PER_SM * THREADS / T;
    const long long ctas = std::min<long long>(p.M, static_cast<long long>(per_sm) * dev.sm_count);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    lc.blockDim = dim3(T, 1, 1);
    lc.dynamicSmemBytes = kWeights;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, f);
}

template <int HK, int XK>
cudaError_t launch_norm(const NormParams &p, bool vec, const DeviceView &dev, cudaStream_t stream)
{
    // Rows off 16-byte boundaries: the flat kernel where the tensors are dense and
    // single elements would make narrow accesses (flat against direct, bf16: one row
    // of 1537 3.8 / 4.8 us, 1111 rows 6.6 / 10.4; 1111 of 513 5.3 / 4.9, 16384 26 / 86;
    // 4096 of 3943 31 / 151, of 301 14.5 / 8.6; 304 of 15001 20 / 37; fp32: 2000 rows of
    // 8001 60 / 71, 100 6.7 / 5.0; 4096 of 3943 65 / 60, of 2001 45 / 30).
    const int span = p.D + 7;
    const bool wide = HK == W8A8_IN_FP32 ? p.D > 4096 && p.M >= 2 * dev.sm_count : p.D >= 512;
    if (!vec && wide && span <= kRegRow && p.ld_h == p.D &&
        p.ld_x == p.D && p.ld_xo == p.D && p.ld_y == p.D && on(p.h, 16) && on(p.x, 16) &&
        on(p.x_out, 16) && on(p.y, p.y_kind == W8A8_NORM_SAME ? 16 : 8)) {
        if (span <= 16 * 128)
            return launch_flat_t<HK, XK, 128, 6>(p, dev, stream);
        if (span <= 16 * 256)
            return launch_flat_t<HK, XK, 256, 3>(p, dev, stream);
        if (span <= 16 * 512)
            return launch_flat_t<HK, XK, 512, 1>(p, dev, stream);
        return launch_flat_t<HK, XK, 1024, 1>(p, dev, stream);
    }
    // The ring where each of its CTAs gets several rows, and rows are long
    // enough to be worth a CTA (16384 rows of 768 to FP8: 26 against 33 us; of 512
    // 19.5 against 18.9, of 256 14 against 10).
    if (vec && p.D >= 640 && p.D <= 16 * kRingThreads &&
        p.M >= 2ll * dev.sm_count * std::min(24, std::max(1, 768 * 16 / p.D))) {
        RingParams r = {};
        r.n = p;
        r.inv_d = 1.f / static_cast<float>(p.D);
        r.wait_limit = dev.wait_limit;
        // whole warps of 16 columns a thread, 32-byte rows out
        constexpr int kHB = HK == W8A8_IN_FP32 ? 4 : 2, kXB = XK == W8A8_IN_FP32 ? 4 : 2;
        const bool full = p.D % 512 == 0 && on(p.x_out, 32) && p.ld_xo * kXB % 32 == 0 &&
                          (p.y_kind != W8A8_NORM_SAME || (on(p.y, 32) && p.ld_y * kHB % 32 == 0));
        if (p.D <= 16 * 256)
            return full ? launch_ring_t<HK, XK, 256, 3, true>(r, dev, stream)
                        : launch_ring_t<HK, XK, 256, 3, false>(r, dev, stream);
        return full ? launch_ring_t<HK, XK, kRingThreads, 1, true>(r, dev, stream)
                    : launch_ring_t<HK, XK, kRingThreads, 1, false>(r, dev, stream);
    }
    return vec ? launch_norm<HK, XK, 8>(p, stream) : launch_norm<HK, XK, 1>(p, stream);
}

template <int KIND> cudaError_t launch_quant(QuantParams p, bool vec, cudaStream_t stream)
{
    const bool held = p.K <= kRegRow;
    p.row_threads = row_threads(p.K);
    void (*kernel)(QuantParams) =
        vec ? (held ? k_quant_int8<KIND, 8, true> : k_quant_int8<KIND, 8, false>)
            : (held ? k_quant_int8<KIND, 1, true> : k_quant_int8<KIND, 1, false>);
    return launch_rows(kernel, p, p.M, p.row_threads, 0, stream);
}

}  // namespace
}  // namespace w8a8

extern "C" w8a8_status w8a8_sandwich_norm(const void *h_dev, w8a8_in_dtype h_dtype, int64_t ld_h,
                                          const void *x_dev, w8a8_in_dtype x_dtype, int64_t ld_x,
                                          const void *w_post_dev, const void *gate_dev,
                                          int64_t gate_rows, const void *w_pre_dev,
                                          float res_scale, float eps, void *x_out_dev,
                                          int64_t ld_xo, void *y_dev, float *scales_dev,
                                          w8a8_norm_out y_kind, int64_t ld_y, int64_t M, int64_t D,
                                          w8a8_stream_t stream)
{
    using namespace w8a8;
    if (M < 0 || D < 0)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size");
    if (h_dtype < W8A8_IN_BF16 || h_dtype > W8A8_IN_FP32 || x_dtype < W8A8_IN_BF16 ||
        x_dtype > W8A8_IN_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown input dtype");
    if (y_kind < W8A8_NORM_SAME || y_kind > W8A8_NORM_INT8)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown form of y");
    if (x_dtype != h_dtype && x_dtype != W8A8_IN_FP32)
        return record_error(W8A8_ERR_UNSUPPORTED, "x must have h's type or fp32");
    if (gate_dev && gate_rows < 1)
        return record_error(W8A8_ERR_INVALID_ARG, "gate_rows must be positive");
    ld_h = ld_h ? ld_h : D;
    ld_x = ld_x ? ld_x : D;
    ld_xo = ld_xo ? ld_xo : D;
    ld_y = ld_y ? ld_y : D;
    if (ld_h < D || ld_x < D || ld_xo < D || ld_y < D)
        return record_error(W8A8_ERR_INVALID_ARG, "a row stride is shorter than its row");
    if (M == 0 || D == 0)
        return W8A8_OK;
    if (!h_dev || !x_dev || !y_dev || (y_kind != W8A8_NORM_SAME && !scales_dev))
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (M > (1ll << 31) - 1 || D > W8A8_NORM_MAX_D)
        return record_error(W8A8_ERR_UNSUPPORTED, "M of 2^31 or more, or D above W8A8_NORM_MAX_D");
    const int hb = h_dtype == W8A8_IN_FP32 ? 4 : 2, xb = x_dtype == W8A8_IN_FP32 ? 4 : 2;
    const int yb = y_kind == W8A8_NORM_SAME ? hb : 1;
    if (!on(h_dev, hb) || !on(w_post_dev, hb) || !on(gate_dev, hb) || !on(w_pre_dev, hb) ||
        !on(x_dev, xb) || !on(x_out_dev, xb) || !on(y_dev, yb) || !on(scales_dev, 4))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    // Eight elements at a time where every row of every tensor allows it
    // (y's eight INT8 or E4M3 codes are one 8-byte store), else one.
    const bool vec = D % 8 == 0 && on(h_dev, 16) && on(x_dev, 16) && on(w_post_dev, 16) &&
                     on(gate_dev, 16) && on(w_pre_dev, 16) && on(x_out_dev, 16) &&
                     on(y_dev, yb == 1 ? 8 : 16) && ld_h * hb % 16 == 0 && ld_x * xb % 16 == 0 &&
                     (!x_out_dev || ld_xo * xb % 16 == 0) && ld_y * yb % (yb == 1 ? 8 : 16) == 0;
    if (y_kind == W8A8_NORM_FP8 && (!vec || D < 16 || D % 16 != 0))
        return record_error(W8A8_ERR_UNSUPPORTED, "FP8 codes need D to be a multiple of 16, rows of h, x "
                                                  "and x_out on 16-byte boundaries and of y on 8-byte ones");
    NormParams p = {};
    p.h = h_dev;
    p.x = x_dev;
    p.w_post = w_post_dev;
    p.gate = gate_dev;
    p.w_pre = w_pre_dev;
    p.x_out = x_out_dev;
    p.y = y_dev;
    p.scales = scales_dev;
    p.M = M;
    p.D = static_cast<int>(D);
    p.ld_h = ld_h;
    p.ld_x = ld_x;
    p.ld_xo = ld_xo;
    p.ld_y = ld_y;
    p.gate_rows = gate_rows;
    p.res_scale = res_scale;
    p.eps = eps;
    p.y_kind = y_kind;
    DeviceView dev;
    if (const int st = device_view(&dev); st != W8A8_OK)
        return static_cast<w8a8_status>(st);
    p.status = dev.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (h_dtype == W8A8_IN_FP32)
        e = launch_norm<W8A8_IN_FP32, W8A8_IN_FP32>(p, vec, dev, s);
    else if (h_dtype == W8A8_IN_BF16)
        e = x_dtype == W8A8_IN_FP32 ? launch_norm<W8A8_IN_BF16, W8A8_IN_FP32>(p, vec, dev, s)
                                    : launch_norm<W8A8_IN_BF16, W8A8_IN_BF16>(p, vec, dev, s);
    else
        e = x_dtype == W8A8_IN_FP32 ? launch_norm<W8A8_IN_FP16, W8A8_IN_FP32>(p, vec, dev, s)
                                    : launch_norm<W8A8_IN_FP16, W8A8_IN_FP16>(p, vec, dev, s);
    return e == cudaSuccess ? W8A8_OK : cuda_error("kernel launch", e);
}

extern "C" w8a8_status w8a8_quantize_int8_per_token(const void *X_dev, w8a8_in_dtype x_dtype,
                                                    int64_t ld_x, void *A_dev, int64_t ld_a,
                                                    float *a_s_dev, int64_t M, int64_t K,
                                                    w8a8_stream_t stream)
{
    using namespace w8a8;
    if (M < 0 || K < 0)
        return record_error(W8A8_ERR_INVALID_ARG, "negative size");
    if (x_dtype < W8A8_IN_BF16 || x_dtype > W8A8_IN_FP32)
        return record_error(W8A8_ERR_INVALID_ARG, "unknown input dtype");
    ld_x = ld_x ? ld_x : K;
    ld_a = ld_a ? ld_a : K;
    if (ld_x < K || ld_a < K)
        return record_error(W8A8_ERR_INVALID_ARG, "a row stride is shorter than its row");
    if (M == 0 || K == 0)
        return W8A8_OK;
    if (!X_dev || !A_dev || !a_s_dev)
        return record_error(W8A8_ERR_INVALID_ARG, "null pointer argument");
    if (M > (1ll << 31) - 1 || K > (1ll << 30))
        return record_error(W8A8_ERR_UNSUPPORTED, "M of 2^31 or more, or K above 2^30");
    const int xb = x_dtype == W8A8_IN_FP32 ? 4 : 2;
    if (!on(X_dev, xb) || !on(a_s_dev, 4))
        return record_error(W8A8_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
    const bool vec = K % 8 == 0 && on(X_dev, 16) && on(A_dev, 8) && ld_x * xb % 16 == 0 && ld_a % 8 == 0;
    QuantParams p = {};
    p.X = X_dev;
    p.A = static_cast<uint8_t *>(A_dev);
    p.a_s = a_s_dev;
    p.M = M;
    p.K = static_cast<int>(K);
    p.ld_x = ld_x;
    p.ld_a = ld_a;
    if (W8A8_DEBUG_BOUNDS && status_word_address(&p.status) != cudaSuccess)
        p.status = nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = x_dtype == W8A8_IN_BF16   ? launch_quant<W8A8_IN_BF16>(p, vec, s)
                          : x_dtype == W8A8_IN_FP16 ? launch_quant<W8A8_IN_FP16>(p, vec, s)
                                                    : launch_quant<W8A8_IN_FP32>(p, vec, s);
    return e == cudaSuccess ? W8A8_OK : cuda_error("kernel launch", e);
}
