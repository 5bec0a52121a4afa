// Numbers as unevaluated sums of two fp32, of some 47 bits: T. J. Dekker, "A floating-point
// technique for extending the available precision", Numerische Mathematik 18, 1971; sums
// without a comparison after D. E. Knuth, "The Art of Computer Programming", vol. 2, 4.2.2.
// The fp64 units of a GB300 are few and slow (eight fp64 scores a lane took a warp 25 us), its
// fp32 units are not.
#pragma once

#include <stdint.h>

namespace w8a8 {

struct Pair32 {
    float h, l;             // |l| at most half a unit of h
};

__device__ __forceinline__ Pair32 two_sum(float a, float b)             // exact
{
    const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Pair32 join(float a, float b)                // exact for |a| >= |b|
{
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair32 operator+(Pair32 a, Pair32 b)         // off by 2^-46 of the sizes
{
    const Pair32 s = two_sum(a.h, b.h);
    return join(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair32 operator*(Pair32 a, Pair32 b)         // off by 2^-45 of the product
{
    const float p = __fmul_rn(a.h, b.h), e = __fmaf_rn(a.h, b.h, -p);
    return join(p, __fadd_rn(e, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}

// exp(x) for x <= 0; 0 below -80 (whose exponential is below 2^-115).  x is reduced by a
// multiple n of ln 2 in three parts, the first two of 15 bits, whose products with n are
// exact (after W. J. Cody and W. Waite, "Software Manual for the Elementary Functions", 1980); then
// the power series, from f^7 on in fp32: |f| < 0.35, so those terms are below 2^-22.
__device__ __forceinline__ Pair32 exp_pair(Pair32 x)
{
    if (!(x.h >= -80.f))
        return {x.h != x.h ? x.h : 0.f, 0.f};
    const float n = rintf(__fmul_rn(x.h, 1.44269504f));
    const Pair32 t = two_sum(x.h, __fmul_rn(n, -0x1.62e4p-1f));
    const Pair32 u = two_sum(t.h, __fmul_rn(n, -0x1.7f7cp-20f));
    const Pair32 f = join(u.h, __fadd_rn(__fadd_rn(t.l, u.l), __fmaf_rn(n, -0x1.1cf79ap-36f, x.l)));
    float q = 1.f / 39916800.f;
    q = __fmaf_rn(q, f.h, 1.f / 3628800.f);
    q = __fmaf_rn(q, f.h, 1.f / 362880.f);
    q = __fmaf_rn(q, f.h, 1.f / 40320.f);
    q = __fmaf_rn(q, f.h, 1.f / 5040.f);
    Pair32 s = {q, 0.f};
    s = s * f + Pair32{0x1.6c16c2p-10f, -0x1.27d27ep-35f};
    s = s * f + Pair32{0x1.111112p-7f, -0x1.ddddep-32f};
    s = s * f + Pair32{0x1.555556p-5f, -0x1.555556p-30f};
    s = s * f + Pair32{0x1.555556p-3f, -0x1.555556p-28f};
    s = s * f + Pair32{.5f, 0.f};
    s = s * f + Pair32{1.f, 0.f};
    s = s * f + Pair32{1.f, 0.f};
    const float scale = __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23);
    return {s.h * scale, s.l * scale};
}

// 1 / d for d from 1 to 2^20, from an approximation that is within 2^-22
__device__ __forceinline__ Pair32 inverse(Pair32 d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.h));
    const float p = __fmul_rn(d.h, r), low = __fmaf_rn(d.h, r, -p);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(1.f, p), low), __fmul_rn(d.l, r));
    return join(r, __fmul_rn(r, __fmaf_rn(e, e, e)));
}

__device__ __forceinline__ Pair32 sigmoid(float l)
{
    const Pair32 e = exp_pair({-fabsf(l), 0.f}), q = inverse(Pair32{1.f, 0.f} + e);
    return l >= 0.f ? q : e * q;
}

}  // namespace w8a8
