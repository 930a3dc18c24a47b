// Activations and their derivatives in fp32, and bf16 pieces of rows (linear.cu, swiglu.cu).
#pragma once

#include "common.cuh"
#include "moe_linear.h"

namespace moe {

// Eight bf16 values of a 16-byte piece of a row.
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(w[i]); f[2 * i + 1] = bf16_hi(w[i]); }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// 2^x, 1 / x: the hardware's approximations (relative errors 2^-22 and 2^-23),
// results below 2^-126 flushed to 0, without the instructions that would keep them.
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two fp32 values at a time
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 / (1 + exp(-z)), off by less than 2^-17 of itself: the power of two's exponent
// is rounded to fp32, by 2^-18 at |z| = 88 and 2^-21 at 8.  Below 2^-126 (z < -87.3)
// the result is 0.
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_ftz(1.0f + ex2_ftz(-1.44269504f * z)); }

// h = Phi(-|z|), the normal distribution function, as 2^(-z^2 / (2 ln 2) + Q(|z|)):
//   Q(x) = log2(Phi(-x) exp(x^2 / 2))
// is smooth and flat (-1 at 0, near -log2(x sqrt(2 pi)) far out), and a polynomial
// of degree 8 gives it on [0, 13] to where z Phi(z) in fp32 is off by less than
// 2e-7 in absolute terms and 1.1e-3 of itself in the negative tail, where bf16
// rounds by up to 3.9e-3 (a minimax fit by linear programming, the error weighted
// by x Phi(-x) and bounded in the tail).  Beyond 13 the power is below 2^-126 and
// flushed to 0.  Degree 6 on [0, 5.5] is two instructions less for two values
// (4096 x 512 -> 16384, bound by its epilogue, takes 90 us and not 93), but off by
// 60 % of itself at -9.
__device__ __forceinline__ float2 normal_tail(float2 z, float2 s) {   // s = z^2
    const float2 x = make_float2(fminf(fabsf(z.x), 13.0f), fminf(fabsf(z.y), 13.0f));
    float2 q = fma2(both(4.58275622e-08f), x, both(-2.67672431e-06f));
    q = fma2(q, x, both(6.6674671e-05f));
    q = fma2(q, x, both(-0.000940348429f));
    q = fma2(q, x, both(0.00850551203f));
    q = fma2(q, x, both(-0.0539515316f));
    q = fma2(q, x, both(0.26291585f));
    q = fma2(q, x, both(-1.15129435f));
    q = fma2(q, x, both(-0.999985456f));
    q = fma2(s, both(-0.72134752f), q);
    return make_float2(ex2_ftz(q.x), ex2_ftz(q.y));
}

// z Phi(z) = max(z, 0) - |z| h.  The factor |z| is capped where h is 0 already,
// so that an infinite z gives infinity (or 0) and not infinity times 0.
__device__ __forceinline__ float2 gelu2(float2 z) {
    const float2 h = normal_tail(z, mul2(z, z));
    return fma2(make_float2(fmaxf(-fabsf(z.x), -32.0f), fmaxf(-fabsf(z.y), -32.0f)), h,
                make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f)));
}

// Phi(z) + z phi(z), phi(z) = e / sqrt(2 pi) with e = exp(-z^2 / 2), which the
// slope needs in any case.  With it the tail h = Phi(-|z|) is cheaper than by
// normal_tail (24 against 28 us for 4099 x 5120 values): with x = |z| / sqrt(2),
//   2 h = erfc(x) = (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) e,  t = 1 / (1 + p x)
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: absolute
// error below 1.5e-7).  The slope at -|z| is s = h - |z| phi(z), one product with
// e, and at |z| it is 1 - s: neither side loses its small values to a 1/2.  |z| is
// capped where e is 0 already, so that an infinite z gives 0 or 1.  In fp32 the
// slope is off by less than 3e-7, and by less than 3e-4 of itself for z below -1.
__device__ __forceinline__ float2 gelu_slope2(float2 z) {
    const float2 w = mul2(mul2(z, z), both(-0.72134752f)), e = make_float2(ex2_ftz(w.x), ex2_ftz(w.y));
    const float2 m = make_float2(fminf(fabsf(z.x), 32.0f), fminf(fabsf(z.y), 32.0f));
    const float2 d = fma2(m, both(0.3275911f * 0.70710678f), both(1.0f));
    const float2 t = make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
    float2 q = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
    q = fma2(q, t, both(0.5f * 1.421413741f));
    q = fma2(q, t, both(0.5f * -0.284496736f));
    q = fma2(q, t, both(0.5f * 0.254829592f));
    const float2 s = mul2(fma2(m, both(-0.39894228f), mul2(q, t)), e);   // NaN where z is: e is
    return make_float2(z.x < 0.0f ? s.x : 1.0f - s.x, z.y < 0.0f ? s.y : 1.0f - s.y);
}

// act of N values.  The choice is made once for all of them, so the code that
// is passed over is one jump away.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // keeps NaN
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= sigmoid_fast(v[i]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 y = gelu2(make_float2(v[i], v[i + 1]));
            v[i] = y.x;
            v[i + 1] = y.y;
        }
    }
}

// v *= act'(z) for N values
template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&v)[N], const float (&z)[N]) {
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = z[i] > 0.0f ? v[i] : 0.0f;
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = sigmoid_fast(z[i]);
            v[i] *= s * fmaf(z[i], 1.0f - s, 1.0f);
        }
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 d = gelu_slope2(make_float2(z[i], z[i + 1]));
            v[i] *= d.x;
            v[i + 1] *= d.y;
        }
    }
}

}  // namespace moe
