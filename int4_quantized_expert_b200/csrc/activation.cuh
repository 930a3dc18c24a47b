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

// 1 / (1 + exp(-z)) with the hardware exponential and division: a few ulps of
// fp32.  For z below about -88 exp overflows to infinity and the result is 0.
__device__ __forceinline__ float sigmoid_fast(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2), from which
// the density is e / sqrt(2 pi).  With x = |z| / sqrt(2),
//   erfc(x) = (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) exp(-x^2),  t = 1 / (1 + p x)
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: absolute
// error below 1.5e-7), and Phi = erfc(x) / 2 for z < 0, 1 - erfc(x) / 2 above.
// CUDA's erff costs about three times the instructions, which a tile's
// epilogue does not hide at short contraction lengths; the error here is far
// below the bf16 step the result is rounded to.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float x = fabsf(z) * 0.70710678f;
    e = __expf(-0.5f * z * z);
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float half_erfc = 0.5f * q * t * e;
    return z < 0.0f ? half_erfc : 1.0f - half_erfc;
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
        for (int i = 0; i < N; ++i) {
            float e;
            v[i] *= normal_cdf(v[i], e);
        }
    }
}

__device__ __forceinline__ float act_slope(int act, float z) {
    if (act == MOE_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == MOE_ACT_SILU) {
        const float s = sigmoid_fast(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if (act == MOE_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z * 0.39894228f, e, c);
    }
    return 1.0f;
}

}  // namespace moe
