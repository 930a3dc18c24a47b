// SwiGLU on rows gu = [g | u]: h = silu(g) u, and its gradient ("Llama 开源模型
// 系列" (docs.ifdog.com), "SwiGLU：门控激活的数学").
//
// HBM-bound: 6 bytes (forward) and 10 bytes (backward) per hidden value, each
// read or written once, 16 bytes at a time; fp32 in between, one rounding.
#include "activation.cuh"
#include "linear.cuh"

namespace moe {

constexpr int SG_THREADS = 256;

template <bool BACKWARD>
__global__ void __launch_bounds__(SG_THREADS) swiglu_kernel(const bf16* __restrict__ gu, const bf16* __restrict__ dh,
                                                            int64_t n8, int F, bf16* __restrict__ out) {
    griddep_launch_dependents();
    griddep_wait();
    const int f8 = F / 8;
    for (int64_t i = blockIdx.x * int64_t(SG_THREADS) + threadIdx.x; i < n8; i += int64_t(gridDim.x) * SG_THREADS) {
        const int64_t r = i / f8;
        const int64_t gi = r * 2 * F + (i - r * f8) * 8;
        float g[8], u[8], a[8], b[8];
        unpack8(*reinterpret_cast<const uint4*>(gu + gi), g);
        unpack8(*reinterpret_cast<const uint4*>(gu + gi + F), u);
        if (BACKWARD) {
            float d[8];
            unpack8(*reinterpret_cast<const uint4*>(dh + i * 8), d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sigmoid_fast(g[j]);
                a[j] = d[j] * u[j] * (s * fmaf(g[j], 1.0f - s, 1.0f));
                b[j] = d[j] * (g[j] * s);
            }
            *reinterpret_cast<uint4*>(out + gi) = pack8(a);
            *reinterpret_cast<uint4*>(out + gi + F) = pack8(b);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = g[j] * sigmoid_fast(g[j]) * u[j];
            *reinterpret_cast<uint4*>(out + i * 8) = pack8(a);
        }
    }
}

namespace {

template <bool BACKWARD>
moe_status launch(const bf16* gu, const bf16* dh, int32_t n, int32_t F, bf16* out, cudaStream_t stream) {
    if (n == 0) return MOE_OK;
    const int64_t n8 = int64_t(n) * (F / 8);
    int64_t blocks = ceil_div(n8, SG_THREADS);
    if (blocks > 148 * 32) blocks = 148 * 32;
    return launch_pdl(swiglu_kernel<BACKWARD>, dim3(unsigned(blocks)), dim3(SG_THREADS), 0, stream, gu, dh, n8, F, out);
}

}  // namespace

moe_status launch_swiglu(const bf16* gu, int32_t n, int32_t F, bf16* h, cudaStream_t stream) {
    return launch<false>(gu, nullptr, n, F, h, stream);
}

moe_status launch_swiglu_backward(const bf16* dh, const bf16* gu, int32_t n, int32_t F, bf16* dgu,
                                  cudaStream_t stream) {
    return launch<true>(gu, dh, n, F, dgu, stream);
}

}  // namespace moe
