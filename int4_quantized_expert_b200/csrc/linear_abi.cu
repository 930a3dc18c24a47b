// extern "C" entry points of include/moe_linear.h: argument checks and the
// stream-ordered launches of each operation.
#include "linear.cuh"
#include "moe_linear.h"

using namespace moe;

namespace {

constexpr int kMaxRows = 1 << 20;
constexpr int kMaxWidth = 65536;
constexpr int kMaxExperts = 256;

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

bool rows_ok(int32_t n) { return n >= 0 && n <= kMaxRows; }
bool width_ok(int32_t v) { return v >= 8 && v <= kMaxWidth && v % 8 == 0; }

// A buffer of a call: a null pointer is allowed when it is optional or empty.
struct Buf {
    const void* p;
    int64_t bytes;
    bool required, output;
};

template <int N>
moe_status check_buffers(const Buf (&b)[N]) {
    for (const Buf& x : b) {
        if (!x.p && x.required && x.bytes > 0) return MOE_ERR_INVALID_ARG;
        if (!aligned16(x.p)) return MOE_ERR_INVALID_ARG;
    }
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            if (i == j || !b[i].output || !b[i].p || !b[j].p) continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p), y = reinterpret_cast<uintptr_t>(b[j].p);
            if (x < y + uintptr_t(b[j].bytes) && y < x + uintptr_t(b[i].bytes)) return MOE_ERR_INVALID_ARG;
        }
    return MOE_OK;
}

const bf16* in(const void* p) { return static_cast<const bf16*>(p); }

}  // namespace

extern "C" {

moe_status moe_linear_forward(const void* x, int32_t T, int32_t K, const void* w, int32_t N, const void* bias,
                              int32_t activation, const void* residual, void* preact, void* y, void* stream) {
    if (!rows_ok(T) || !width_ok(K) || !width_ok(N)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
    const int64_t t = T, k = K, n = N;
    const Buf bufs[] = {{x, t * k * 2, true, false},
                        {w, n * k * 2, T > 0, false},
                        {bias, n * 2, false, false},
                        {residual == y ? nullptr : residual, t * n * 2, false, false},
                        {preact, t * n * 2, false, true},
                        {y, t * n * 2, true, true}};
    const moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    LinParams p = {};
    p.E = 1;
    p.rows = T;
    p.out = y;
    p.act = activation;
    p.bias = in(bias);
    p.residual = in(residual);
    p.preact = static_cast<bf16*>(preact);
    return launch_linear(LIN_FWD, in(w), in(x), N, K, p, as_stream(stream));
}

moe_status moe_linear_backward(const void* dy, const void* x, int32_t T, int32_t K, const void* w, int32_t N,
                               int32_t activation, const void* preact, void* dz, void* dx, void* dw, void* dbias,
                               int32_t grad_dtype, void* stream) {
    if (!rows_ok(T) || !width_ok(K) || !width_ok(N)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
    if (grad_dtype != MOE_DTYPE_BF16 && grad_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    const bool act = activation != MOE_ACT_NONE, fp32 = grad_dtype == MOE_DTYPE_FP32;
    const int64_t t = T, k = K, n = N, gb = fp32 ? 4 : 2;
    if (!act) preact = dz = nullptr;
    const Buf bufs[] = {{dy, t * n * 2, dx || dw || dbias, false},
                        {x, t * k * 2, dw != nullptr, false},
                        {w, n * k * 2, dx && T > 0, false},
                        {preact, t * n * 2, act && (dx || dw || dbias), false},
                        {dz, t * n * 2, act && (dx || dw), true},
                        {dx, t * k * 2, false, true},
                        {dw, n * k * gb, false, true},
                        {dbias, n * gb, false, true}};
    moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    cudaStream_t st = as_stream(stream);
    if (T == 0) {   // empty sums
        if (dw && cudaMemsetAsync(dw, 0, size_t(n * k * gb), st) != cudaSuccess) return MOE_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, size_t(n * gb), st) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dx && !dw) dz = nullptr;   // only the products read it
    if (dbias || dz) {
        s = launch_act_grad(in(dy), in(preact), T, N, activation, static_cast<bf16*>(dz), dbias, fp32, st);
        if (s != MOE_OK) return s;
    }
    const bf16* d = act ? static_cast<const bf16*>(dz) : in(dy);
    LinParams p = {};
    p.E = 1;
    p.rows = T;
    if (dx) {
        p.out = dx;
        s = launch_linear(LIN_DX, in(w), d, N, K, p, st);
        if (s != MOE_OK) return s;
    }
    if (dw) {
        p.out = dw;
        p.out_fp32 = fp32;
        s = launch_linear(LIN_DW, in(x), d, N, K, p, st);
    }
    return s;
}

moe_status moe_grouped_linear_forward(const void* x, int32_t n, int32_t K, const void* w, int32_t E, int32_t N,
                                      const int32_t* offsets, void* y, int32_t y_dtype, void* stream) {
    if (!rows_ok(n) || !width_ok(K) || !width_ok(N) || E < 1 || E > kMaxExperts) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (y_dtype != MOE_DTYPE_BF16 && y_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    const int64_t t = n, k = K;
    const bool fp32 = y_dtype == MOE_DTYPE_FP32;
    const Buf bufs[] = {{x, t * k * 2, true, false},
                        {w, int64_t(E) * N * k * 2, n > 0, false},
                        {offsets, (int64_t(E) + 1) * 4, true, false},
                        {y, t * N * (fp32 ? 4 : 2), true, true}};
    const moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    LinParams p = {};
    p.offsets = offsets;
    p.E = E;
    p.rows = n;
    p.out = y;
    p.out_fp32 = fp32;
    return launch_linear(LIN_FWD, in(w), in(x), N, K, p, as_stream(stream));
}

moe_status moe_grouped_linear_backward(const void* dy, const void* x, int32_t n, int32_t K, const void* w, int32_t E,
                                       int32_t N, const int32_t* offsets, void* dx, void* dw, int32_t dw_dtype,
                                       void* stream) {
    if (!rows_ok(n) || !width_ok(K) || !width_ok(N) || E < 1 || E > kMaxExperts) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (dw_dtype != MOE_DTYPE_BF16 && dw_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    const int64_t t = n, k = K, mats = int64_t(E) * N * k;
    const bool fp32 = dw_dtype == MOE_DTYPE_FP32;
    const Buf bufs[] = {{dy, t * N * 2, dx || dw, false},
                        {x, t * k * 2, dw != nullptr, false},
                        {w, mats * 2, dx && n > 0, false},
                        {offsets, (int64_t(E) + 1) * 4, true, false},
                        {dx, t * k * 2, false, true},
                        {dw, mats * (fp32 ? 4 : 2), false, true}};
    moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    cudaStream_t st = as_stream(stream);
    if (n == 0) {
        if (dw && cudaMemsetAsync(dw, 0, size_t(mats * (fp32 ? 4 : 2)), st) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    LinParams p = {};
    p.offsets = offsets;
    p.E = E;
    p.rows = n;
    if (dx) {
        p.out = dx;
        s = launch_linear(LIN_DX, in(w), in(dy), N, K, p, st);
        if (s != MOE_OK) return s;
    }
    if (dw) {
        p.out = dw;
        p.out_fp32 = fp32;
        s = launch_linear(LIN_DW, in(x), in(dy), N, K, p, st);
    }
    return s;
}

moe_status moe_swiglu_forward(const void* gu, int32_t n, int32_t F, void* h, void* stream) {
    if (!rows_ok(n) || !width_ok(F)) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t v = int64_t(n) * F;
    const Buf bufs[] = {{gu, v * 4, true, false}, {h, v * 2, true, true}};
    const moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    return launch_swiglu(in(gu), n, F, static_cast<bf16*>(h), as_stream(stream));
}

moe_status moe_swiglu_backward(const void* dh, const void* gu, int32_t n, int32_t F, void* dgu, void* stream) {
    if (!rows_ok(n) || !width_ok(F)) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t v = int64_t(n) * F;
    const Buf bufs[] = {{dh, v * 2, true, false}, {gu, v * 4, true, false}, {dgu, v * 4, true, true}};
    const moe_status s = check_buffers(bufs);
    if (s != MOE_OK) return s;
    return launch_swiglu_backward(in(dh), in(gu), n, F, static_cast<bf16*>(dgu), as_stream(stream));
}

moe_status moe_linear_device_status(void* stream) { return linear_device_status(as_stream(stream)); }

}  // extern "C"
