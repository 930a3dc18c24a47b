/*
 * moe_linear.h -- C ABI of libmoe_int4, second part: matrix products with
 * bf16 weights around and inside a mixture-of-experts layer, with their
 * gradients, for NVIDIA B200 (sm_100a):
 *
 *   moe_linear_*          a projection with bias, activation and residual
 *   moe_grouped_linear_*  one matrix per expert on rows sorted by expert
 *   moe_swiglu_*          the step between an expert's two products
 *
 * With moe_route these run (and train) the bf16 form of the routed experts,
 * before moe_quantize_int4 / moe_quantize_fp8_rows turn their weights into
 * what moe_ffn_forward takes ("1 卡跑通 Llama 4" (discosf.com), "FP8 / Int4
 * 混合量化"; "Llama 开源模型系列" (docs.ifdog.com), "SwiGLU：门控激活的数学").
 *
 * The conventions of moe_int4.h hold: device pointers of the current device,
 * 16-byte aligned; dense row-major matrices; weights stored "nt" ([out, in]);
 * nothing is allocated, kept or synchronized; argument errors return before
 * anything is launched; all work is enqueued in order on `stream`.  In
 * addition:
 *   - Outputs may not overlap inputs or one another, except that
 *     moe_linear_forward's y may be its residual.
 *   - A size of zero rows is allowed: there is nothing to do, except that
 *     weight and bias gradients are set to zero.
 *   - Results do not depend on timing: the same call gives the same bits.
 *   - The calls need no scratch, so calls on different streams may overlap.
 */
#ifndef MOE_LINEAR_H
#define MOE_LINEAR_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,   /* max(z, 0); the gradient at 0 is 0 */
    MOE_ACT_SILU = 2,   /* z / (1 + exp(-z)) */
    MOE_ACT_GELU = 3    /* z Phi(z), Phi the normal distribution function (the exact form) */
} moe_activation;
/*
 * Before the one rounding, values and slopes are off by less than 2^-20 (1 + |z|)
 * and, where z < -2, by less than 2^-9 of themselves (SiLU: 2^-16); what a factor
 * below 2^-126 makes is 0.  Infinite z: GELU and its slope take their limits;
 * SiLU (and SwiGLU) follow the formula in IEEE arithmetic, which gives NaN at
 * minus infinity and for the slope at both.
 */

/*
 * moe_linear_forward:
 *   z = x W^T + bias;   y = bf16(act(z) + residual)
 * with fp32 accumulation; z stays fp32 up to the one rounding of y.
 *   x  bf16 [T, K];  w  bf16 [N, K];  bias  bf16 [N] or NULL
 *   activation  a moe_activation
 *   residual  bf16 [T, N] or NULL (may be y itself)
 *   preact  bf16 [T, N] or NULL: receives bf16(z), which the backward pass
 *           needs with an activation
 *   y  bf16 [T, N]
 * Requires 0 <= T <= 1048576; K and N multiples of 8 in [8, 65536].
 */
MOE_API moe_status moe_linear_forward(const void* x, int32_t T, int32_t K, const void* w, int32_t N,
                                      const void* bias, int32_t activation, const void* residual, void* preact,
                                      void* y, void* stream);

/*
 * moe_linear_backward -- the gradients of moe_linear_forward:
 *   dz = dy * act'(preact);  dx = dz W;  dw = dz^T x;  dbias = sum_t dz[t]
 * (the residual's gradient is dy itself).  dz is computed in fp32; dbias sums
 * it unrounded, the products take it rounded to bf16: the tensor cores' operands
 * are bf16, and dz as a sum of two of them would double the operations.  With
 * normal inputs and GELU, dx and bf16 dw are then off by 2.3e-3 of their norms
 * (1.7e-3 from their own rounding), fp32 dw by 1.7e-3.
 *   dy  bf16 [T, N];  x  bf16 [T, K];  w  bf16 [N, K]
 *   preact  bf16 [T, N] as moe_linear_forward wrote it; not read when
 *           activation is MOE_ACT_NONE (NULL is fine there)
 *   dz  bf16 [T, N] (output): required with an activation when dx or dw is
 *       wanted; not written when activation is MOE_ACT_NONE (dy is dz)
 *   dx  bf16 [T, K], or NULL if not wanted (w is then not read)
 *   dw  [N, K] of grad_dtype, or NULL if not wanted (x is then not read)
 *   dbias  [N] of grad_dtype, or NULL if not wanted
 *   grad_dtype  MOE_DTYPE_BF16 or MOE_DTYPE_FP32
 * Sizes as in moe_linear_forward.
 */
MOE_API moe_status moe_linear_backward(const void* dy, const void* x, int32_t T, int32_t K, const void* w,
                                       int32_t N, int32_t activation, const void* preact, void* dz, void* dx,
                                       void* dw, void* dbias, int32_t grad_dtype, void* stream);

/*
 * moe_grouped_linear_forward -- one product per expert on rows sorted by
 * expert:
 *   y[r] = x[r] W[e]^T   for offsets[e] <= r < offsets[e + 1]
 * with fp32 accumulation.
 *   x  bf16 [n, K];  w  bf16 [E, N, K]
 *   offsets  int32 [E + 1] on the device, ascending, within 0 .. n, as
 *            moe_route writes them.  Experts may be empty.
 *   y  [n, N] of y_dtype (MOE_DTYPE_BF16 or MOE_DTYPE_FP32); rows before
 *      offsets[0] and from offsets[E] on are left as they were.
 * An expert whose two offsets are out of order or out of range, or whose range
 * overlaps an earlier expert's, is taken as empty and reported by
 * moe_linear_device_status; the other experts' results are as ever.
 * Requires 0 <= n <= 1048576; 1 <= E <= 256; K and N multiples of 8 in
 * [8, 65536].
 */
MOE_API moe_status moe_grouped_linear_forward(const void* x, int32_t n, int32_t K, const void* w, int32_t E,
                                              int32_t N, const int32_t* offsets, void* y, int32_t y_dtype,
                                              void* stream);

/*
 * moe_grouped_linear_backward -- its gradients:
 *   dx[r] = dy[r] W[e];   dw[e] = sum over the rows r of e of dy[r]^T x[r]
 *   dy  bf16 [n, N];  x  bf16 [n, K];  w  bf16 [E, N, K]
 *   dx  bf16 [n, K], or NULL if not wanted (w is then not read); rows outside
 *       offsets[0] .. offsets[E] are left as they were
 *   dw  [E, N, K] of dw_dtype, or NULL if not wanted (x is then not read);
 *       an empty expert's gradient is set to zero
 * Sizes and offsets as in moe_grouped_linear_forward.
 */
MOE_API moe_status moe_grouped_linear_backward(const void* dy, const void* x, int32_t n, int32_t K, const void* w,
                                               int32_t E, int32_t N, const int32_t* offsets, void* dx, void* dw,
                                               int32_t dw_dtype, void* stream);

/*
 * moe_swiglu_forward -- h = bf16(silu(g) * u) on rows gu = [g | u] ("SwiGLU：
 * 门控激活的数学"), in fp32 with one rounding.
 *   gu  bf16 [n, 2 F];  h  bf16 [n, F]
 * moe_swiglu_backward -- its gradient, with s = 1 / (1 + exp(-g)):
 *   dg = dh u s (1 + g (1 - s));   du = dh g s
 *   dh  bf16 [n, F];  gu  bf16 [n, 2 F];  dgu  bf16 [n, 2 F] = [dg | du]
 * Requires 0 <= n <= 1048576; F a multiple of 8 in [8, 65536].
 */
MOE_API moe_status moe_swiglu_forward(const void* gu, int32_t n, int32_t F, void* h, void* stream);
MOE_API moe_status moe_swiglu_backward(const void* dh, const void* gu, int32_t n, int32_t F, void* dgu,
                                       void* stream);

/*
 * moe_linear_device_status -- SYNCHRONIZES `stream`, then returns what the
 * kernels behind moe_linear_* and moe_grouped_linear_* reported on the
 * current device since the last such query, and clears it: MOE_OK,
 * MOE_ERR_TIMEOUT (a bounded device wait gave up; outputs are invalid; also
 * where offsets were reported as well), MOE_ERR_INVALID_ARG (offsets out of
 * order or out of range, or ranges that overlap) or MOE_ERR_CUDA.  One status
 * word per device serves every stream: a query takes what any stream reported,
 * and of queries at the same time one gets a report.  It lives in the library,
 * so nothing has to be passed or cleared.  Not to be called while `stream` is
 * being captured.
 */
MOE_API moe_status moe_linear_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LINEAR_H */
