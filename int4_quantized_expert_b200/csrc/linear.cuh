// Matrix products with bf16 weights (linear, grouped linear, their gradients)
// and SwiGLU rows: host interface of the kernels in linear.cu and swiglu.cu.
#pragma once

#include "common.cuh"

namespace moe {

// out[col][lane] of one launch:
//   LIN_FWD  y[r][n]     = sum_k x[r][k] W[e][n][k]      lanes n, columns rows r of expert e
//   LIN_DX   dx[r][k]    = sum_n dy[r][n] W[e][n][k]     lanes k, columns rows r of expert e
//   LIN_DW   dw[e][n][k] = sum_r dy[r][n] x[r][k]        lanes k, columns n
enum LinMode : int32_t { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

struct LinParams {
    const int32_t* offsets;   // [E + 1] row ranges, or NULL: one matrix, all rows
    int32_t E;
    int32_t rows;             // rows of x / dy / y
    int32_t F;                // output features (lanes): N, K, K by mode
    int32_t C;                // contraction length: K, N, (rows of the expert)
    int32_t NC;               // LIN_DW: columns N
    int32_t n_fblocks;        // ceil(F / 128)
    int32_t bn;               // most columns of a tile: 16 to 320
    int32_t chunks;           // chunks of the rows when there are no offsets
    int32_t box;              // rows of a TMA box of B (LIN_DW: 64 columns n of each of 64 rows)
    int32_t stages;           // slots of the operand ring
    int32_t ring_bytes;       // its size
    int32_t tmem_cols;        // tensor memory columns
    int32_t split;            // CTAs (pairs) of a cluster that share a tile's contraction
    void* out;
    int32_t out_fp32;
    int32_t act;              // moe_activation (LIN_FWD)
    const bf16* bias;         // [F] or NULL
    const bf16* residual;     // [rows, F] or NULL
    bf16* preact;             // [rows, F] or NULL
};

// a: W [E, N, K] (LIN_FWD, LIN_DX) or x [rows, K] (LIN_DW); b: x or dy
moe_status launch_linear(int mode, const bf16* a, const bf16* b, int32_t N, int32_t K, LinParams prm,
                         cudaStream_t stream);

// dz = dy * act'(z) (written when dz is given) and dbias = sum of the rows of dz
moe_status launch_act_grad(const bf16* dy, const bf16* z, int32_t T, int32_t N, int32_t act, bf16* dz, void* dbias,
                           int32_t dbias_fp32, cudaStream_t stream);

moe_status launch_swiglu(const bf16* gu, int32_t n, int32_t F, bf16* h, cudaStream_t stream);
moe_status launch_swiglu_backward(const bf16* dh, const bf16* gu, int32_t n, int32_t F, bf16* dgu,
                                  cudaStream_t stream);

moe_status set_wait_limit_linear(uint32_t cycles);
// Takes the current device's status word, leaving it clear (synchronizes `stream`).
moe_status linear_device_status(cudaStream_t stream);

}  // namespace moe
