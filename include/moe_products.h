/*
 * moe_products.h -- C ABI of the matrix products that run next to the 4-bit
 * layer of moe_w4a16.h (GB300, sm_103a): experts held in 16 bits, with the
 * gradients that tuning them takes, and projections or experts held in FP8 with
 * one scale per block, with the quantisation that feeds them.
 *
 * Conventions as in moe_w4a16.h: device pointers owned by the caller, no
 * allocation, no synchronisation, `stream` a cudaStream_t passed as void*,
 * return values from moe_status.  Strides count elements; the innermost
 * dimension of every matrix is contiguous.
 *
 * Groups.  Rows of one expert are consecutive: expert e has the rows
 * [offsets[e], offsets[e + 1]) of the row matrices (x, dy, outputs by row),
 * offsets int32 [num_experts + 1] on the device, not decreasing, inside
 * [0, rows].  An expert may have no rows.  Rows that no expert has are not read
 * and not written.  Offsets that break the rule never lead to an access outside
 * the arguments; the workspace's status then holds MOE_ERR_INVALID and the
 * outputs of the experts concerned are unspecified.
 *
 * Workspace.  MOE_PRODUCTS_WORKSPACE_BYTES, 256-byte aligned, its first
 * MOE_PRODUCTS_WORKSPACE_HEAD_BYTES zeroed by the caller once before its first
 * use and left alone after that; one workspace
 * serves any sequence of calls on one stream (calls that may run at the same
 * time need one each).  Its first word is the device status that
 * moe_get_status reads and clears.
 *
 * Layouts.  Any sizes and strides are computed; outputs must not overlap inputs.  The tensor-core kernels take
 * operands whose base addresses and strides are multiples of 16 bytes (see each
 * function); others run a plain kernel at a small fraction of the speed.
 */
#ifndef MOE_PRODUCTS_H
#define MOE_PRODUCTS_H

#include <stdint.h>

#include "moe_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_dtype { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

#define MOE_PRODUCTS_WORKSPACE_BYTES ((int64_t)48 << 20)
#define MOE_PRODUCTS_WORKSPACE_HEAD_BYTES 8192

/* y[r] = W[e] x[r] for every row r of expert e.
 *   dtype   MOE_BF16 or MOE_FP16: the type of x, w and out
 *   x       [rows, K], row stride x_stride >= K
 *   w       [num_experts, N, K], strides w_stride_e, w_stride_n >= K
 *   out     [rows, N], row stride out_stride >= N
 * Sums are fp32, rounded once to dtype.  num_experts 1..1024, N, K >= 1,
 * 0 <= rows < 2^31 - 1024 (0 is a no-op).  Tensor cores: x, w and out on 16-byte
 * boundaries, every stride a multiple of 8. */
int moe_grouped_mm(int dtype, const void* x, int64_t x_stride, const void* w, int64_t w_stride_e,
                   int64_t w_stride_n, const int32_t* offsets, int num_experts, int rows, int N, int K,
                   void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes, void* stream);

/* The gradient by the rows: dx[r] = W[e]^T dy[r].  dy [rows, N], dx [rows, K];
 * otherwise as moe_grouped_mm. */
int moe_grouped_mm_dx(int dtype, const void* dy, int64_t dy_stride, const void* w, int64_t w_stride_e,
                      int64_t w_stride_n, const int32_t* offsets, int num_experts, int rows, int N, int K,
                      void* dx, int64_t dx_stride, void* workspace, int64_t workspace_bytes, void* stream);

/* The gradient by the weights: dW[e] = sum over the rows r of e of dy[r] x[r]^T,
 * zero for an expert without rows.
 *   dw          [num_experts, N, K], strides dw_stride_e, dw_stride_n >= K, of
 *               type dw_dtype: dtype or MOE_FP32
 *   accumulate  0: dw is written; 1 (MOE_FP32 only): the gradient is added to it
 *               (values below 2^-126 may count as zeros there; the part of an
 *               expert without rows is left as it is)
 * The same inputs give the same bits. */
int moe_grouped_mm_dw(int dtype, const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                      const int32_t* offsets, int num_experts, int rows, int N, int K, int dw_dtype,
                      int accumulate, void* dw, int64_t dw_stride_e, int64_t dw_stride_n, void* workspace,
                      int64_t workspace_bytes, void* stream);

/* FP8 blocks of 1 x 128: row r of the output quantises
 *   v = x[row_index ? row_index[r] : r]                       [K]      (gated 0)
 *   v = silu(g) * u, g = the first K values of the row, u the next K   (gated 1)
 * with, per block of 128 columns (the last may be shorter),
 *   s = max(max |v| / 448, 2^-126),  q = e4m3(v * (1 / s)),
 * each operation rounded to fp32, q to nearest even; silu(g) = g / (1 + exp(-g)),
 * 0 below g = -88.72, where exp(-g) passes the largest fp32 number.
 * A NaN or an infinity in a block makes s a NaN or an infinity, so
 * the block's values q * s are not finite.
 *   dtype   MOE_BF16 or MOE_FP16: the type of x [x_rows, K or 2K], row stride
 *           x_stride
 *   row_index int32 [rows], or NULL (then rows == x_rows); an index outside
 *           [0, x_rows) makes a row of zeros
 *   q       uint8 E4M3 [rows, K], row stride q_stride >= K
 *   scale   fp32: the scale of row r, block b at scale[r * scale_stride_m + b *
 *           scale_stride_g]
 * rows == 0 is a no-op. */
int moe_quant_fp8_block(int dtype, const void* x, int64_t x_stride, int x_rows, const int32_t* row_index,
                        int rows, int K, int gated, void* q, int64_t q_stride, float* scale,
                        int64_t scale_stride_m, int64_t scale_stride_g, void* stream);

/* The product of block-scaled FP8 operands:
 *   y[r, n] = sum over blocks b of 128 columns of
 *             xs[r, b] * ws[e, n / 128, b] * sum_{k in b} x[r, k] w[e, n, k]
 * over the rows r of expert e, or with offsets == NULL (num_experts == 1) over
 * all rows.
 *   x       uint8 E4M3 [rows, K], row stride x_stride >= K
 *   x_scale fp32, entry (r, b) at x_scale[r * xs_stride_m + b * xs_stride_g]
 *   w       uint8 E4M3 [num_experts, N, K], strides w_stride_e, w_stride_n >= K
 *   w_scale fp32, entry (e, n / 128, b) at w_scale[e * ws_stride_e + (n / 128) *
 *           ws_stride_n + b * ws_stride_k]
 *   out     [rows, N] of type out_dtype (MOE_BF16, MOE_FP16 or MOE_FP32), row
 *           stride out_stride >= N
 * Each block's sum and the sum over blocks are fp32, rounded once to out_dtype.
 * rows == 0 is a no-op.  Tensor cores: x and w on 16-byte boundaries with strides
 * multiples of 16, out on a 16-byte boundary with a stride multiple of 16 bytes. */
int moe_gemm_fp8_block(const void* x, int64_t x_stride, const float* x_scale, int64_t xs_stride_m,
                       int64_t xs_stride_g, const void* w, int64_t w_stride_e, int64_t w_stride_n,
                       const float* w_scale, int64_t ws_stride_e, int64_t ws_stride_n, int64_t ws_stride_k,
                       const int32_t* offsets, int num_experts, int rows, int N, int K, int out_dtype,
                       void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes, void* stream);

/* Calls that are captured into a CUDA graph.  A replay runs on whatever stream it is
 * launched on, so a captured call takes a workspace that no call outside the graph
 * uses, one for each stream of the capture, kept until the graph is gone.  These
 * tell the owner of workspaces what that takes.
 *
 * The capture that `stream` is in: its number into *id (never used again in the
 * process), 0 if it is in none. */
int moe_capture_id(void* stream, uint64_t* id);

/* Exchanges the calling thread's capture interaction mode (cudaStreamCaptureMode) with
 * *mode: in mode 2, relaxed, a thread that captures may allocate, and zero and wait
 * for a workspace on a stream outside the capture. */
int moe_capture_mode(int* mode);

/* A word on the host that is 0 and becomes 1 once the graph that `stream` is being
 * captured into and every executable graph made of it are gone and their replays
 * have finished.  The word is never freed. */
int moe_capture_watch(void* stream, const int32_t** gone);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PRODUCTS_H */
