/*
 * gemm_f32_lm -- layer norm and the loss over a vocabulary, with their
 * gradients, on row-major matrices for NVIDIA GB300 (sm_103a): the last rows
 * of a language model, next to the products of gemm_f32.h and in the same
 * library.
 *
 * The rules of gemm_f32.h hold here too: caller-owned device pointers, every
 * call asynchronous on `stream` and never synchronising the host, return code
 * 0 or a negative GEMM_F32_E* code, nothing printed or thrown, device-side
 * failures read later through gemm_f32_status(), gemm_f32_last_kernel() and
 * gemm_f32_last_launches() for what the call launched.
 *
 * Types: matrices hold fp32 (GEMM_F32_TYPE_F32) or bfloat16
 * (GEMM_F32_TYPE_BF16) elements, with a row stride in elements of at least
 * the row's length.  Pointers are aligned to their element.  Row statistics,
 * losses and every sum are fp32; an output in bfloat16 is rounded once, from
 * its fp32 value.  Two matrices overlap when the address ranges from their
 * first to their last element do, so two column slices of one matrix overlap.
 *
 * Scratch: the library owns one scratch buffer per (device, stream), grown
 * with cudaMalloc (which synchronises the device) by the first call that
 * needs more, kept for the next calls and freed by gemm_f32_release().  A
 * call that is captured into a CUDA graph takes memory of the graph's own
 * instead, during the capture: no call before it is needed, replays run
 * beside any other call, and the memory comes back to the library when the
 * graph and what was instantiated from it are destroyed.  Host threads may
 * call on one stream: each call's kernels are queued together.  Where the
 * memory cannot be had the call returns GEMM_F32_ESCRATCH and launches
 * nothing.
 *
 * gemm_f32_last_kernel() names the kernel of a call's main pass: for the norms
 * "layer_norm_stream_kernel" or "layer_norm_grad_stream_kernel" (many rows),
 * "layer_norm_kernel" or "layer_norm_grad_kernel" (few rows, or rows too wide
 * for the others), "norm_columns_kernel" (gradient of no rows); for the losses
 * the kernel of the logits, "half_gemm_kernel" or, of few rows,
 * "few_gemm_kernel"; "memset" for the loss of no rows.
 *
 * Every sum is taken in a fixed order: the same call on the same inputs
 * gives the same bits.
 */
#ifndef GEMM_F32_LM_H
#define GEMM_F32_LM_H

#include <stddef.h>

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

enum gemm_f32_type {
    GEMM_F32_TYPE_F32 = 0,
    GEMM_F32_TYPE_BF16 = 1
};

/* Layer norm of each row of x (rows x width):
 *     mean = sum_d x_d / width
 *     rstd = 1 / sqrt(sum_d (x_d - mean)^2 / width + eps)
 *     y_d  = (x_d - mean) * rstd * weight_d + bias_d
 * x and y hold `type`, weight and bias (width elements) `weight_type`, which
 * is `type` or fp32.  weight may be NULL (1), bias may be NULL (0); mean and
 * rstd (rows fp32 values each, what the gradient needs) may be NULL.  y may
 * be x itself, with the same stride.  The variance is summed from the
 * centred values.  rows == 0 does nothing.
 * Returns 0, GEMM_F32_EINVAL (unknown type, width < 1, rows < 0, a stride
 * below width, eps negative or not finite, a null or misaligned pointer, y
 * overlapping x otherwise), GEMM_F32_EDEVICE or GEMM_F32_ELAUNCH. */
int gemm_f32_layer_norm(int type, int weight_type, long long rows, int width, const void* x,
                        long long ldx, const void* weight, const void* bias, float eps, void* y,
                        long long ldy, float* mean, float* rstd, gemm_f32_stream_t stream);

/* Gradients of gemm_f32_layer_norm for dy, the gradient of y.  With
 * hat_d = (x_d - mean) * rstd and g_d = dy_d * weight_d, per row:
 *     dx_d = rstd * (g_d - sum(g) / width - hat_d * sum(g * hat) / width)
 * and over the rows:
 *     dweight_d = sum dy_d * hat_d,   dbias_d = sum dy_d
 * mean and rstd are those of the forward call.  dx holds `type`, dweight and
 * dbias `weight_type`; each of the three may be NULL when it is not wanted.
 * dx may be dy or x itself, with the same stride.  rows == 0 writes zeros
 * into dweight and dbias.  Returns as gemm_f32_layer_norm, and
 * GEMM_F32_ESCRATCH. */
int gemm_f32_layer_norm_grad(int type, int weight_type, long long rows, int width, const void* dy,
                             long long lddy, const void* x, long long ldx, const void* weight,
                             const float* mean, const float* rstd, void* dx, long long lddx,
                             void* dweight, void* dbias, gemm_f32_stream_t stream);

enum gemm_f32_reduction {
    GEMM_F32_SUM = 0,
    GEMM_F32_MEAN = 1    /* divided by the number of rows that count (at least 1) */
};

/* Softmax cross entropy over a vocabulary:
 *     z = x w^T                 x: rows x width, w: vocab x width
 *     lse_t  = log sum_v exp(z_tv)
 *     loss_t = lse_t - z_t,targets[t],   0 where targets[t] == ignore_index
 *     total  = sum_t loss_t, divided for GEMM_F32_MEAN
 * The logits z are never stored: each tile of them leaves its row maxima and
 * sums of exponentials, which are joined per row.  x and w hold `type`; with
 * fp32 the products are computed from three-part bfloat16 splits of the
 * operands on the tensor cores, to about fp32's own rounding (an infinite
 * operand gives NaN).  targets are 32- or 64-bit integers (target_bits).  A
 * target outside [0, vocab) that is not ignore_index counts as ignored and
 * is reported by gemm_f32_status() as GEMM_F32_ETARGET.
 * loss (rows), lse (rows) and total (1) are fp32; each may be NULL.
 * rows == 0 sets total to 0.
 * Returns 0, GEMM_F32_EINVAL (unknown type, reduction or target_bits, a
 * negative size, width or vocab < 1 or above 2^31 - 257, a stride below
 * width, a null or misaligned pointer), GEMM_F32_ESCRATCH, GEMM_F32_EDEVICE or
 * GEMM_F32_ELAUNCH. */
int gemm_f32_vocab_loss(int type, long long rows, int width, int vocab, const void* x,
                        long long ldx, const void* w, long long ldw, const void* targets,
                        int target_bits, long long ignore_index, int reduction, float* loss,
                        float* lse, float* total, gemm_f32_stream_t stream);

/* The same with the gradients of grad_scale * total:
 *     g_tv = s * (exp(z_tv - lse_t) - [v == targets[t]]),  0 in ignored rows
 *     dx = g w,   dw = g^T x        (s = grad_scale, divided for GEMM_F32_MEAN)
 * dx (rows x width) and dw (vocab x width) hold `type`; either may be NULL.
 * Neither may overlap an input.  The logits are computed once, for a piece of
 * the rows at a time: of a piece the library keeps exp(z - maximum of its
 * tile) in scratch, in 16 bits for bfloat16 operands, and turns it into
 * g / s in place, rounded to bfloat16 (two parts of it with at most 32 rows,
 * three for fp32 operands).
 * `piece_bytes` bounds that part of the scratch (0: 4 GiB);
 * pieces are at least 256 rows.  With more than one piece and bfloat16
 * operands, dw is summed in fp32 scratch.  Besides the piece the scratch holds
 * what TMA cannot read where it lies: the three parts of fp32 operands (6 bytes
 * an element of x, and of w with more than 128 rows), copies of matrices whose
 * rows are not on 16-byte boundaries; and partial tiles of the products. */
int gemm_f32_vocab_loss_grad(int type, long long rows, int width, int vocab, const void* x,
                             long long ldx, const void* w, long long ldw, const void* targets,
                             int target_bits, long long ignore_index, int reduction,
                             float grad_scale, float* loss, float* lse, float* total, void* dx,
                             long long lddx, void* dw, long long lddw, size_t piece_bytes,
                             gemm_f32_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_LM_H */
