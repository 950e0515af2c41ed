/*
 * gemm_f32_block -- what stands between a model's blocks, on row-major
 * matrices for NVIDIA GB300 (sm_103a): the norms after and before a block
 * with its gate and residual, activations kept in 8 bits for the backward
 * pass, and the gradients that are computed from them.  In the same library
 * as the products (gemm_f32.h) and the norms and losses (gemm_f32_lm.h),
 * whose rules hold here too: caller-owned device pointers, every call
 * asynchronous on `stream` and never synchronising the host, return code 0 or
 * a negative GEMM_F32_E* code, nothing printed or thrown, device-side
 * failures read later through gemm_f32_status(); types, strides, alignment,
 * scratch and CUDA graphs as in gemm_f32_lm.h.
 *
 * gemm_f32_last_kernel() names the kernel of a call's main pass:
 * "block_norm_kernel" or "block_norm_grad_kernel" for rows of up to 32768
 * columns and for wider ones where eight SMs hold two rows of each matrix and
 * the vectors: forward up to 131072 (bfloat16, one vector, no gate) and 40960
 * (fp32, four vectors and a gate matrix); the gradient for rms norms on both
 * ends without a gate per channel alone, up to 65536 (bfloat16 without a gate)
 * and 36864 (fp32 with a gate matrix).  "block_norm_wide_kernel" or
 * "block_norm_grad_wide_kernel" beyond that, "block_columns_kernel" (gradient
 * of no rows), "checkpoint_kernel", "restore_kernel", "half_gemm_kernel"
 * (weight gradient), "memset" (weight gradient of no rows).
 *
 * Every sum is fp32 and taken in a fixed order: the same call on the same
 * inputs gives the same bits.
 */
#ifndef GEMM_F32_BLOCK_H
#define GEMM_F32_BLOCK_H

#include <stddef.h>

#include "gemm_f32_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum gemm_f32_norm {
    GEMM_F32_NORM_LAYER = 0,    /* (x - mean) * rstd * weight + bias */
    GEMM_F32_NORM_RMS = 1       /* x * rstd * weight, rstd of the mean square; no bias */
};

/* One block's end, the parameters that its forward call and its gradient
 * share.  Zero-initialise it and set what is there. */
typedef struct gemm_f32_block {
    int type;                 /* of the matrices: GEMM_F32_TYPE_* */
    int weight_type;          /* of the vectors: `type` or fp32 */
    int norm;                 /* of both norms: GEMM_F32_NORM_* */
    int post;                 /* 1: the block's output is normed before it is added */
    long long rows;
    int width;
    float eps;                /* forward only */
    float residual_scale, branch_scale;
    const void* weight;       /* of the norm of h: width values, or NULL (1) */
    const void* bias;         /* or NULL (0) */
    const void* post_weight;  /* of the block's output's norm, as weight and bias */
    const void* post_bias;
    const void* gate;         /* NULL (1), `width` values of weight_type (ld_gate 0), or a
                                 matrix of `type` with row stride ld_gate */
    long long ld_gate;
} gemm_f32_block_t;

/* Rows as they are (codes NULL), or kept in 8 bits by gemm_f32_checkpoint. */
typedef struct gemm_f32_rows {
    const void* data;
    long long ld;             /* elements */
    const unsigned char* codes;
    long long ld_codes;       /* bytes */
    const unsigned char* exponents;
    long long ld_exponents;   /* bytes */
} gemm_f32_rows_t;

/* The end of a block and the norm that the next one begins with:
 *     p = branch, or with `post` its norm:  (branch - mean_b) * rstd_b * post_weight + post_bias
 *     h = residual_scale * residual + branch_scale * gate * p
 *     y = (h - mean) * rstd * weight + bias
 * with each row's mean = sum_d x_d / width (0 for GEMM_F32_NORM_RMS) and
 * rstd = 1 / sqrt(sum_d (x_d - mean)^2 / width + eps); y and its statistics
 * come from h before h is rounded.  h may be NULL where it is not wanted.
 * stats (may be NULL) receives fp32 rows of `rows` values each: mean and rstd
 * of h and, with `post`, mean_b and rstd_b.  y and h may each be branch,
 * residual or a gate matrix itself, with the same stride; they overlap
 * nothing else.  rows == 0 does nothing.
 * Returns 0, GEMM_F32_EINVAL (an unknown type or norm, width < 1 or above
 * 2^31 - 1025, rows < 0, a stride below width, eps negative, eps or a scale
 * not finite, a null or misaligned pointer, a bias with GEMM_F32_NORM_RMS,
 * post_weight or post_bias without `post`, outputs that overlap),
 * GEMM_F32_EDEVICE or GEMM_F32_ELAUNCH. */
int gemm_f32_block_norm(const gemm_f32_block_t* block, const void* branch, long long ld_branch,
                        const void* residual, long long ld_residual, void* y, long long ldy, void* h,
                        long long ldh, float* stats, gemm_f32_stream_t stream);

/* Its gradients, for dy, the gradient of y, and dh, the one that reaches h
 * from further on (NULL: 0).  With hat = (h - mean) * rstd, g = dy * weight,
 * and likewise hat_b of the branch:
 *     d   = dh + rstd * (g - sum(g) / width - hat * sum(g * hat) / width)
 *     dresidual = residual_scale * d
 *     e   = branch_scale * d * gate,   dgate = branch_scale * d * p
 *     dbranch = e, or with `post`, e_b = e * post_weight:
 *               rstd_b * (e_b - sum(e_b) / width - hat_b * sum(e_b * hat_b) / width)
 * and over the rows:
 *     dweight = sum dy * hat,  dbias = sum dy,
 *     dpost_weight = sum e * hat_b,  dpost_bias = sum e,
 *     dgate of a vector gate the sum of its rows
 * (without the sum(g) and sum(e_b) terms for GEMM_F32_NORM_RMS).  stats is
 * what the forward call wrote; h its output and branch its input, each as it
 * was or as gemm_f32_checkpoint kept it.  branch is read only with `post` or
 * a gate, and may be NULL otherwise.  Matrices hold block->type, vectors
 * block->weight_type; every output may be NULL when it is not wanted.
 * dresidual, dbranch and a dgate matrix may each be dy, dh, h, branch or a
 * gate matrix itself (not 8-bit codes), with the same stride; they overlap
 * nothing else.  rows == 0 writes zeros into the vectors.  Returns as
 * gemm_f32_block_norm, and GEMM_F32_ESCRATCH. */
int gemm_f32_block_norm_grad(const gemm_f32_block_t* block, const void* dy, long long lddy,
                             const void* dh, long long lddh, const gemm_f32_rows_t* h,
                             const gemm_f32_rows_t* branch, const float* stats, void* dbranch,
                             long long ld_dbranch, void* dresidual, long long ld_dresidual,
                             void* dgate, long long ld_dgate, void* dweight, void* dbias,
                             void* dpost_weight, void* dpost_bias, gemm_f32_stream_t stream);

#define GEMM_F32_SAVED_BLOCK 32   /* columns that share an exponent */

/* Keeps x (rows x width) in 8 bits.  Every 32 columns of a row share a power
 * of two, the least that takes their largest finite magnitude to 448 or below
 * (and no less than 2^-126); a code is x over that power, rounded to the
 * nearest e4m3 value, ties to even (to the one below where that would stand
 * for 2^128).  So a value is off by at most 2^-4 of itself or 2^-10 of the
 * power.  Infinities and NaN are kept as NaN.
 * codes: rows of ld_codes bytes, a multiple of 16 and at least width rounded
 * up to 32, on a 16-byte boundary; all codes of a block are written, 0 from
 * column `width` on.  exponents: rows of ld_exponents bytes, a multiple of 16
 * and at least ceil(width / 32), on a 16-byte boundary; each the power's
 * exponent + 127.  Both hold all bytes of their rows, the last row included
 * (rows * ld bytes).  Returns as gemm_f32_block_norm. */
int gemm_f32_checkpoint(int type, long long rows, int width, const void* x, long long ldx,
                        unsigned char* codes, long long ld_codes, unsigned char* exponents,
                        long long ld_exponents, gemm_f32_stream_t stream);

/* Brings such rows back: code times power, exact in fp32 and, but for values
 * below 2^-126, in bfloat16.  Returns as gemm_f32_block_norm. */
int gemm_f32_restore(int type, long long rows, int width, const unsigned char* codes,
                     long long ld_codes, const unsigned char* exponents, long long ld_exponents,
                     void* out, long long ldo, gemm_f32_stream_t stream);

/* Weight gradient of a product y = x w^T whose x (rows x width) was kept in 8
 * bits:
 *     dw = dy^T x            dy: rows x out, dw: out x width
 * dy holds `type`; dw holds dw_type, `type` or fp32, and with `accumulate`
 * (fp32 only) is added to.  The values of x are exact on the tensor cores; a
 * dy of fp32 goes in three parts of bfloat16, to about fp32's own rounding (an
 * infinite one gives NaN).
 * Scratch: x in bfloat16 (2 bytes an element), the three parts of an fp32 dy
 * (6 bytes an element) or a copy of a dy whose rows are not on 16-byte
 * boundaries, and partial tiles.  rows == 0 gives zeros (or adds nothing).
 * Returns as gemm_f32_block_norm (and GEMM_F32_EINVAL for rows, width or out
 * above 2^31 - 1025), and GEMM_F32_ESCRATCH. */
int gemm_f32_weight_grad(int type, long long rows, int width, int out, const void* dy, long long lddy,
                         const unsigned char* codes, long long ld_codes,
                         const unsigned char* exponents, long long ld_exponents, int dw_type, void* dw,
                         long long lddw, int accumulate, gemm_f32_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_BLOCK_H */
