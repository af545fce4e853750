/*
 * qgemm_fused: the A8W8 product as a feed-forward block uses it, for AMD
 * Instinct MI355X (gfx950): with bias, activation and residual in its epilogue,
 * as a gated pair, with 8-bit checkpoints of what the activation sees and the
 * backward passes that read them; and the int8 quantiser.
 *
 * The conventions are qgemm.h's: device pointers owned by the caller,
 * row-major matrices with a leading dimension in elements, every call
 * asynchronous on `stream`, arguments checked on the host before any launch,
 * the same status codes, and qgemm_last_kernel() names what was launched.  A call
 * whose outputs have no rows (M = 0) or, of the products, no columns (N = 0) checks its
 * sizes only and launches nothing (but M = 0 clears a dbias).  With rows, K = 0, for the
 * gradients N = 0 too, and for int8_quantize and int8_dequantize n < 1, are
 * QG_ERR_INVALID_ARGUMENT, whether anything would be written or not.
 * int8 sums wrap mod 2^32, as qgemm_a8w8's do.
 *
 * int8 form: the values t of a row, or of each block of 32 columns of it (the
 * last one may be shorter), share one fp32 scale.  With a = max |t|:
 *     code  = rint(fl32(t * fl32(127 / a)))     ties to even
 *     scale = fl32(a / 127)
 * and t ~ code * scale.  (With a < 2^-100 both t and a are multiplied by 2^60
 * first, which keeps 127 / a finite.)  Zeros alone give codes 0 and scale 1;
 * a NaN or an infinity among them gives codes 0 and scale NaN.
 *
 * Workspaces: as many bytes as the call's own *_workspace_bytes function asks
 * for (0: NULL is fine), 256-byte aligned, not cleared; calls that overlap in
 * time must not share one.
 */
#ifndef QGEMM_FUSED_H
#define QGEMM_FUSED_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(z), in fp32:
 *   NONE z;  RELU max(z, 0);  SILU z / (1 + exp(-z));
 *   GELU z (1 + erf(z / sqrt 2)) / 2;
 *   GELU_TANH z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2
 * The exponential and the reciprocal are the hardware's.  Off by at most, relative to the
 * value: SILU (|z| + 4) 2^-23; GELU (z^2 + 5) 2^-23; GELU_TANH (|y| + 2) 2^-21, with
 * y = sqrt(8 / pi) (z + 0.044715 z^3); magnitudes below 2^-119 may be given as 0. */
typedef enum {
    QG_ACT_NONE = 0, QG_ACT_RELU = 1, QG_ACT_SILU = 2, QG_ACT_GELU = 3, QG_ACT_GELU_TANH = 4
} qg_activation;

/* Longest row of int8_quantize with one scale a row, and most output columns (N) of
 * the gradients. */
#define QG_INT8_ROW_MAX_COLUMNS 65536
#define QG_A8W8_GRAD_MAX_COLUMNS 65535

/*
 * Product with bias, activation and residual:
 *
 *   z[m,n]   = fl32(fl32((float)(sum_k A[m,k] W[k,n]) * act_scale[m]) * weight_scale[n])  (+ bias[n], rounded)
 *   out[m,n] = round(act(z[m,n]) + residual[m,n])
 *
 *   A, W, b_trans, act_scale, weight_scale and their lengths: as qgemm_a8w8.
 *   bias: fp32 [N], or NULL.
 *   residual: [M,N] of out's type, or NULL; it may be out itself (same rows).
 *   out: QG_FP32, QG_BF16 or QG_FP16, rounded once.
 *   checkpoint: NULL, or int8 [M,N] that receives z in int8 form by blocks of 32,
 *     checkpoint_scale [M, (N + 31) / 32] its scales.
 * QG_ERR_UNSUPPORTED, here and in the calls below, if operands pass the spans that
 * qgemm_a8w8 takes, a leading dimension of an output, residual or checkpoint is 2^22 or
 * more, or there are about 2^23 tiles of 64 x 128 sums (2 N columns of a pair, 2 M rows of a
 * gradient).
 */
size_t qgemm_a8w8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                         const int8_t* A, int64_t lda,
                                         const int8_t* W, int64_t ldw, int b_trans, int with_checkpoint);
qg_status qgemm_a8w8_linear(int64_t M, int64_t N, int64_t K,
                            const int8_t* A, int64_t lda,
                            const int8_t* W, int64_t ldw, int b_trans,
                            const float* act_scale, int64_t act_scale_len,
                            const float* weight_scale, int64_t weight_scale_len,
                            const float* bias, qg_activation activation,
                            const void* residual, int64_t ld_residual,
                            void* out, qg_dtype out_dtype, int64_t ldo,
                            int8_t* checkpoint, int64_t ld_checkpoint,
                            float* checkpoint_scale, int64_t ld_checkpoint_scale,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * Gated pair: with g and u the two products, each as z above (without bias),
 *
 *   out[m,n] = round(act(g[m,n]) * u[m,n])
 *
 *   W_gate, W_up: int8 [K,N], or [N,K] with b_trans, each with its own leading
 *     dimension and scale.
 *   checkpoint: NULL, or int8 [2,M,N]: g's codes, then u's from row M on;
 *     checkpoint_scale [2, M, (N + 31) / 32] likewise.
 */
size_t qgemm_a8w8_gated_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                        const int8_t* A, int64_t lda,
                                        const int8_t* W_gate, int64_t ld_gate,
                                        const int8_t* W_up, int64_t ld_up, int b_trans, int with_checkpoint);
qg_status qgemm_a8w8_gated(int64_t M, int64_t N, int64_t K,
                           const int8_t* A, int64_t lda,
                           const int8_t* W_gate, int64_t ld_gate,
                           const int8_t* W_up, int64_t ld_up, int b_trans,
                           const float* act_scale, int64_t act_scale_len,
                           const float* gate_scale, int64_t gate_scale_len,
                           const float* up_scale, int64_t up_scale_len,
                           qg_activation activation,
                           void* out, qg_dtype out_dtype, int64_t ldo,
                           int8_t* checkpoint, int64_t ld_checkpoint,
                           float* checkpoint_scale, int64_t ld_checkpoint_scale,
                           void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Gradients with respect to what A stands for, x = A * act_scale (straight through
 * its rounding; the weights are constants), and the bias, from the checkpoint:
 *
 *   linear   p = dy act'(z);                     dx[m,k] = sum_n (p weight_scale)[m,n] W[k,n];  dbias[n] = sum_m p[m,n]
 *   gated    p = dy u act'(g),  q = dy act(g);   dx[m,k] = sum_n (p gate_scale)[m,n] W_gate[k,n] + (q up_scale)[m,n] W_up[k,n]
 *
 * with z, g, u as the checkpoint holds them (the gradient of a residual is dy
 * itself).  act'(0) of RELU is 0.  The factors (p weight_scale), and in the gated
 * form p's and q's together, are held in 16-bit fixed point for each row: with
 * a = the largest magnitude among the row's, t = rint(value * 32639 / a).  Sums over n
 * are exact; an error of a factor is at most a / 65278 (and four roundings in
 * fp32 on the way; more where a is below 2^-110, whose scale is no normal
 * number).  A row that holds a NaN or an infinity among its factors gives a dx
 * row of NaN.
 *   dy: QG_BF16 or QG_FP16 [M,N]; dx: [M,K] of that type.
 *   checkpoint, checkpoint_scale: as the forward call left them.  For the linear
 *     form with QG_ACT_NONE both may be NULL.
 *   activation: the forward call's, which the checkpoint does not hold.
 *   dbias: fp32 [N], or NULL.  Its sums are fp32 in a fixed order.
 * Results repeat bit for bit.  N > QG_A8W8_GRAD_MAX_COLUMNS is
 * QG_ERR_UNSUPPORTED.  M == 0 writes dbias = 0.
 */
size_t qgemm_a8w8_linear_grad_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                              const int8_t* W, int64_t ldw, int b_trans, int with_bias);
qg_status qgemm_a8w8_linear_grad(int64_t M, int64_t N, int64_t K,
                                 const void* dy, qg_dtype dtype, int64_t ld_dy,
                                 const int8_t* W, int64_t ldw, int b_trans,
                                 const float* weight_scale, int64_t weight_scale_len,
                                 const int8_t* checkpoint, int64_t ld_checkpoint,
                                 const float* checkpoint_scale, int64_t ld_checkpoint_scale,
                                 qg_activation activation,
                                 void* dx, int64_t ld_dx, float* dbias,
                                 void* workspace, size_t workspace_bytes,
                                 void* stream);
size_t qgemm_a8w8_gated_grad_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                             const int8_t* W_gate, int64_t ld_gate,
                                             const int8_t* W_up, int64_t ld_up, int b_trans);
qg_status qgemm_a8w8_gated_grad(int64_t M, int64_t N, int64_t K,
                                const void* dy, qg_dtype dtype, int64_t ld_dy,
                                const int8_t* W_gate, int64_t ld_gate,
                                const int8_t* W_up, int64_t ld_up, int b_trans,
                                const float* gate_scale, int64_t gate_scale_len,
                                const float* up_scale, int64_t up_scale_len,
                                const int8_t* checkpoint, int64_t ld_checkpoint,
                                const float* checkpoint_scale, int64_t ld_checkpoint_scale,
                                qg_activation activation,
                                void* dx, int64_t ld_dx,
                                void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * x [M,n] (QG_FP32, QG_BF16 or QG_FP16) to int8 form.  block 0: one scale a row
 * (scale [M], ld_scale >= 1; what qgemm_a8w8 and the calls above take as A and
 * act_scale), n at most QG_INT8_ROW_MAX_COLUMNS, else QG_ERR_UNSUPPORTED.  block
 * 32: one scale per block, scale [M, (n + 31) / 32].
 */
qg_status int8_quantize(int64_t M, int64_t n,
                        const void* x, qg_dtype type, int64_t ldx, int block,
                        int8_t* codes, int64_t ldc,
                        float* scale, int64_t ld_scale,
                        void* stream);

/* code * scale in fp32, rounded once to out_type (QG_FP32, QG_BF16 or QG_FP16). */
qg_status int8_dequantize(int64_t M, int64_t n,
                          const int8_t* codes, int64_t ldc,
                          const float* scale, int64_t ld_scale, int block,
                          void* out, qg_dtype out_type, int64_t ldo,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif
