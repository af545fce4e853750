/*
 * qgemm_mx: what feeds a quantised product and what follows it, for AMD
 * Instinct MI355X (gfx950): root-mean-square norm with the residual's
 * addition and an 8- or 4-bit output, its gradient, microscaled (MX)
 * quantisation and the MX matrix product.
 *
 * The conventions are qgemm.h's: device pointers owned by the caller,
 * row-major matrices with a leading dimension in elements, every call
 * asynchronous on `stream`, arguments checked on the host before any launch,
 * the same status codes, and qgemm_last_kernel() names what was launched.
 * A call with M == 0 (or N == 0 for the product) checks its sizes only,
 * and launches nothing unless an output has elements all the same.
 *
 * MX format (OCP microscaling): 32 consecutive values of a row, a block,
 * share one scale byte b that stands for 2^(b - 127); 255 stands for NaN.
 * Elements are e4m3 (QG_MXFP8, one byte each, bias 7, largest 448) or e2m1
 * (QG_MXFP4, two to a byte, the even column in the low four bits, bias 1,
 * largest 6).  Quantising takes b = clamp(floor(log2 max|v|) - E + 127, 0,
 * 254) with E = 8 (e4m3) or 2 (e2m1), rounds v / 2^(b - 127) to the nearest
 * element, ties to even, and saturates.  A block whose values are all zero
 * gets b = 0, one that holds a NaN or an infinity b = 255 and zero elements.
 * Rows whose length is no multiple of 32 are filled up with zeros: a row of
 * n values has B = (n + 31) / 32 scale bytes and 32 B elements (32 B or
 * 16 B bytes).
 */
#ifndef QGEMM_MX_H
#define QGEMM_MX_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest row of the norm and its gradient. */
#define QG_RMS_NORM_MAX_COLUMNS 65536

/*
 * Root-mean-square norm of every row, after adding the residual:
 *
 *   h[m,:] = round(x[m,:] + residual[m,:])      to x's type; h = x without one
 *   r[m]   = 1 / sqrt(sum_j h[m,j]^2 / n + eps)
 *   y[m,j] = h[m,j] * r[m] * weight[j]
 *
 * The norm sees h as it is stored, so a later reader of h (the gradient)
 * sees the same values.  Sums and r are fp32; a row whose sum of squares
 * passes fp32's range gives r = 0, and one whose squares fall below it r = 1 /
 * sqrt(eps), infinity with eps = 0.  `format` is the form y takes:
 *   QG_FP32, QG_BF16, QG_FP16: out is y, [M,n], rounded once; row_scale
 *     (may be NULL) receives r.  16-bit formats need x of the same type.
 *   QG_INT8: with t = fl32(h * weight) and a = max_j |t[m,j]|,
 *       out[m,j]     = rint(fl32(t[m,j] * fl32(127 / a)))    int8, ties to even
 *       row_scale[m] = a * r[m] / 127
 *     so y ~ out * row_scale, the left operand and act_scale of qgemm_a8w8.
 *     r scales a whole row, so the codes do not depend on it: they are
 *     exactly these fp32 steps.  (Rows with a < 2^-100 are multiplied by
 *     2^60 first, which keeps 127 / a finite.)  A row of zeros gives codes 0
 *     and scale 1, a row whose t holds a NaN or an infinity codes 0 and scale
 *     NaN.
 *   QG_MXFP8, QG_MXFP4: out and block_scale hold t in MX form (t, not y:
 *     again the codes do not depend on r), row_scale[m] = r[m]: the left
 *     operand and act_scale of mx_matmul.  out rows hold 32 B elements,
 *     block_scale is [M,B].
 *   x, residual (may be NULL): `type` QG_FP32, QG_BF16 or QG_FP16, [M,n].
 *   weight: [n], weight_type `type` or QG_FP32.
 *   h: [M,n] of `type`, written if residual is given (then required); it may
 *     be x or residual itself.  ldo is in bytes for QG_MXFP4 (else elements).
 *   eps: finite, >= 0.
 * Requires n >= 1; n > QG_RMS_NORM_MAX_COLUMNS is QG_ERR_UNSUPPORTED.
 * Pointers need only their type's alignment.
 */
qg_status rms_norm(int64_t M, int64_t n,
                   const void* x, qg_dtype type, int64_t ldx,
                   const void* residual, int64_t ld_residual,
                   const void* weight, qg_dtype weight_type, float eps,
                   void* h, int64_t ldh,
                   void* out, qg_dtype format, int64_t ldo,
                   uint8_t* block_scale, int64_t ld_block_scale,
                   float* row_scale,
                   void* stream);

/*
 * Gradient of the norm, straight through a quantised output.  With
 * g = dy * weight:
 *
 *   dx[m,j]    = r g[m,j] - h[m,j] r^3 / n * sum_i g[m,i] h[m,i]  (+ dh[m,j])
 *   dweight[j] = sum_m dy[m,j] h[m,j] r[m]
 *
 * dx is the gradient of x and of the residual alike; dh (may be NULL) is the
 * gradient that reaches h from elsewhere (the residual stream).
 *   dy, h, dh, dx: `type`, [M,n]; dx may be dy or dh itself.
 *   rstd: fp32 [M], r as rms_norm left it.
 *   weight, dweight: [n] of weight_type (`type` or QG_FP32).
 *   workspace: rms_norm_grad_workspace_bytes(M, n) bytes, 16-byte aligned,
 *     not cleared; calls that overlap in time must not share one.  What a
 *     larger M, n or both asks for is enough as well, though it may be less:
 *     the call then runs on fewer workgroups.
 * Sums are fp32 in a fixed order, which depends on the sizes and the workspace's
 * alone: results repeat bit for bit.  M == 0 writes dweight = 0.
 */
size_t rms_norm_grad_workspace_bytes(int64_t M, int64_t n);
qg_status rms_norm_grad(int64_t M, int64_t n,
                        const void* dy, qg_dtype type, int64_t ld_dy,
                        const void* h, int64_t ldh,
                        const void* weight, qg_dtype weight_type,
                        const float* rstd,
                        const void* dh, int64_t ld_dh,
                        void* dx, int64_t ld_dx, void* dweight,
                        void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * x [M,n] (`type` QG_FP32, QG_BF16 or QG_FP16) to MX form.  format QG_MXFP8
 * or QG_MXFP4; codes rows hold 32 B elements at a stride of ldc bytes, scale
 * is [M,B] at a stride of lds bytes.  mx_matmul's fast kernels want ldc a
 * multiple of 16 and lds a multiple of 4.  QG_ERR_UNSUPPORTED, here and in
 * mx_dequantize, for 2^32 or more blocks.
 */
qg_status mx_quantize(int64_t M, int64_t n,
                      const void* x, qg_dtype type, int64_t ldx,
                      void* codes, qg_dtype format, int64_t ldc,
                      uint8_t* scale, int64_t lds,
                      void* stream);

/*
 * The values that an MX matrix stands for: out[m,j] = element * 2^(b - 127),
 * j < n, rounded once to out_type (exact in fp32 and, away from its
 * subnormals, in bf16); b = 255 gives NaN.
 */
qg_status mx_dequantize(int64_t M, int64_t n,
                        const void* codes, qg_dtype format, int64_t ldc,
                        const uint8_t* scale, int64_t lds,
                        void* out, qg_dtype out_type, int64_t ldo,
                        void* stream);

/*
 * Product of an MX activation and an MXFP4 weight on the scaled matrix cores:
 *
 *   out[m,n] = act_scale[m] * sum_k A[m,k] 2^(as[m,k/32]-127) W[n,k] 2^(ws[n,k/32]-127)
 *
 *   A: a_format QG_MXFP8 or QG_MXFP4, [M,K], row stride lda bytes;
 *   W: QG_MXFP4 [N,K], row stride ldw bytes; a_scale [M,K/32], w_scale
 *   [N,K/32], strides in bytes.  K: a multiple of 32, K >= 32.
 *   act_scale: fp32 [M], or NULL for 1.
 *   out: QG_FP32, QG_BF16 or QG_FP16, [M,N], rounded once.
 * Operands with 16-byte aligned rows, scale rows at multiples of 4 bytes and
 * readable to the end of the 4-byte word that holds their last byte take the
 * fast kernels; `scale_rows_padded` says that they are readable so, the last
 * row's too.  All others run a slower kernel that reads bytes.
 * Accuracy: every product is exact, and sums are fp32, whatever the output's
 * type.  (With e4m3 activations the matrix cores would cut off what lies 2^-14
 * below the largest of 16 products; the activations are split in two by
 * magnitude and multiplied twice, so that nothing is.)  Sums are added in a
 * fixed order: results repeat bit for bit.
 * An element whose block scale is 255 gives NaN.
 * QG_ERR_UNSUPPORTED if 512 rows of an operand span 2^31 bytes, or the output
 * has 2^23 or more tiles of 256 x 256.
 */
qg_status mx_matmul(int64_t M, int64_t N, int64_t K,
                    const void* A, qg_dtype a_format, int64_t lda,
                    const uint8_t* a_scale, int64_t ld_a_scale,
                    const void* W, int64_t ldw,
                    const uint8_t* w_scale, int64_t ld_w_scale,
                    int scale_rows_padded,
                    const float* act_scale,
                    void* out, qg_dtype out_type, int64_t ldo,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif
