/*
 * tilegemm_ops.h -- C ABI of the operators around the block-scaled products
 * of tilegemm.h: what makes a block-scaled operand, what a training step
 * does with the 8-bit operand it kept, and the product of a few rows with
 * 4-bit weights.
 *
 *   training   rmsnorm_mxfp8 (or mxfp8_quantize) -> gemm_mxfp8;
 *              backward: gemm_wgrad_mxfp8 on the kept operand,
 *              gemm_bf16_ex for the input gradient, rmsnorm_backward
 *   serving    rmsnorm -> gemv_mxfp4
 *
 * Conventions as in tilegemm.h: the caller owns every buffer and the stream;
 * calls only enqueue kernels on `stream` (no allocation, no
 * synchronisation, no state kept), so they can be captured in HIP graphs;
 * arguments are checked before anything is enqueued and a status other than
 * GEMM_OK and GEMM_ERR_HIP leaves every output untouched.  Sizes and
 * leading dimensions count elements; matrices are row-major; pointers are
 * aligned to their element size (GEMM_ERR_MISALIGNED) and need no more than
 * that.  Sizes are below 2^31, and N of the row operators below 2^28
 * (GEMM_ERR_UNSUPPORTED).  Outputs overlap
 * neither inputs nor each other unless a call says so.  The same call on
 * the same values gives the same bits.
 *
 * Block-scaled rows (MXFP8): N a multiple of 32 elements (GEMM_ERR_UNSUPPORTED
 * otherwise); element n of a row has the value e4m3(Q[n]) * 2^(SF[n / 32] -
 * 127), Q and SF as gemm_mxfp8 takes an operand and its scales.  A block's
 * scale is the least power of two 2^e, e >= -127, with max|x| <= 448 * 2^e,
 * so that no element is clipped; elements are x / 2^e rounded to nearest
 * even.  An element that is NaN or infinite becomes the e4m3 NaN and does
 * not count towards its block's scale.
 */
#ifndef TILEGEMM_OPS_H
#define TILEGEMM_OPS_H

#include "tilegemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {                   /* element types of activations and weights */
    GEMM_TYPE_F32 = 0,
    GEMM_TYPE_BF16 = 1,
    GEMM_TYPE_FP16 = 2
} gemm_elem_type;

/*
 * mxfp8_quantize -- the rows x N matrix X (x_type) as block-scaled rows.
 *   X: ldx >= N    Q: e4m3 codes, ldq >= N    SF: e8m0 codes, rows x N/32,
 *   ldsf >= N/32 (GEMM_ERR_BAD_LD otherwise)
 * rows or N == 0: nothing is enqueued.  Negative sizes: GEMM_ERR_INVALID_SIZE;
 * another x_type: GEMM_ERR_UNSUPPORTED; X, Q or SF NULL:
 * GEMM_ERR_NULL_POINTER.
 */
gemm_status mxfp8_quantize(int64_t rows, int64_t N, const void *X, int64_t ldx, int x_type,
                           void *Q, int64_t ldq, void *SF, int64_t ldsf, hipStream_t stream);

/*
 * rmsnorm -- root-mean-square norm of each row, after the residual's addition:
 *     h = x + r  (rounded to `type`; h = x without R)
 *     rstd = 1 / sqrt(sum_n h[n]^2 / N + eps)       y[n] = h[n] * w[n] * rstd
 * with the sum and rstd in fp64, products in fp32 (by the rounded rstd) and y
 * rounded once.  y is the norm of the rounded h, the row that the next layer and
 * rmsnorm_backward read.
 *   X, R (NULL: no residual), H, Y: rows x N of `type`, ldx, ldr, ldh, ldy >= N
 *   W: N elements of w_type, which is `type` or GEMM_TYPE_F32
 *     (GEMM_ERR_UNSUPPORTED otherwise)
 *   H: h is written there when not NULL; H may be X or R (same leading
 *     dimension).  Y may be X or R too, unless H is the same.
 *   rstd: `rows` floats, or NULL
 *   eps: finite, >= 0 (GEMM_ERR_UNSUPPORTED otherwise)
 * A row with a NaN gives NaN.  One with an infinity, or whose sum of squares
 * exceeds fp32, has rstd 0: NaN at its infinities, zeros elsewhere.  With eps 0
 * a row of zeros has an infinite rstd and gives NaN.  rows or N == 0: nothing is
 * enqueued.
 */
gemm_status rmsnorm(int64_t rows, int64_t N, const void *X, int64_t ldx, const void *R, int64_t ldr,
                    int type, const void *W, int w_type, float eps, void *H, int64_t ldh,
                    void *Y, int64_t ldy, float *rstd, hipStream_t stream);

/*
 * rmsnorm_mxfp8 -- rmsnorm with y given out as block-scaled rows (quantised
 * from y as it is before any rounding: codes and scales that the roundings of
 * fp32 could change are taken in fp64): the A and SFA of
 * gemm_mxfp8, and the 8-bit copy that gemm_wgrad_mxfp8 reads in the backward
 * pass.  N a multiple of 32.  Everything else as rmsnorm.
 */
gemm_status rmsnorm_mxfp8(int64_t rows, int64_t N, const void *X, int64_t ldx, const void *R, int64_t ldr,
                          int type, const void *W, int w_type, float eps, void *H, int64_t ldh,
                          void *Q, int64_t ldq, void *SF, int64_t ldsf, float *rstd, hipStream_t stream);

/*
 * rmsnorm_backward -- gradients of rmsnorm (and, through the quantisation as
 * if it were the identity, of rmsnorm_mxfp8), from the gradient dY of y:
 *     g = dy * w     dx[n] = dh[n] + rstd * g[n] - h[n] * rstd^3 * (sum_j g[j] h[j]) / N
 *     dw[n] = sum over rows of dy[n] * h[n] * rstd
 * dx is the gradient of x and of r alike (h is their sum).
 *   dY, H, dH (NULL: none; the gradient that reaches h from elsewhere),
 *     dX: rows x N of `type`, leading dimensions >= N; dX may be dY, or dH
 *   W as rmsnorm; rstd: `rows` floats as rmsnorm wrote them
 *   dW: N floats, overwritten, or NULL: not computed (rows == 0: zeros)
 *   workspace: device memory, 256-byte aligned (GEMM_ERR_MISALIGNED), of at
 *     least rmsnorm_backward_workspace_bytes(rows, N) bytes
 *     (GEMM_ERR_WORKSPACE); not needed without dW.  Calls sharing it must be
 *     ordered.  Its contents need no initialisation.
 */
gemm_status rmsnorm_backward(int64_t rows, int64_t N, const void *dY, int64_t lddy, const void *H, int64_t ldh,
                             int type, const void *W, int w_type, const float *rstd, const void *dH, int64_t lddh,
                             void *dX, int64_t lddx, float *dW, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t N);

/*
 * gemm_wgrad_mxfp8 -- weight gradient from an 8-bit activation kept for the
 * backward pass: D = A^T.B + C summed over K tokens,
 *     D[m][n] = C[m][n] + sum_{k<K} bf16(A[k*lda + m]) * e4m3(B[k*ldb + n]) * 2^(SFB[k*ldsfb + n/32] - 127)
 * A is the output gradient, K x M; B and SFB are the block-scaled rows that
 * mxfp8_quantize or rmsnorm_mxfp8 wrote, K x N, each token's scales running
 * along N.  Every e4m3 * 2^e is exact in bf16, so the bf16 matrix
 * instructions see the kept values themselves; fp32 accumulation.  (Scales
 * below 2^-117 reach bf16's subnormals, and above 2^119 its end.)
 *   M, N, K < 2^31; N a multiple of 32; lda >= M, ldb >= N, ldsfb >= N/32,
 *   ldd >= N, ldc >= N (C NULL: 0; C == D with ldc == ldd accumulates in
 *   place); out_type as gemm_bf16 (C and D); leading dimensions below 8 MiB
 *   in bytes.
 *   workspace: device memory, 256-byte aligned, or NULL.  With at least
 *     gemm_wgrad_mxfp8_workspace_bytes(M, N, K) bytes, grids too small to fill
 *     the GPU cut K into ranges and sum the fp32 partial products in order, and
 *     A whose rows do not start on 16 bytes is copied first where M is no
 *     multiple of 8 and the product large; a smaller one or NULL runs without
 *     (the same result up to summation order).
 *     Calls sharing it must be ordered.
 * Scale code 0xFF and e4m3 NaN give NaN in the column's outputs.  K == 0:
 * D = C (or 0).
 */
gemm_status gemm_wgrad_mxfp8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                             const void *B, int64_t ldb, const void *SFB, int64_t ldsfb,
                             const void *C, int64_t ldc, void *D, int64_t ldd, int out_type,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t gemm_wgrad_mxfp8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * gemv_mxfp4 -- a few rows times 4-bit weights with group scales, D = X.W^T + C:
 *     D[m][n] = C[m][n] + sum_{k<K} x[m][k] * e2m1(W, n*ldw + k) * 2^(SFW[n*ldsfw + k/kblock] - 127)
 * W and SFW as gemm_mxfp4 and gemm_mx_kblock take B and SFB (ldw in
 * elements, even); X is not quantised: the products of its 16-bit elements
 * with the weights are exact and summed in fp32.  Made for M up
 * to 16 and bound by the reading of W; any M up to 2^20 is right.
 *   x_type: GEMM_TYPE_BF16 or GEMM_TYPE_FP16    out_type as gemm_bf16 (C, D)
 *   K a multiple of 32; kblock as gemm_mx_kblock: 32 times a power of two, or
 *   any multiple of 32 that is at least K (GEMM_ERR_UNSUPPORTED otherwise)
 *   ldx, ldw >= K; ldsfw >= ceil(K / kblock); C NULL: 0; C == D with
 *   ldc == ldd accumulates in place.
 *   workspace: device memory, 256-byte aligned, or NULL.  With at least
 *     gemv_mxfp4_workspace_bytes(M, N, K) bytes (at most 64 MiB or 32 rows'
 *     partial sums), calls whose X exceeds the LDS of a compute unit, and
 *     those of few rows of W, cut K into ranges and sum the fp32 partial
 *     sums in order; a smaller one or NULL runs
 *     uncut, slower (the same result up to summation order).  Calls sharing it
 *     must be ordered.
 * Leading dimensions below 8 MiB in bytes (ldd's holds N below 2^21 with fp32
 * results and 2^22 with bf16 ones), ldsfw below 2^23.  Weights beyond bf16's
 * range (4 and 6 at 2^126, 2 to 6 at 2^127) are infinite.
 * Scale code 0xFF gives NaN in the row's outputs.
 */
gemm_status gemv_mxfp4(int64_t M, int64_t N, int64_t K, int64_t kblock, const void *X, int64_t ldx, int x_type,
                       const void *W, int64_t ldw, const void *SFW, int64_t ldsfw,
                       const void *C, int64_t ldc, void *D, int64_t ldd, int out_type,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t gemv_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* TILEGEMM_OPS_H */
