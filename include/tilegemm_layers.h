/*
 * tilegemm_layers.h -- C ABI of operators of a feed-forward layer's linear
 * parts: the gated block with its backward pass, products of 8-bit integers
 * with scales per row and column, and the clipping of gradients by their
 * common norm.
 *
 *   training   (rmsnorm ->) gemm_glu -> gemm_bf16; backward: gemm_glu_backward
 *              (-> rmsnorm_backward), grad_clip before the optimiser
 *   serving    (rmsnorm ->) gemm_glu, or int8_quantize -> gemm_int8
 *
 * Conventions as in tilegemm_ops.h: the caller owns every buffer and the
 * stream; calls only enqueue kernels on `stream` (no allocation, no
 * synchronisation, no state kept), so they can be captured in HIP graphs;
 * arguments are checked before anything is enqueued and a status other than
 * GEMM_OK and GEMM_ERR_HIP leaves every output untouched.  Sizes and leading
 * dimensions count elements; matrices are row-major; pointers are aligned to
 * their element size (GEMM_ERR_MISALIGNED) and need no more than that, though
 * operands whose rows start on 16 bytes run faster.  Sizes are below 2^31 and
 * leading dimensions below 8 MiB in bytes, but for int8_quantize's
 * (GEMM_ERR_UNSUPPORTED).  Outputs and
 * workspaces overlap neither inputs nor each other (GEMM_ERR_UNSUPPORTED)
 * unless a call says so: an input's piece of memory, from its first element to
 * its last, holds no result.  Results of one leading dimension may lie row by
 * row next to each other, as the halves of one tensor.  The same call on the
 * same values gives the same bits.
 */
#ifndef TILEGEMM_LAYERS_H
#define TILEGEMM_LAYERS_H

#include "tilegemm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {                   /* activations of the gated block */
    GEMM_ACT_SILU = 0,           /* g / (1 + e^-g) */
    GEMM_ACT_GELU = 1,           /* g Phi(g), Phi the normal distribution's */
    GEMM_ACT_GELU_TANH = 2,      /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
    GEMM_ACT_RELU = 3            /* max(g, 0) */
} gemm_act;

/*
 * gemm_glu -- gated block of a feed-forward layer, both products, the
 * activation and their product in one kernel:
 *     g = X.Wg^T     u = X.Wu^T     H[m][f] = act(g[m][f]) * u[m][f]
 * Sums and activation in fp32, H rounded once.
 *   X: M x K, Wg, Wu: F x K (two tensors, or the halves of one), H: M x F, all
 *     of `type`, GEMM_TYPE_BF16 or GEMM_TYPE_FP16 (GEMM_ERR_UNSUPPORTED
 *     otherwise); ldx, ldwg, ldwu >= K, ldh >= F (GEMM_ERR_BAD_LD)
 *   G, U: M x F, g and u rounded to `type`, what gemm_glu_backward reads; NULL:
 *     not kept (each for itself).  ldg, ldu >= F.
 *   workspace: device memory, 256-byte aligned (GEMM_ERR_MISALIGNED), or NULL.
 *     With at least gemm_glu_workspace_bytes(M, F, K) bytes, large calls whose
 *     operand rows do not start on 16 bytes copy them there first; a smaller one
 *     or NULL runs without, slower (the same result up to summation order).
 *     Calls sharing it must be ordered.  Its contents need no initialisation.
 * Up to 32 rows of X run a kernel made for the reading of the weights.  M and F
 * below 2^27.  M or F == 0: nothing is enqueued; K == 0: g = u = 0.
 */
gemm_status gemm_glu(int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                     const void *Wu, int64_t ldwu, int type, int act, void *H, int64_t ldh, void *G, int64_t ldg,
                     void *U, int64_t ldu, void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t gemm_glu_workspace_bytes(int64_t M, int64_t F, int64_t K);

/*
 * gemm_glu_backward -- gradients of gemm_glu from the gradient dH of H:
 *     dg = dH * u * act'(g)      du = dH * act(g)
 *     dX = dg.Wg + du.Wu         dWg = Cg + dg^T.X      dWu = Cu + du^T.X
 * dg and du are computed in fp32 from the kept G and U and rounded to `type`
 * (the products' operands): in fp16 past 65504 they are infinities, below 2^-14
 * multiples of 2^-24.  The products are summed in fp32.  relu'(0) = 0.
 *   dH, G, U: M x F, X: M x K, Wg, Wu: F x K of `type` as in gemm_glu
 *   dX: M x K of `type`, or NULL: not computed (Wg and Wu are not read)
 *   dWg, dWu: F x K of grad_type, which is `type` or GEMM_TYPE_F32
 *     (GEMM_ERR_UNSUPPORTED otherwise), or both NULL: not computed (X is not read)
 *   Cg, Cu: F x K of grad_type added to them, or both NULL; Cg may be dWg and
 *     Cu dWu with the same leading dimension (gradients accumulated in place)
 *   workspace: device memory, 256-byte aligned (GEMM_ERR_MISALIGNED), of at
 *     least gemm_glu_backward_workspace_bytes(M, F, K) bytes
 *     (GEMM_ERR_WORKSPACE): dg and du, and copies of X and the weights, rows
 *     laid along the sums.  Calls sharing it must be ordered.  Its contents
 *     need no initialisation.
 * M < 2^21, F < 2^20, and m f + (m + 2 f) k < 2^24, where m, f, k are M, F, K
 * divided by 64 and rounded up (GEMM_ERR_UNSUPPORTED).  M == 0: dWg = Cg and dWu
 * = Cu, or zeros.
 */
gemm_status gemm_glu_backward(int64_t M, int64_t F, int64_t K, const void *dH, int64_t lddh, const void *G,
                              int64_t ldg, const void *U, int64_t ldu, const void *X, int64_t ldx, const void *Wg,
                              int64_t ldwg, const void *Wu, int64_t ldwu, int type, int act, void *dX, int64_t lddx,
                              const void *Cg, int64_t ldcg, const void *Cu, int64_t ldcu, void *dWg, int64_t lddwg,
                              void *dWu, int64_t lddwu, int grad_type, void *workspace, size_t workspace_bytes,
                              hipStream_t stream);

size_t gemm_glu_backward_workspace_bytes(int64_t M, int64_t F, int64_t K);

/*
 * int8_quantize -- the rows x N matrix X (x_type) as 8-bit integers with one
 * scale a row:
 *     S[r] = max(max_n |x[r][n]| / 127, 2^-126) in fp32     Q[r][n] = x[r][n] / S[r] rounded to nearest even
 * of the exact quotient; codes lie in -127 .. 127.  A row with a NaN or an
 * infinity has codes 0 and the scale NaN, so that its products are NaN.
 *   X: ldx >= N    Q: int8, ldq >= N    S: `rows` floats
 * rows == 0: nothing is enqueued.  N < 2^28.  N == 0: S = 2^-126.
 */
gemm_status int8_quantize(int64_t rows, int64_t N, const void *X, int64_t ldx, int x_type, void *Q, int64_t ldq,
                          float *S, hipStream_t stream);

/*
 * gemm_int8 -- D = A.B + C of 8-bit integers with a scale for each row of A
 * (token) and of B (channel):
 *     D[m][n] = C[m][n] + SA[m] * SB[n] * sum_k A[m][k] * B[n][k]
 * The integer sum is exact (K < 2^17, GEMM_ERR_UNSUPPORTED otherwise); it,
 * SA * SB, their product and the sum with C are each rounded to fp32, D then to
 * out_type.
 *   A: M x K, B: N x K int8, lda, ldb >= K; SA: M floats, SB: N floats
 *   out_type: GEMM_TYPE_F32, GEMM_TYPE_BF16 or GEMM_TYPE_FP16, of C and D
 *   C: M x N, NULL: 0; ldc >= N, or 0: one row for all (a bias); C == D with
 *     ldc == ldd accumulates in place; C and D overlap in no other way
 *     (GEMM_ERR_UNSUPPORTED)
 *   workspace as in gemm_glu, gemm_int8_workspace_bytes(M, N, K) bytes
 * Up to 32 rows of A run a kernel made for the reading of B.  M and N below
 * 2^27.  M or N == 0: nothing is enqueued; K == 0: D = C, or 0.
 */
gemm_status gemm_int8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const float *SA, const void *B,
                      int64_t ldb, const float *SB, const void *C, int64_t ldc, void *D, int64_t ldd, int out_type,
                      void *workspace, size_t workspace_bytes, hipStream_t stream);

size_t gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * grad_norm -- norm of n gradients taken together: the root of the sum of all
 * their elements' squares, summed in fp64, rounded to fp32.
 *   grads[i]: sizes[i] elements (>= 0, contiguous) of types[i], a
 *     gemm_elem_type each; the three arrays are host memory, read during the
 *     call.  Sums do not depend on addresses, but on sizes and their order.
 *   norm: one float
 *   workspace: device memory, 256-byte aligned (GEMM_ERR_MISALIGNED), of at
 *     least grad_workspace_bytes(n) bytes (GEMM_ERR_WORKSPACE).  Calls sharing
 *     it must be ordered.  Its contents need no initialisation.
 * n < 2^20; sizes below 2^40, of all together too (GEMM_ERR_UNSUPPORTED).  A
 * NaN gives NaN.  n == 0: 0.
 */
gemm_status grad_norm(int64_t n, const void *const *grads, const int64_t *sizes, const int *types, float *norm,
                      void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * grad_clip -- n gradients scaled down to a common norm:
 *     out[i] = grads[i] * min(1, max_norm / (norm + 1e-6))
 * the factor in fp32, products rounded once.
 *   given: NULL: the norm is computed as by grad_norm and written to *norm;
 *     otherwise one float, read in its place (a norm that ranks have summed),
 *     and norm may be NULL (else it receives a copy; it may be `given`)
 *   out: n tensors of the same sizes and types; out NULL or out[i] == grads[i]:
 *     in place, where a factor of 1 leaves them untouched.  No result shares
 *     memory with another or with another's gradient (GEMM_ERR_UNSUPPORTED).
 *   max_norm >= 0, not NaN (GEMM_ERR_UNSUPPORTED otherwise); infinite: the
 *     factor is 1 for an infinite norm too
 *   Everything else as grad_norm; workspace is needed without `given` only.
 * A norm that is NaN makes every gradient NaN; an infinite one under a finite
 * max_norm zeros (NaN for infinities).
 */
gemm_status grad_clip(int64_t n, const void *const *grads, void *const *out, const int64_t *sizes, const int *types,
                      float max_norm, const float *given, float *norm, void *workspace, size_t workspace_bytes,
                      hipStream_t stream);

size_t grad_workspace_bytes(int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* TILEGEMM_LAYERS_H */
