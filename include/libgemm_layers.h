/*
 * libgemm_layers — what the feed-forward layer of a language model needs
 * around its products: the product with its bias, activation and residual in
 * the epilogue, its gradients, a whole layer of experts for a few tokens, and
 * the orthogonalised update of its weights.
 *
 *   gemm_linear               C <- act(alpha * A * B + bias) + beta * R
 *   gemm_linear_backward      D <- (alpha * A * B) act'(Z), and its column sums
 *   gemm_activation_backward  D <- A act'(Z), and its column sums
 *   gemm_experts_layer        tokens -> their experts' gated layers, weighted
 *                             and added
 *   gemm_orthogonalize        O <- alpha * (G brought near its orthogonal
 *                             factor) + beta * O
 *   gemm_linear_kernel_name, gemm_linear_backward_kernel_name,
 *   gemm_orthogonalize_kernel_name   the kernel a call would launch (host
 *                             only; "" for an empty problem, NULL for invalid
 *                             arguments)
 *   gemm_*_workspace_size     bytes of workspace a call needs (host only; 0
 *                             for sizes out of range)
 *
 * Ownership, synchronisation, streams and errors are libgemm.h's: the caller
 * owns every buffer, a call only enqueues on `stream`, keeps nothing between
 * calls, and may be captured into a graph; every argument that the host can
 * see is checked before any HIP call, and an invalid call changes nothing.
 * A workspace is 16-byte aligned device memory of at least the size asked
 * for, holds nothing between calls, and is used by one call at a time: two
 * calls (or two graphs) that share an output or a workspace must be ordered
 * by the caller.  Sums are formed in fp32 in an order that the arguments
 * decide (sizes, alignment, workspace), so a call gives the same result on
 * every run.
 *
 * 16-bit types below are bf16 or fp16, `in` saying which (GEMM_INPUT_BF16 or
 * GEMM_INPUT_F16).  Matrices are row-major with a leading dimension unless an
 * order says otherwise, and take any alignment of their element size; rows
 * that start at multiples of 16 bytes with extents of a multiple of 8
 * elements run fastest.
 *
 * Activations are those of gemm_activation_t, evaluated in fp32.  A NaN stays a
 * NaN in each of them and in its slope, ReLU's too (the epilogues of libgemm.h
 * give 0 there).  At infinities GELU and SiLU, and their slopes, take their
 * limits.
 */
#ifndef LIBGEMM_LAYERS_H
#define LIBGEMM_LAYERS_H

#include "libgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest sizes of gemm_experts_layer. */
#define GEMM_LAYER_MAX_TOKENS 64
#define GEMM_LAYER_MAX_EXPERTS 1024
#define GEMM_LAYER_MAX_TOP_K 32
/* Largest number of steps of gemm_orthogonalize. */
#define GEMM_ORTHOGONALIZE_MAX_STEPS 32

typedef enum gemm_weights_t {
    GEMM_WEIGHTS_SAME = 0, /* of the activations' type */
    GEMM_WEIGHTS_E4M3 = 1, /* 8-bit codes with block scales */
    GEMM_WEIGHTS_E5M2 = 2
} gemm_weights_t;

/* Bytes of workspace of gemm_linear and gemm_linear_backward.  From 1024 rows
 * and columns on, where K or N is not a multiple of 8, it holds copies of A and B. */
size_t gemm_linear_workspace_size(int64_t M, int64_t N, int64_t K);

/* Z = alpha * A * B + bias,  C = act(Z) + beta * R.
 *   A        M x K, 16-bit, row-major (lda >= K).
 *   B        K x N, of A's type, in either order: column-major (ldb >= K) is
 *            a weight stored one row per output, row-major (ldb >= N) one row
 *            per input.
 *   bias     N values of A's type, or NULL.
 *   R        M x N of C's type, ldr >= N; read only when beta != 0, and then
 *            not NULL.  R may be C itself (the same address and leading
 *            dimension); any other overlap is refused.
 *   C        M x N of typeC: A's type or fp32; ldc >= N.
 *   Z        M x N of A's type, ldz >= N, or NULL: the activation's input,
 *            which gemm_linear_backward reads.
 * alpha * A * B, the bias, the activation and the residual are fp32; C and Z
 * are each rounded once, to nearest even.  alpha == 0 or K == 0: A and B are
 * not read and the product is 0 (whatever alpha is, where K == 0).  N at most
 * 2^28 here and in both gradients (GEMM_ERR_UNSUPPORTED beyond).
 *   workspace   gemm_linear_workspace_size() bytes.  It may be NULL (with 0
 *            bytes): calls of few rows may then run slower, and give sums in
 *            another order. */
gemm_status_t gemm_linear(int64_t M, int64_t N, int64_t K, float alpha,
                          const void *A, int64_t lda, const void *B, int64_t ldb,
                          gemm_order_t orderB, gemm_input_t in, const void *bias,
                          gemm_activation_t act, float beta, const void *R, int64_t ldr,
                          void *C, int64_t ldc, gemm_output_t typeC, void *Z, int64_t ldz,
                          void *workspace, size_t workspace_bytes, hipStream_t stream);

const char *gemm_linear_kernel_name(int64_t M, int64_t N, int64_t K, float alpha,
                                    const void *A, int64_t lda, const void *B, int64_t ldb,
                                    gemm_order_t orderB, gemm_input_t in, const void *bias,
                                    gemm_activation_t act, float beta, const void *R, int64_t ldr,
                                    void *C, int64_t ldc, gemm_output_t typeC, void *Z,
                                    int64_t ldz, void *workspace, size_t workspace_bytes);

/* The gradient that a product brings to an activation, taken through it:
 *   D = (alpha * A * B) * act'(Z),   dbias_j <- sum over i of D(i, j) + beta * dbias_j.
 * With C = act(Z), Z = X * W1 + b1 and Y = C * W2: A is the gradient of Y, B
 * is W2 transposed, D the gradient of Z and dbias that of b1; the gradients
 * of X and W1 are then products of D.
 *   A, B     as for gemm_linear.
 *   Z        M x N of A's type, ldz >= N.  Not read when act is GEMM_ACT_NONE
 *            (and may then be NULL).  ReLU's slope at 0 is 0; where Z <= 0 its
 *            D is 0 whatever the gradient, infinities and NaN too.
 *   D        M x N of typeD (A's type or fp32), ldd >= N, not overlapping
 *            what is read; D may be Z itself where it has its type (the same
 *            address and leading dimension).
 *   dbias    N floats, or NULL.  It sums D before D is rounded.  beta == 0
 *            does not read it.
 *   workspace   gemm_linear_workspace_size() bytes, needed with dbias; else
 *            as for gemm_linear. */
gemm_status_t gemm_linear_backward(int64_t M, int64_t N, int64_t K, float alpha,
                                   const void *A, int64_t lda, const void *B, int64_t ldb,
                                   gemm_order_t orderB, gemm_input_t in, const void *Z,
                                   int64_t ldz, gemm_activation_t act, void *D, int64_t ldd,
                                   gemm_output_t typeD, float beta, float *dbias,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

const char *gemm_linear_backward_kernel_name(int64_t M, int64_t N, int64_t K, float alpha,
                                             const void *A, int64_t lda, const void *B,
                                             int64_t ldb, gemm_order_t orderB, gemm_input_t in,
                                             const void *Z, int64_t ldz, gemm_activation_t act,
                                             void *D, int64_t ldd, gemm_output_t typeD,
                                             float beta, float *dbias, void *workspace,
                                             size_t workspace_bytes);

/* Bytes of workspace of gemm_activation_backward. */
size_t gemm_activation_backward_workspace_size(int64_t M, int64_t N);

/* The same where no product makes the incoming gradient: D = A * act'(Z),
 * dbias_j <- sum over i of D(i, j) + beta * dbias_j.
 *   A        M x N of typeA (fp32 or 16-bit), lda >= N.
 *   Z        M x N of typeZ (fp32 or 16-bit), ldz >= N; not read when act is
 *            GEMM_ACT_NONE.
 *   D        M x N of typeD (fp32 or 16-bit), ldd >= N, or NULL (the sums
 *            alone).  D may be A or Z itself where it has its type (the same
 *            address and leading dimension).
 *   dbias    N floats, or NULL.  One of D and dbias is given.
 *   workspace   gemm_activation_backward_workspace_size() bytes, needed with
 *            dbias. */
gemm_status_t gemm_activation_backward(int64_t M, int64_t N, const void *A, int64_t lda,
                                       gemm_input_t typeA, const void *Z, int64_t ldz,
                                       gemm_input_t typeZ, gemm_activation_t act, void *D,
                                       int64_t ldd, gemm_output_t typeD, float beta,
                                       float *dbias, void *workspace, size_t workspace_bytes,
                                       hipStream_t stream);

/* Bytes of workspace of gemm_experts_layer. */
size_t gemm_experts_layer_workspace_size(int64_t tokens, int64_t experts, int64_t top_k,
                                         int64_t D, int64_t H);

/* A layer of experts for a few tokens, whole, in two kernels.  For token t
 * with experts e_j = ids[t*top_k + j] and weights w_j = weights[t*top_k + j]:
 *   h_j = act(Up_e[0 .. H) x_t) * (Up_e[H .. 2H) x_t),
 *   Y_t <- sum over j of w_j Down_e h_j + beta * Y_t.
 *   X        tokens x D, 16-bit, ldx >= D.
 *   ids, weights   tokens x top_k, as gemm_experts_route gives them.  An id
 *            outside [0, experts) takes no part, whatever its weight; an id
 *            that a token holds twice counts with the sum of its weights.
 *   up       expert e's 2H x D weights at up + e*stride_up, element (r, k) at
 *            r*ld_up + k: the rows of the activated half, then those of the
 *            half it multiplies.
 *   down     D x H weights, element (d, h) at d*ld_down + h of expert e.
 *   type     GEMM_WEIGHTS_SAME: weights of X's type, the scales unused; else
 *            codes of a byte, and element (r, k) is multiplied by
 *            scale[(k/128)*lds + r/128] of its expert (fp32, strides
 *            stride_scale_*; the blocks of 128 of gemm_f8_block_quantize with
 *            block 128).  Products take the codes' values in X's type,
 *            exactly; X is not rounded further.
 *   X, up and down are 16-byte aligned, their rows' and experts' strides
 *            multiples of 16 bytes; the bytes of a row up to the next
 *            multiple of 16 are read and must be readable; their values are
 *            not used.  Scales are 4-byte aligned.
 *   act      GEMM_ACT_RELU, _GELU or _SILU.
 *   Y        tokens x D of typeY (X's type or fp32), ldy >= D; beta == 0 does
 *            not read it.  A token without experts gets beta * Y.
 *   workspace   gemm_experts_layer_workspace_size() bytes.
 * Sums are fp32; w h is formed in fp32 and enters the second product as two
 * pieces of X's type, which hold 16 of its 24 bits in bf16 and 22 in fp16 (there
 * from 2^-10 up to 2^20: below in steps of 2^-31, beyond it gives infinities
 * or NaN).
 * At least one expert, one choice, no more choices than experts, and H >= 1
 * (GEMM_ERR_INVALID_ARG).  At most GEMM_LAYER_MAX_TOKENS tokens, _EXPERTS
 * experts and _TOP_K choices (GEMM_ERR_UNSUPPORTED beyond: gemm_experts_f8
 * takes more tokens, with 8-bit operands); H at most 2^17, ldx 2^23, ld_up and
 * ld_down 2^25. */
gemm_status_t gemm_experts_layer(int64_t tokens, int64_t experts, int64_t top_k, int64_t D,
                                 int64_t H, const void *X, int64_t ldx, gemm_input_t in,
                                 const int32_t *ids, const float *weights, gemm_weights_t type,
                                 const void *up, int64_t ld_up, int64_t stride_up,
                                 const float *scale_up, int64_t lds_up, int64_t stride_scale_up,
                                 const void *down, int64_t ld_down, int64_t stride_down,
                                 const float *scale_down, int64_t lds_down,
                                 int64_t stride_scale_down, gemm_activation_t act, float beta,
                                 void *Y, int64_t ldy, gemm_output_t typeY, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace of gemm_orthogonalize. */
size_t gemm_orthogonalize_workspace_size(int64_t M, int64_t N, int64_t batch);

/* Newton-Schulz steps that bring the singular values of each M x N matrix G
 * towards 1 and keep its singular vectors (an update's step in Muon):
 *   X <- G / max(|G|, eps), |G| the root of the sum of squares;
 *   `steps` times, on X or (when M > N) its transpose:
 *     A = X X^T,   X <- a X + (b A + c A^2) X;
 *   O <- alpha * X + beta * O.
 *   G        M x N of type in (fp32, bf16 or fp16), ldg >= N.
 *   coefficients   3*steps floats in host memory, a, b, c of each step, read
 *            before the call returns; NULL: 3.4445, -4.7750, 2.0315 in each.
 *   eps      >= 0.  A matrix of zeros gives beta * O whatever it is.
 *   O        M x N of typeO (any), ldo >= N; beta == 0 does not read it.
 *            O = alpha * X + beta * O is a weight's step with its decay.  O
 *            may not overlap G.
 *   batch    matrices strideG and strideO elements apart; strideO is at
 *            least what a matrix of O spans, (M - 1)*ldo + N.
 *   workspace   gemm_orthogonalize_workspace_size() bytes.
 * The sum of squares is formed in 64 bits.  X is kept between the steps to 22
 * bits of each element or to 2^-35 of its norm, whichever is more, also where
 * G's norm is far below eps.  The products take fp16 roundings of X, of E = A
 * - s I with s the mean of A's eigenvalues, and of (b + 2 c s) E + c E^2, and
 * add in fp32, which leaves X between 2^-16 and 2^-9 of its norm from the
 * exact steps' (five usual steps on matrices of 64 x 64 to 2048 x 2048; random
 * ones 2^-10 to 2^-12): about bf16's own rounding or less.  All are scaled by
 * powers of two so that steps whose singular values stay below 2 and whose
 * coefficients stay below 16 in magnitude are within fp16's range; others may
 * give infinities or NaN.  A matrix with an infinity or a NaN gives NaN
 * throughout.
 * steps in 1 .. GEMM_ORTHOGONALIZE_MAX_STEPS; M and N at most 2^20, and less
 * than 2^24 blocks of 64 x 64 in a matrix (GEMM_ERR_UNSUPPORTED beyond). */
gemm_status_t gemm_orthogonalize(int64_t M, int64_t N, const void *G, int64_t ldg,
                                 gemm_input_t in, int64_t steps, const float *coefficients,
                                 float eps, float alpha, float beta, void *O, int64_t ldo,
                                 gemm_output_t typeO, int64_t batch, int64_t strideG,
                                 int64_t strideO, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

const char *gemm_orthogonalize_kernel_name(int64_t M, int64_t N, int64_t batch);

#ifdef __cplusplus
}
#endif

#endif /* LIBGEMM_LAYERS_H */
