/*
 * libgemm_experts — 8-bit products whose operands carry one fp32 scale for
 * each block of 128 along the contracted dimension, and what a layer of
 * experts needs around them: making such operands, the products over the
 * rows each expert was given, and the routing that gives them.
 *
 *   gemm_f8_block_quantize   rows -> 8-bit codes and scales, in the direction
 *                            of a forward product, of a backward one, or both
 *   gemm_f8_block            C <- alpha * A * B + beta * C
 *   gemm_experts_f8          the same, each run of A's rows with its own B
 *   gemm_experts_f8_wgrad    the same, each run of the contracted dimension
 *                            with its own C (the experts' weight gradients)
 *   gemm_experts_route       router logits -> chosen experts, weights, and
 *                            the rows of each expert
 *   gemm_experts_route_backward  d weights -> d logits
 *   gemm_f8_block_kernel_name, gemm_experts_f8_kernel_name,
 *   gemm_experts_f8_wgrad_kernel_name   the kernel a call would launch (host
 *                            only; "" for an empty problem, NULL for invalid
 *                            arguments)
 *   gemm_experts_rows, gemm_experts_route_workspace_size   sizes of outputs
 *                            and of the router's workspace (host only)
 *
 * Block-scaled operands
 *   An operand of R rows (rows of A, columns of B) contracted over K is
 *     codes   R x K bytes, E4M3 or E5M2, contiguous along K: element (r, k)
 *             at codes[r*ld + k]; 16-byte aligned, ld a multiple of 16, at
 *             least K.  Whole 16-byte chunks are read, so the bytes from K to
 *             the next multiple of 16 of a row must be readable; their values
 *             are not used.
 *     scale   ceil(K/128) x ceil(R/block) floats, contiguous along the rows:
 *             element (r, k) is multiplied by
 *             scale[(k/128)*lds + r/block].  block is 1 (a scale for each
 *             row: activations, gradients) or 128 (a scale for each
 *             128 x 128 block: weights).  4-byte aligned, lds at least
 *             ceil(R/block) where there is more than one row of scales.
 *   Any K, M and N are accepted; the last block of K may be short.
 *
 * Arithmetic
 *   C(i, j) = alpha * sum over blocks kb of
 *             scaleA * scaleB * (sum over the block's k of A(i, k) B(j, k))
 *             + beta * C(i, j).
 *   A block's 128 products are summed by one matrix instruction into fp32,
 *   with that instruction's precision (see gemm_f8 in libgemm.h: products
 *   below 2^-13 of the largest of 8 neighbours are cut off); the scaled block
 *   sums are added in fp32, in order of k within each of up to 8 shares of the
 *   blocks, and the shares' sums in a fixed order.  How many shares there are
 *   goes by the sizes of the call, so the result is the same on every run.
 *   The two scales are multiplied first, in fp32: where their product is
 *   subnormal, 0 or infinite there, that is what the sum is multiplied by,
 *   though the sum times both might be in range.
 *   The rest is gemm_f8's: alpha*acc +
 *   beta*C in fp32, rounded to nearest-even into typeC; beta == 0 does not
 *   read C; alpha == 0 or K == 0 gives beta * C.  NaN and infinite codes and
 *   scales propagate.
 *
 * Ownership, synchronisation, streams and errors are libgemm.h's: the caller
 * owns every buffer, a call only enqueues on `stream`, keeps nothing between
 * calls, and may be captured into a graph; every argument that the host can
 * see is checked before any HIP call, and an invalid call changes nothing.
 * A call that one launch of fewer than 2^32 threads does not hold (2^23 tiles
 * of a product, 2^24 blocks of 64 rows and 128 columns to quantise) is
 * GEMM_ERR_UNSUPPORTED.
 * What only the device can see (offsets, indices) is held within the
 * documented buffers there: bad values give wrong rows, never an access
 * outside.  Two calls that share an output or a workspace must be ordered by
 * the caller.
 */
#ifndef LIBGEMM_EXPERTS_H
#define LIBGEMM_EXPERTS_H

#include "libgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest sizes of gemm_experts_route. */
#define GEMM_ROUTE_MAX_EXPERTS 1024
#define GEMM_ROUTE_MAX_TOP_K 32
#define GEMM_ROUTE_MAX_GROUPS 64

typedef enum gemm_score_t {
    GEMM_SCORE_SOFTMAX = 0, /* over the token's experts */
    GEMM_SCORE_SIGMOID = 1  /* of each logit */
} gemm_score_t;

/* X (rows x cols, of type in) to 8-bit codes and scales.
 * For each block, with F the format's largest finite value (448, 57344):
 *   s = max(max |x| / F, 2^-126),   code = nearest(x / s), ties to even,
 * both quotients rounded to fp32 first, the code saturated; the value it
 * stands for is code * s.  A block that holds an infinity or a NaN gets the
 * scale NaN and the NaN code 0x7F throughout.
 *   X           element (r, c) of batch entry b at
 *               X[b*strideX + index(r)*ldx + c]; ldx >= cols; aligned to its
 *               element size.
 *   index       NULL: index(r) = r, and X has `rows` rows.  Else `rows` int32
 *               on the device (the rows of a dispatch): row r of the result
 *               is X's row index[r], of x_rows; an index outside [0, x_rows)
 *               gives a row of zeros.  batch must be 1.
 *   block       1 or 128, as above.
 *   Q, S        for products that contract over the columns (the rows of X
 *               stay rows): codes at Q[b*strideQ + r*ldq + c], scales at
 *               S[b*strideS + (c/128)*lds + r/block].  NULL, NULL: not wanted.
 *   QT, ST      for products that contract over the rows (a weight's use in
 *               a backward product, activations and gradients in a weight's
 *               gradient): codes at QT[b*strideQT + c*ldqt + r], scales at
 *               ST[b*strideST + (r/128)*ldst + c/block].  NULL, NULL: not
 *               wanted.  At least one direction must be wanted.  With block
 *               128 the two hold the same codes and scales.
 * ldq >= cols, lds >= ceil(rows/block), ldqt >= rows, ldst >=
 * ceil(cols/block) (lds and ldst only where there is more than one row of
 * scales); slices of one output must not overlap when batch > 1.
 * Nothing outside the rows x cols codes and their scales is written.
 * rows == 0, cols == 0 or batch == 0: nothing is done. */
gemm_status_t gemm_f8_block_quantize(int64_t rows, int64_t cols, const void *X, int64_t ldx,
                                     gemm_input_t in, const int32_t *index, int64_t x_rows,
                                     gemm_f8_format_t format, int64_t block,
                                     uint8_t *Q, int64_t ldq, float *S, int64_t lds,
                                     uint8_t *QT, int64_t ldqt, float *ST, int64_t ldst,
                                     int64_t batch, int64_t strideX, int64_t strideQ,
                                     int64_t strideS, int64_t strideQT, int64_t strideST,
                                     hipStream_t stream);

/* C (M x N) <- alpha * A * B + beta * C, A an operand of M rows, B one of N
 * rows (B's element (k, j) is code row j, column k).  C of typeC, in either
 * order.  batch, strideA and strideB (codes; multiples of 16), strideScaleA
 * and strideScaleB (floats) and strideC (elements) as for gemm_f8; 0 shares
 * an operand or its scales.  lda or ldb of 4 MiB or more is
 * GEMM_ERR_UNSUPPORTED. */
gemm_status_t gemm_f8_block(int64_t M, int64_t N, int64_t K, float alpha,
                            const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                            const float *scaleA, int64_t ldsa, int64_t blockA,
                            const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                            const float *scaleB, int64_t ldsb, int64_t blockB,
                            float beta, void *C, int64_t ldc, gemm_order_t orderC,
                            gemm_output_t typeC, int64_t batch, int64_t strideA,
                            int64_t strideB, int64_t strideScaleA, int64_t strideScaleB,
                            int64_t strideC, hipStream_t stream);

/* The experts' products: rows offsets[e] .. offsets[e+1]-1 of A times B_e,
 * into the same rows of C (row-major).  A has `rows` rows, a scale for each
 * row (block 1); B_e is at B + e*strideB with scales at
 * scaleB + e*strideScaleB, blockB 1 or 128.
 *   offsets     experts + 1 int32 on the device, not falling, within
 *               [0, rows]; an empty segment is allowed.  A segment that
 *               falls or leaves [0, rows] is cut to what lies within.
 * Rows of C outside every segment are left as they were.  rows is the
 * number of rows the buffers have: the work goes by the segments.  The
 * kernel is chosen by the mean length, so one expert that has most of a small
 * call's rows takes longer than as many rows spread out.  lda and ldb as for
 * gemm_f8_block.  The gradient with respect to A is this call with B_e
 * quantised the other way. */
gemm_status_t gemm_experts_f8(int64_t experts, int64_t rows, int64_t N, int64_t K,
                              const int32_t *offsets, float alpha,
                              const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                              const float *scaleA, int64_t ldsa,
                              const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                              const float *scaleB, int64_t ldsb, int64_t blockB,
                              int64_t strideB, int64_t strideScaleB,
                              float beta, void *C, int64_t ldc, gemm_output_t typeC,
                              hipStream_t stream);

/* The experts' weight gradients: C_e (M x N, row-major, at C + e*strideC) <-
 * alpha * sum over t in [offsets[e], offsets[e+1]) of A(i, t) B(t, j) + beta * C_e.
 * A is an operand of M rows and B one of N rows, both contracted over `rows`
 * positions with block 1 (QT and ST of gemm_f8_block_quantize).  offsets as
 * for gemm_experts_f8; a segment that is not empty starts at a multiple of
 * 128, so that no block of 128 holds rows of two experts (gemm_experts_route's
 * align); others give wrong sums.  An empty segment, wherever it starts, gives
 * beta * C_e.  lda and ldb as for gemm_f8_block: fewer than 4 Mi positions. */
gemm_status_t gemm_experts_f8_wgrad(int64_t experts, int64_t M, int64_t N, int64_t rows,
                                    const int32_t *offsets, float alpha,
                                    const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                                    const float *scaleA, int64_t ldsa,
                                    const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                                    const float *scaleB, int64_t ldsb,
                                    float beta, void *C, int64_t ldc, int64_t strideC,
                                    gemm_output_t typeC, hipStream_t stream);

const char *gemm_f8_block_kernel_name(int64_t M, int64_t N, int64_t K, float alpha,
                                      const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                                      const float *scaleA, int64_t ldsa, int64_t blockA,
                                      const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                                      const float *scaleB, int64_t ldsb, int64_t blockB,
                                      float beta, void *C, int64_t ldc, gemm_order_t orderC,
                                      gemm_output_t typeC, int64_t batch, int64_t strideA,
                                      int64_t strideB, int64_t strideScaleA,
                                      int64_t strideScaleB, int64_t strideC);
const char *gemm_experts_f8_kernel_name(int64_t experts, int64_t rows, int64_t N, int64_t K,
                                        const int32_t *offsets, float alpha,
                                        const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                                        const float *scaleA, int64_t ldsa,
                                        const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                                        const float *scaleB, int64_t ldsb, int64_t blockB,
                                        int64_t strideB, int64_t strideScaleB,
                                        float beta, void *C, int64_t ldc, gemm_output_t typeC);
const char *gemm_experts_f8_wgrad_kernel_name(
    int64_t experts, int64_t M, int64_t N, int64_t rows, const int32_t *offsets, float alpha,
    const uint8_t *A, int64_t lda, gemm_f8_format_t formatA, const float *scaleA, int64_t ldsa,
    const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb,
    float beta, void *C, int64_t ldc, int64_t strideC, gemm_output_t typeC);

/* Rows that gemm_experts_route's segments need at most:
 * tokens*top_k + min(experts, tokens*top_k)*(align - 1); 0 for sizes out of
 * range. */
int64_t gemm_experts_rows(int64_t tokens, int64_t experts, int64_t top_k, int64_t align);

/* Bytes of workspace gemm_experts_route needs (0 for sizes out of range). */
size_t gemm_experts_route_workspace_size(int64_t tokens, int64_t experts, int64_t top_k);

/* Chooses top_k of the experts for each token and lays their rows out.
 * For token t with logits l (fp32, bf16 or fp16; ldl >= experts between
 * tokens):
 *   scores      s = softmax(l) or sigmoid(l)
 *   keys        s + bias (fp32 per expert; NULL: none), which only the
 *               choice uses
 *   groups      experts in `groups` equal runs; when groups > 1, a group's
 *               rank is the sum of its group_top (1 or 2) largest keys, and
 *               only the top_groups of largest rank take part
 *   choice      the top_k largest keys, in falling order
 *   weights     s of the chosen, divided by their sum when `renormalise`
 *               (0 where that sum is 0 in 64 bits: sigmoids of logits below
 *               -709), times scale
 * Keys and ranks are compared as if computed exactly (64 bits decide where
 * 32 are too close); equal ones go to the lower index.  A logit, or a logit's
 * key, of -infinity or NaN marks an expert that cannot be chosen and adds
 * nothing to its group's rank; groups without others come last.  Where fewer
 * than top_k can be chosen, the other slots hold id -1 and weight 0.  Under
 * softmax, a token with a NaN or +infinity among its logits has no scores:
 * its ids are -1 and its weights NaN.
 *   keep        one byte per token (NULL: all): a token whose byte is 0 (the
 *               padding of a batch) gets ids -1, weights 0 and no rows.
 *   ids, weights   tokens x top_k, contiguous.
 *   offsets     experts + 1: expert e's segment is rows offsets[e] ..
 *               offsets[e+1]-1, its length rounded up to a multiple of align
 *               (1 .. 65536).
 *   row_tokens  `rows` entries: the token of each row, by rising token (a
 *               token gives an expert one row); -1 in a segment's filling
 *               and behind the last segment.
 *   places      tokens x top_k: the row of each slot, or -1.
 *   rows        at least gemm_experts_rows(tokens, experts, top_k, align).
 * offsets, row_tokens and places are all given or all NULL (ids and weights
 * only; align and rows are then not used).
 *   workspace   16-byte aligned, gemm_experts_route_workspace_size() bytes on
 *               the device, not needed without offsets; it holds nothing
 *               between calls.
 * At most GEMM_ROUTE_MAX_EXPERTS experts, _TOP_K choices and _GROUPS groups
 * (GEMM_ERR_UNSUPPORTED beyond); top_k at most the experts of top_groups
 * groups; rows below 2^31.  tokens == 0: offsets are 0 and row_tokens -1. */
gemm_status_t gemm_experts_route(int64_t tokens, int64_t experts, const void *logits, int64_t ldl,
                                 gemm_input_t in, const float *bias, const uint8_t *keep,
                                 gemm_score_t score, int64_t groups, int64_t top_groups,
                                 int64_t group_top, int64_t top_k, int renormalise, float scale,
                                 int32_t *ids, float *weights, int64_t align, int64_t rows,
                                 int32_t *offsets, int32_t *row_tokens, int32_t *places,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The gradient of gemm_experts_route's weights with respect to the logits
 * (the choice is held fixed, the bias has no gradient): d_logits (tokens x
 * experts, the logits' type, ldd >= experts) is written whole, zero where
 * nothing flows.  ids as gemm_experts_route gave them; an id outside
 * [0, experts) takes no part (its weight was 0), and a token without ids has
 * zero gradients.  d_weights tokens x top_k. */
gemm_status_t gemm_experts_route_backward(int64_t tokens, int64_t experts, const void *logits,
                                          int64_t ldl, gemm_input_t in, gemm_score_t score,
                                          int64_t top_k, int renormalise, float scale,
                                          const int32_t *ids, const float *d_weights,
                                          void *d_logits, int64_t ldd, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGEMM_EXPERTS_H */
