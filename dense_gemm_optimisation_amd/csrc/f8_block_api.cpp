// C ABI of libgemm_experts.h: argument validation, canonicalisation and
// dispatch.  Every check runs before any HIP call, so an invalid call has no
// effect.  A column-major C is computed as its row-major transpose, which
// swaps the two operands: both are contiguous along the contracted dimension.
#include "libgemm_experts.h"

#include <cstdint>
#include <initializer_list>

#include "arg_checks.hpp"
#include "f8_block.hpp"

using namespace libgemm;

namespace libgemm {
// The test switches that gemm_test_switches set (api.cpp).
int test_switches();
}  // namespace libgemm

namespace {

static_assert(GEMM_ROUTE_MAX_EXPERTS == ROUTE_MAX_EXPERTS && GEMM_ROUTE_MAX_TOP_K == ROUTE_MAX_TOP_K,
              "the header's limits are the kernels'");

gemm_status_t status_of(hipError_t e) {
    if (e == hipErrorInvalidConfiguration) return GEMM_ERR_UNSUPPORTED;
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

bool misaligned(const void *p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool format_ok(int f) { return f == GEMM_F8_E4M3 || f == GEMM_F8_E5M2; }
bool block_ok(int64_t b) { return b == 1 || b == 128; }
bool output_ok(int t) { return t == GEMM_OUTPUT_F32 || t == GEMM_OUTPUT_BF16 || t == GEMM_OUTPUT_F16; }
bool input_ok(int t) { return t == GEMM_INPUT_F32 || t == GEMM_INPUT_BF16 || t == GEMM_INPUT_F16; }
int type_bytes(int t) { return t == 0 ? 4 : 2; }  // of gemm_output_t and gemm_input_t alike

// Sizes far enough from the ends of int64 for every extent below to be computed.
constexpr int64_t MOST = int64_t(1) << 40;
bool any_over(std::initializer_list<int64_t> sizes) {
    for (int64_t s : sizes)
        if (s < 0 || s > MOST) return true;
    return false;
}
// (n - 1) * stride + span elements, of up to 4 bytes, leave the address space.
constexpr int64_t MOST_EXTENT = INT64_MAX / 8;
bool extent_over(int64_t n, int64_t stride, int64_t span) {
    return span > MOST_EXTENT || (n > 1 && (too_big(n - 1, stride) || (n - 1) * stride > MOST_EXTENT - span));
}

// Checks one operand of R rows over K and gives the ranges it touches.  The
// sizes are within MOST.
bool operand_ok(const uint8_t *x, int64_t ld, int format, const float *s, int64_t lds, int64_t block,
                int64_t R, int64_t K, int64_t batch, int64_t stride, int64_t sstride, Range &rx,
                Range &rs) {
    if (x == nullptr || s == nullptr || !format_ok(format) || !block_ok(block)) return false;
    if (misaligned(x, 16) || misaligned(s, 4) || ld % 16 != 0 || ld < K) return false;
    if (batch > 1 && stride % 16 != 0) return false;
    const int64_t sr = ceil_div(R, block), kb = ceil_div(K, 128);
    if (kb > 1 && lds < sr) return false;
    const int64_t span_x = (R - 1) * ld + K, span_s = (kb - 1) * lds + sr;
    if (extent_over(batch, stride, span_x) || extent_over(batch, sstride, span_s)) return false;
    rx = range_of(x, span_x, batch, stride, 1);
    rs = range_of(s, span_s, batch, sstride, 4);
    return true;
}

BlockOperand operand(const uint8_t *x, int64_t ld, int format, const float *s, int64_t lds, int64_t block,
                     int64_t stride, int64_t sstride) {
    return BlockOperand{x, ld, stride, s, lds, sstride, block == 128 ? 7 : 0, format == GEMM_F8_E5M2};
}

constexpr int64_t MOST_LD = int64_t(1) << 22;  // a tile's rows are addressed with 32-bit offsets

// Validates a product of any kind and builds its canonical problem; k tells
// what runs (None: nothing to do).
gemm_status_t block_plan(Segments segments, int64_t M, int64_t N, int64_t K, const int32_t *offsets,
                         float alpha, const uint8_t *A, int64_t lda, int formatA, const float *scaleA,
                         int64_t ldsa, int64_t blockA, const uint8_t *B, int64_t ldb, int formatB,
                         const float *scaleB, int64_t ldsb, int64_t blockB, float beta, void *C,
                         int64_t ldc, int orderC, int typeC, int64_t batch, int64_t strideA,
                         int64_t strideB, int64_t strideScaleA, int64_t strideScaleB, int64_t strideC,
                         BlockProblem &p, BlockKernel &k) {
    k = BlockKernel::None;
    if (!output_ok(typeC) || !valid_order(orderC) || !format_ok(formatA) || !format_ok(formatB) ||
        !block_ok(blockA) || !block_ok(blockB))
        return GEMM_ERR_INVALID_ARG;
    if (any_over({M, N, K, batch, lda, ldb, ldsa, ldsb, ldc}) || strideA < 0 || strideB < 0 ||
        strideScaleA < 0 || strideScaleB < 0 || strideC < 0)
        return GEMM_ERR_INVALID_ARG;
    const int64_t min_ldc = orderC == GEMM_ROW_MAJOR ? N : M;
    if (ldc < (min_ldc > 1 ? min_ldc : 1)) return GEMM_ERR_INVALID_ARG;
    if (too_big(M, ldc) || too_big(N, ldc) || too_big(M, lda) || too_big(N, ldb) ||
        too_big(ceil_div(K, 128), ldsa) || too_big(ceil_div(K, 128), ldsb))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || batch == 0) return GEMM_OK;

    const int64_t slices_a = segments == Segments::None ? batch : 1;
    const int64_t slices_b = segments == Segments::Contracted ? 1 : batch;
    const int64_t slices_c = segments == Segments::Rows ? 1 : batch;
    const int esize = type_bytes(typeC);
    const int64_t span_c = span(M, N, orderC, ldc);
    if (C == nullptr || misaligned(C, esize)) return GEMM_ERR_INVALID_ARG;
    if ((slices_c > 1 && strideC < span_c) || extent_over(slices_c, strideC, span_c)) return GEMM_ERR_INVALID_ARG;
    const Range rc = range_of(C, span_c, slices_c, strideC, esize);
    if (segments != Segments::None) {
        if (offsets == nullptr || misaligned(offsets, 4)) return GEMM_ERR_INVALID_ARG;
        const int64_t limit = segments == Segments::Rows ? M : K;
        if (limit > INT32_MAX) return GEMM_ERR_INVALID_ARG;  // offsets are int32
        if (overlap(rc, range_of(offsets, batch + 1, 1, 0, 4))) return GEMM_ERR_INVALID_ARG;
    }
    const bool reads = K > 0 && alpha != 0.0f;
    if (reads) {
        Range ra, rsa, rb, rsb;
        if (!operand_ok(A, lda, formatA, scaleA, ldsa, blockA, M, K, slices_a, strideA, strideScaleA, ra, rsa) ||
            !operand_ok(B, ldb, formatB, scaleB, ldsb, blockB, N, K, slices_b, strideB, strideScaleB, rb, rsb))
            return GEMM_ERR_INVALID_ARG;
        if (overlap(rc, ra) || overlap(rc, rsa) || overlap(rc, rb) || overlap(rc, rsb))
            return GEMM_ERR_INVALID_ARG;
        if (lda >= MOST_LD || ldb >= MOST_LD) return GEMM_ERR_UNSUPPORTED;
    }
    p = BlockProblem{};
    p.segments = segments;
    p.K = reads ? K : 0;
    p.alpha = reads ? alpha : 0.0f;
    p.beta = beta;
    p.C = C;
    p.ldc = ldc;
    p.sC = slices_c > 1 ? strideC : 0;
    p.out = static_cast<int>(typeC);
    p.batch = batch;
    p.offsets = offsets;
    const BlockOperand a = operand(A, lda, formatA, scaleA, ldsa, blockA, slices_a > 1 ? strideA : 0,
                                   slices_a > 1 ? strideScaleA : 0);
    const BlockOperand b = operand(B, ldb, formatB, scaleB, ldsb, blockB, slices_b > 1 ? strideB : 0,
                                   slices_b > 1 ? strideScaleB : 0);
    const bool row = orderC == GEMM_ROW_MAJOR;
    p.M = row ? M : N;
    p.N = row ? N : M;
    p.a = row ? a : b;
    p.b = row ? b : a;
    const int switches = test_switches();
    k = block_choose(p, (switches & GEMM_TEST_FORCE_GENERAL) != 0, (switches & GEMM_TEST_NO_SPLITK) == 0);
    return GEMM_OK;
}

gemm_status_t block_run(gemm_status_t st, const BlockProblem &p, BlockKernel k, hipStream_t stream) {
    return st != GEMM_OK ? st : status_of(launch_block(k, p, stream));
}

const char *block_name(gemm_status_t st, BlockKernel k) {
    return st != GEMM_OK ? nullptr : block_kernel_name(k);
}

gemm_status_t dense_plan(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A, int64_t lda,
                         gemm_f8_format_t formatA, const float *scaleA, int64_t ldsa, int64_t blockA,
                         const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB, const float *scaleB,
                         int64_t ldsb, int64_t blockB, float beta, void *C, int64_t ldc,
                         gemm_order_t orderC, gemm_output_t typeC, int64_t batch, int64_t strideA,
                         int64_t strideB, int64_t strideScaleA, int64_t strideScaleB, int64_t strideC,
                         BlockProblem &p, BlockKernel &k) {
    return block_plan(Segments::None, M, N, K, nullptr, alpha, A, lda, formatA, scaleA, ldsa, blockA, B,
                      ldb, formatB, scaleB, ldsb, blockB, beta, C, ldc, orderC, typeC, batch, strideA,
                      strideB, strideScaleA, strideScaleB, strideC, p, k);
}

gemm_status_t rows_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, const int32_t *offsets,
                        float alpha, const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                        const float *scaleA, int64_t ldsa, const uint8_t *B, int64_t ldb,
                        gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb, int64_t blockB,
                        int64_t strideB, int64_t strideScaleB, float beta, void *C, int64_t ldc,
                        gemm_output_t typeC, BlockProblem &p, BlockKernel &k) {
    return block_plan(Segments::Rows, rows, N, K, offsets, alpha, A, lda, formatA, scaleA, ldsa, 1, B,
                      ldb, formatB, scaleB, ldsb, blockB, beta, C, ldc, GEMM_ROW_MAJOR, typeC, experts, 0,
                      strideB, 0, strideScaleB, 0, p, k);
}

gemm_status_t wgrad_plan(int64_t experts, int64_t M, int64_t N, int64_t rows, const int32_t *offsets,
                         float alpha, const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                         const float *scaleA, int64_t ldsa, const uint8_t *B, int64_t ldb,
                         gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb, float beta, void *C,
                         int64_t ldc, int64_t strideC, gemm_output_t typeC, BlockProblem &p,
                         BlockKernel &k) {
    return block_plan(Segments::Contracted, M, N, rows, offsets, alpha, A, lda, formatA, scaleA, ldsa, 1,
                      B, ldb, formatB, scaleB, ldsb, 1, beta, C, ldc, GEMM_ROW_MAJOR, typeC, experts, 0, 0,
                      0, 0, strideC, p, k);
}

// Sizes of a routing call in range; layout: its rows too.
bool route_sizes_ok(int64_t tokens, int64_t experts, int64_t top_k) {
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= GEMM_ROUTE_MAX_EXPERTS &&
           top_k >= 1 && top_k <= GEMM_ROUTE_MAX_TOP_K && top_k <= experts;
}

}  // namespace

extern "C" {

gemm_status_t gemm_f8_block_quantize(int64_t rows, int64_t cols, const void *X, int64_t ldx,
                                     gemm_input_t in, const int32_t *index, int64_t x_rows,
                                     gemm_f8_format_t format, int64_t block, uint8_t *Q, int64_t ldq,
                                     float *S, int64_t lds, uint8_t *QT, int64_t ldqt, float *ST,
                                     int64_t ldst, int64_t batch, int64_t strideX, int64_t strideQ,
                                     int64_t strideS, int64_t strideQT, int64_t strideST,
                                     hipStream_t stream) {
    if (!input_ok(in) || !format_ok(format) || !block_ok(block)) return GEMM_ERR_INVALID_ARG;
    if (any_over({rows, cols, batch, ldx}) || strideX < 0 || strideQ < 0 || strideS < 0 ||
        strideQT < 0 || strideST < 0)
        return GEMM_ERR_INVALID_ARG;
    if ((Q == nullptr) != (S == nullptr) || (QT == nullptr) != (ST == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (Q == nullptr && QT == nullptr) return GEMM_ERR_INVALID_ARG;
    if (index != nullptr && (any_over({x_rows}) || batch > 1)) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0 || batch == 0) return GEMM_OK;
    const int64_t held = index != nullptr ? x_rows : rows;
    const int esize = type_bytes(in);
    if (ldx < cols || too_big(held, ldx) || misaligned(X, esize) || misaligned(index, 4))
        return GEMM_ERR_INVALID_ARG;
    if (X == nullptr && held > 0) return GEMM_ERR_INVALID_ARG;
    const int64_t span_x = held > 0 ? (held - 1) * ldx + cols : 0;
    if (extent_over(batch, strideX, span_x)) return GEMM_ERR_INVALID_ARG;
    const Range rx = range_of(X, span_x, batch, strideX, esize);
    const Range ri = range_of(index, index != nullptr ? rows : 0, 1, 0, 4);
    Range out[4];
    int n = 0;
    struct Direction {
        const void *codes, *scales;
        int64_t ld, lds, stride, sstride, outer, inner;
    };
    for (const Direction &d : {Direction{Q, S, ldq, lds, strideQ, strideS, rows, cols},
                               Direction{QT, ST, ldqt, ldst, strideQT, strideST, cols, rows}}) {
        if (d.codes == nullptr) continue;
        const int64_t sr = ceil_div(d.outer, block), kb = ceil_div(d.inner, 128);
        if (any_over({d.ld, d.lds}) || d.ld < d.inner || (kb > 1 && d.lds < sr) || misaligned(d.scales, 4))
            return GEMM_ERR_INVALID_ARG;
        if (too_big(d.outer, d.ld) || too_big(kb, d.lds)) return GEMM_ERR_INVALID_ARG;
        const int64_t span_q = (d.outer - 1) * d.ld + d.inner, span_s = (kb - 1) * d.lds + sr;
        if (extent_over(batch, d.stride, span_q) || extent_over(batch, d.sstride, span_s))
            return GEMM_ERR_INVALID_ARG;
        if (batch > 1 && (d.stride < span_q || d.sstride < span_s)) return GEMM_ERR_INVALID_ARG;
        out[n++] = range_of(d.codes, span_q, batch, d.stride, 1);
        out[n++] = range_of(d.scales, span_s, batch, d.sstride, 4);
    }
    for (int i = 0; i < n; ++i) {
        if (overlap(out[i], rx) || overlap(out[i], ri)) return GEMM_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GEMM_ERR_INVALID_ARG;
    }
    QuantizeArgs a{rows, cols, X, ldx, static_cast<int>(in), index, x_rows, format == GEMM_F8_E5M2,
                   static_cast<int>(block), Q, ldq, S, lds, QT, ldqt, ST, ldst, batch, strideX, strideQ,
                   strideS, strideQT, strideST};
    return status_of(launch_quantize(a, stream));
}

gemm_status_t gemm_f8_block(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A, int64_t lda,
                            gemm_f8_format_t formatA, const float *scaleA, int64_t ldsa, int64_t blockA,
                            const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB, const float *scaleB,
                            int64_t ldsb, int64_t blockB, float beta, void *C, int64_t ldc,
                            gemm_order_t orderC, gemm_output_t typeC, int64_t batch, int64_t strideA,
                            int64_t strideB, int64_t strideScaleA, int64_t strideScaleB, int64_t strideC,
                            hipStream_t stream) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = dense_plan(M, N, K, alpha, A, lda, formatA, scaleA, ldsa, blockA, B, ldb,
                                        formatB, scaleB, ldsb, blockB, beta, C, ldc, orderC, typeC, batch,
                                        strideA, strideB, strideScaleA, strideScaleB, strideC, p, k);
    return block_run(st, p, k, stream);
}

const char *gemm_f8_block_kernel_name(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A,
                                      int64_t lda, gemm_f8_format_t formatA, const float *scaleA,
                                      int64_t ldsa, int64_t blockA, const uint8_t *B, int64_t ldb,
                                      gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb,
                                      int64_t blockB, float beta, void *C, int64_t ldc,
                                      gemm_order_t orderC, gemm_output_t typeC, int64_t batch,
                                      int64_t strideA, int64_t strideB, int64_t strideScaleA,
                                      int64_t strideScaleB, int64_t strideC) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = dense_plan(M, N, K, alpha, A, lda, formatA, scaleA, ldsa, blockA, B, ldb,
                                        formatB, scaleB, ldsb, blockB, beta, C, ldc, orderC, typeC, batch,
                                        strideA, strideB, strideScaleA, strideScaleB, strideC, p, k);
    return block_name(st, k);
}

gemm_status_t gemm_experts_f8(int64_t experts, int64_t rows, int64_t N, int64_t K, const int32_t *offsets,
                              float alpha, const uint8_t *A, int64_t lda, gemm_f8_format_t formatA,
                              const float *scaleA, int64_t ldsa, const uint8_t *B, int64_t ldb,
                              gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb, int64_t blockB,
                              int64_t strideB, int64_t strideScaleB, float beta, void *C, int64_t ldc,
                              gemm_output_t typeC, hipStream_t stream) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = rows_plan(experts, rows, N, K, offsets, alpha, A, lda, formatA, scaleA, ldsa,
                                       B, ldb, formatB, scaleB, ldsb, blockB, strideB, strideScaleB, beta,
                                       C, ldc, typeC, p, k);
    return block_run(st, p, k, stream);
}

const char *gemm_experts_f8_kernel_name(int64_t experts, int64_t rows, int64_t N, int64_t K,
                                        const int32_t *offsets, float alpha, const uint8_t *A, int64_t lda,
                                        gemm_f8_format_t formatA, const float *scaleA, int64_t ldsa,
                                        const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                                        const float *scaleB, int64_t ldsb, int64_t blockB, int64_t strideB,
                                        int64_t strideScaleB, float beta, void *C, int64_t ldc,
                                        gemm_output_t typeC) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = rows_plan(experts, rows, N, K, offsets, alpha, A, lda, formatA, scaleA, ldsa,
                                       B, ldb, formatB, scaleB, ldsb, blockB, strideB, strideScaleB, beta,
                                       C, ldc, typeC, p, k);
    return block_name(st, k);
}

gemm_status_t gemm_experts_f8_wgrad(int64_t experts, int64_t M, int64_t N, int64_t rows,
                                    const int32_t *offsets, float alpha, const uint8_t *A, int64_t lda,
                                    gemm_f8_format_t formatA, const float *scaleA, int64_t ldsa,
                                    const uint8_t *B, int64_t ldb, gemm_f8_format_t formatB,
                                    const float *scaleB, int64_t ldsb, float beta, void *C, int64_t ldc,
                                    int64_t strideC, gemm_output_t typeC, hipStream_t stream) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = wgrad_plan(experts, M, N, rows, offsets, alpha, A, lda, formatA, scaleA, ldsa,
                                        B, ldb, formatB, scaleB, ldsb, beta, C, ldc, strideC, typeC, p, k);
    return block_run(st, p, k, stream);
}

const char *gemm_experts_f8_wgrad_kernel_name(int64_t experts, int64_t M, int64_t N, int64_t rows,
                                              const int32_t *offsets, float alpha, const uint8_t *A,
                                              int64_t lda, gemm_f8_format_t formatA, const float *scaleA,
                                              int64_t ldsa, const uint8_t *B, int64_t ldb,
                                              gemm_f8_format_t formatB, const float *scaleB, int64_t ldsb,
                                              float beta, void *C, int64_t ldc, int64_t strideC,
                                              gemm_output_t typeC) {
    BlockProblem p;
    BlockKernel k;
    const gemm_status_t st = wgrad_plan(experts, M, N, rows, offsets, alpha, A, lda, formatA, scaleA, ldsa,
                                        B, ldb, formatB, scaleB, ldsb, beta, C, ldc, strideC, typeC, p, k);
    return block_name(st, k);
}

int64_t gemm_experts_rows(int64_t tokens, int64_t experts, int64_t top_k, int64_t align) {
    if (!route_sizes_ok(tokens, experts, top_k) || align < 1 || align > 65536) return 0;
    const int64_t slots = tokens * top_k;
    return slots + (experts < slots ? experts : slots) * (align - 1);
}

size_t gemm_experts_route_workspace_size(int64_t tokens, int64_t experts, int64_t top_k) {
    if (!route_sizes_ok(tokens, experts, top_k)) return 0;
    return route_workspace(tokens, experts);
}

gemm_status_t gemm_experts_route(int64_t tokens, int64_t experts, const void *logits, int64_t ldl,
                                 gemm_input_t in, const float *bias, const uint8_t *keep,
                                 gemm_score_t score, int64_t groups, int64_t top_groups,
                                 int64_t group_top, int64_t top_k, int renormalise, float scale,
                                 int32_t *ids, float *weights, int64_t align, int64_t rows,
                                 int32_t *offsets, int32_t *row_tokens, int32_t *places, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!input_ok(in) || (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID))
        return GEMM_ERR_INVALID_ARG;
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts || groups < 1 || ldl < experts || ldl > MOST)
        return GEMM_ERR_INVALID_ARG;
    if (tokens > INT32_MAX || experts > GEMM_ROUTE_MAX_EXPERTS || top_k > GEMM_ROUTE_MAX_TOP_K ||
        groups > GEMM_ROUTE_MAX_GROUPS)
        return GEMM_ERR_UNSUPPORTED;
    if (experts % groups != 0) return GEMM_ERR_INVALID_ARG;
    if (groups > 1 && (top_groups < 1 || top_groups > groups || (group_top != 1 && group_top != 2) ||
                       top_k > top_groups * (experts / groups)))
        return GEMM_ERR_INVALID_ARG;
    const bool layout = offsets != nullptr || row_tokens != nullptr || places != nullptr;
    const int esize = type_bytes(in);
    const int64_t slots = tokens * top_k;
    if (extent_over(tokens, ldl, experts)) return GEMM_ERR_INVALID_ARG;
    const Range rl = range_of(logits, tokens > 0 ? (tokens - 1) * ldl + experts : 0, 1, 0, esize);
    const Range rb = range_of(bias, bias != nullptr ? experts : 0, 1, 0, 4);
    const Range rk = range_of(keep, keep != nullptr ? tokens : 0, 1, 0, 1);
    if (tokens > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, esize) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4) ||
        misaligned(offsets, 4) || misaligned(row_tokens, 4) || misaligned(places, 4))
        return GEMM_ERR_INVALID_ARG;
    Range out[6] = {range_of(ids, slots, 1, 0, 4), range_of(weights, slots, 1, 0, 4)};
    int n = 2;
    if (layout) {
        if (align < 1 || align > 65536 || rows < gemm_experts_rows(tokens, experts, top_k, align) ||
            rows > INT32_MAX)
            return GEMM_ERR_INVALID_ARG;
        if (offsets == nullptr || (rows > 0 && row_tokens == nullptr) || (tokens > 0 && places == nullptr))
            return GEMM_ERR_INVALID_ARG;
        const size_t need = gemm_experts_route_workspace_size(tokens, experts, top_k);
        if (tokens > 0 && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 16)))
            return GEMM_ERR_INVALID_ARG;
        out[n++] = range_of(offsets, experts + 1, 1, 0, 4);
        out[n++] = range_of(row_tokens, rows, 1, 0, 4);
        out[n++] = range_of(places, slots, 1, 0, 4);
        out[n++] = range_of(workspace, tokens > 0 ? static_cast<int64_t>(need) : 0, 1, 0, 1);
    }
    for (int i = 0; i < n; ++i) {
        if (overlap(out[i], rl) || overlap(out[i], rb) || overlap(out[i], rk)) return GEMM_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GEMM_ERR_INVALID_ARG;
    }
    if (tokens == 0 && !layout) return GEMM_OK;
    RouteArgs a{tokens, static_cast<int>(experts), logits, ldl, static_cast<int>(in), bias, keep,
                score == GEMM_SCORE_SIGMOID, static_cast<int>(groups), static_cast<int>(top_groups),
                static_cast<int>(group_top), static_cast<int>(top_k), renormalise != 0, scale, ids, weights,
                static_cast<int>(align), rows, offsets, row_tokens, places,
                layout ? workspace : nullptr};
    return status_of(launch_route(a, stream));
}

gemm_status_t gemm_experts_route_backward(int64_t tokens, int64_t experts, const void *logits, int64_t ldl,
                                          gemm_input_t in, gemm_score_t score, int64_t top_k,
                                          int renormalise, float scale, const int32_t *ids,
                                          const float *d_weights, void *d_logits, int64_t ldd,
                                          hipStream_t stream) {
    if (!input_ok(in) || (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID))
        return GEMM_ERR_INVALID_ARG;
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts || ldl < experts || ldd < experts ||
        ldl > MOST || ldd > MOST)
        return GEMM_ERR_INVALID_ARG;
    if (tokens > INT32_MAX || experts > GEMM_ROUTE_MAX_EXPERTS || top_k > GEMM_ROUTE_MAX_TOP_K)
        return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0) return GEMM_OK;
    const int esize = type_bytes(in);
    if (logits == nullptr || ids == nullptr || d_weights == nullptr || d_logits == nullptr ||
        misaligned(logits, esize) || misaligned(d_logits, esize) || misaligned(ids, 4) ||
        misaligned(d_weights, 4))
        return GEMM_ERR_INVALID_ARG;
    if (extent_over(tokens, ldl, experts) || extent_over(tokens, ldd, experts)) return GEMM_ERR_INVALID_ARG;
    const Range rd = range_of(d_logits, (tokens - 1) * ldd + experts, 1, 0, esize);
    if (overlap(rd, range_of(logits, (tokens - 1) * ldl + experts, 1, 0, esize)) ||
        overlap(rd, range_of(ids, tokens * top_k, 1, 0, 4)) ||
        overlap(rd, range_of(d_weights, tokens * top_k, 1, 0, 4)))
        return GEMM_ERR_INVALID_ARG;
    RouteBackwardArgs a{tokens, static_cast<int>(experts), logits, ldl, static_cast<int>(in),
                        score == GEMM_SCORE_SIGMOID, static_cast<int>(top_k), renormalise != 0, scale, ids,
                        d_weights, d_logits, ldd};
    return status_of(launch_route_backward(a, stream));
}

}  // extern "C"
