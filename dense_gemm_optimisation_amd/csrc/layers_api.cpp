// C ABI of libgemm_layers.h: argument validation and dispatch.  Every check
// runs before any HIP call, so an invalid call has no effect.
#include "libgemm_layers.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "arg_checks.hpp"
#include "layers.hpp"

using namespace libgemm;

namespace {

static_assert(GEMM_LAYER_MAX_TOKENS == LAYER_MAX_TOKENS && GEMM_LAYER_MAX_EXPERTS == LAYER_MAX_EXPERTS &&
                  GEMM_LAYER_MAX_TOP_K == LAYER_MAX_TOP_K,
              "the header's limits are the kernels'");

gemm_status_t status_of(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP; }

bool misaligned(const void *p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool type_ok(int t) { return t >= 0 && t <= 2; }       // of gemm_input_t and gemm_output_t
bool half_ok(int t) { return t == 1 || t == 2; }       // bf16 or fp16
bool out_ok(int t, int in) { return t == 0 || t == in; }  // fp32 or the inputs' type
int type_bytes(int t) { return t == 0 ? 4 : 2; }
bool act_ok(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }

// Sizes far enough from the ends of int64 for every extent below to be computed.
constexpr int64_t MOST = int64_t(1) << 40;
bool any_over(std::initializer_list<int64_t> sizes) {
    for (int64_t s : sizes)
        if (s < 0 || s > MOST) return true;
    return false;
}
constexpr int64_t MOST_EXTENT = INT64_MAX / 8;

// A rows x cols matrix of esize bytes, contiguous along a row, `batch` of them
// `stride` elements apart: aligned, wide enough, within the address space.
bool matrix_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int esize, Range &r, int64_t batch = 1,
               int64_t stride = 0) {
    if (p == nullptr || misaligned(p, esize) || ld < cols || stride < 0) return false;
    if (too_big(rows, ld) || rows * ld > MOST_EXTENT) return false;
    const int64_t span = (rows - 1) * ld + cols;
    if (batch > 1 && (too_big(batch - 1, stride) || (batch - 1) * stride > MOST_EXTENT - span)) return false;
    r = range_of(p, span, batch, stride, esize);
    return true;
}
bool meets(Range a, std::initializer_list<Range> others) {
    for (const Range &o : others)
        if (overlap(a, o)) return true;
    return false;
}
Range bytes_at(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p == nullptr ? Range{0, 0} : Range{lo, lo + static_cast<uintptr_t>(bytes)};
}
// Where an output may be an input itself: element by element the same.
bool same_matrix(const void *a, int64_t lda, int ta, const void *b, int64_t ldb, int tb, int64_t rows) {
    return a == b && ta == tb && (lda == ldb || rows == 1);
}

// Columns that the launches of column sums take: less than 2^32 threads.
constexpr int64_t MOST_N = int64_t(1) << 28;
bool linear_sizes_ok(int64_t M, int64_t N, int64_t K) {
    return !any_over({M, N, K}) && !too_big(M, N) && M * N <= MOST_EXTENT / 64;
}

// Validates either direction and chooses the kernel.
gemm_status_t linear_plan(const LinearProblem &q, gemm_order_t orderB, LinearProblem &p, LinearKernel &k) {
    k = LinearKernel::None;
    p = q;
    if (!half_ok(p.in) || !out_ok(p.out, p.in) || !act_ok(p.act) || !valid_order(orderB)) return GEMM_ERR_INVALID_ARG;
    if (any_over({p.lda, p.ldb, p.ldc}) || !linear_sizes_ok(p.M, p.N, p.K)) return GEMM_ERR_INVALID_ARG;
    if (p.N > MOST_N) return GEMM_ERR_UNSUPPORTED;
    if (p.N == 0) return GEMM_OK;
    if (p.M == 0) return p.dbias != nullptr && misaligned(p.dbias, 4) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
    Range rc;
    if (!matrix_ok(p.C, p.M, p.N, p.ldc, type_bytes(p.out), rc)) return GEMM_ERR_INVALID_ARG;
    Range ra{0, 0}, rb{0, 0}, rbias{0, 0}, rr{0, 0}, rz{0, 0}, rd{0, 0};
    if (p.alpha == 0.0f || p.K == 0) p.K = 0, p.alpha = 0.0f;  // nothing, whatever alpha is
    if (p.K > 0) {
        if (!matrix_ok(p.A, p.M, p.K, p.lda, 2, ra)) return GEMM_ERR_INVALID_ARG;
        if (!(p.b_kmajor ? matrix_ok(p.B, p.N, p.K, p.ldb, 2, rb) : matrix_ok(p.B, p.K, p.N, p.ldb, 2, rb)))
            return GEMM_ERR_INVALID_ARG;
    }
    const bool has_z = p.backward ? p.act != GEMM_ACT_NONE : p.Z != nullptr;
    if (has_z && (any_over({p.ldz}) || !matrix_ok(p.Z, p.M, p.N, p.ldz, 2, rz))) return GEMM_ERR_INVALID_ARG;
    const Range rw = bytes_at(p.workspace, int64_t(p.workspace_bytes > uint64_t(MOST) ? MOST : p.workspace_bytes));
    if (p.workspace == nullptr ? p.workspace_bytes != 0 : misaligned(p.workspace, 16)) return GEMM_ERR_INVALID_ARG;
    if (p.backward) {
        if (meets(rc, {ra, rb, rw})) return GEMM_ERR_INVALID_ARG;
        if (has_z && overlap(rc, rz) && !same_matrix(p.C, p.ldc, p.out, p.Z, p.ldz, p.in, p.M)) return GEMM_ERR_INVALID_ARG;
        if (p.dbias != nullptr) {
            if (misaligned(p.dbias, 4) || p.workspace == nullptr ||
                p.workspace_bytes < linear_workspace(p.M, p.N, p.K))
                return GEMM_ERR_INVALID_ARG;
            rd = bytes_at(p.dbias, p.N * 4);
            if (meets(rd, {rc, ra, rb, rz, rw})) return GEMM_ERR_INVALID_ARG;
        }
        if (meets(rw, {ra, rb, rz})) return GEMM_ERR_INVALID_ARG;
    } else {
        if (p.bias != nullptr) {
            if (misaligned(p.bias, 2)) return GEMM_ERR_INVALID_ARG;
            rbias = bytes_at(p.bias, p.N * 2);
        }
        if (p.beta != 0.0f && (any_over({p.ldr}) || !matrix_ok(p.R, p.M, p.N, p.ldr, type_bytes(p.out), rr)))
            return GEMM_ERR_INVALID_ARG;
        if (meets(rc, {ra, rb, rbias, rz, rw}) || meets(rz, {ra, rb, rbias, rr, rw}) || meets(rw, {ra, rb, rbias, rr}))
            return GEMM_ERR_INVALID_ARG;
        if (overlap(rc, rr) && !same_matrix(p.C, p.ldc, p.out, p.R, p.ldr, p.out, p.M)) return GEMM_ERR_INVALID_ARG;
    }
    k = linear_choose(p);
    return GEMM_OK;
}

LinearProblem forward_problem(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *B,
                              int64_t ldb, gemm_order_t orderB, gemm_input_t in, const void *bias,
                              gemm_activation_t act, float beta, const void *R, int64_t ldr, void *C, int64_t ldc,
                              gemm_output_t typeC, void *Z, int64_t ldz, void *workspace, size_t workspace_bytes) {
    LinearProblem p{};
    p.M = M, p.N = N, p.K = K, p.alpha = alpha;
    p.A = A, p.lda = lda, p.B = B, p.ldb = ldb, p.b_kmajor = orderB == GEMM_COL_MAJOR, p.in = int(in);
    p.backward = false, p.act = int(act), p.bias = bias, p.beta = beta, p.R = R, p.ldr = ldr;
    p.C = C, p.ldc = ldc, p.out = int(typeC), p.Z = Z, p.ldz = ldz;
    p.workspace = workspace, p.workspace_bytes = workspace_bytes;
    return p;
}

LinearProblem backward_problem(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *B,
                               int64_t ldb, gemm_order_t orderB, gemm_input_t in, const void *Z, int64_t ldz,
                               gemm_activation_t act, void *D, int64_t ldd, gemm_output_t typeD, float beta,
                               float *dbias, void *workspace, size_t workspace_bytes) {
    LinearProblem p{};
    p.M = M, p.N = N, p.K = K, p.alpha = alpha;
    p.A = A, p.lda = lda, p.B = B, p.ldb = ldb, p.b_kmajor = orderB == GEMM_COL_MAJOR, p.in = int(in);
    p.backward = true, p.act = int(act), p.C = D, p.ldc = ldd, p.out = int(typeD);
    p.Z = const_cast<void *>(Z), p.ldz = ldz, p.dbias = dbias, p.beta_bias = beta;
    p.workspace = workspace, p.workspace_bytes = workspace_bytes;
    return p;
}

bool layer_sizes_ok(int64_t tokens, int64_t experts, int64_t top_k, int64_t D, int64_t H) {
    return !any_over({tokens, experts, top_k, D, H}) && experts >= 1 && top_k >= 1 && top_k <= experts;
}
bool layer_limits_ok(int64_t tokens, int64_t experts, int64_t top_k) {
    return tokens <= GEMM_LAYER_MAX_TOKENS && experts <= GEMM_LAYER_MAX_EXPERTS && top_k <= GEMM_LAYER_MAX_TOP_K;
}

// One of the two weights of a layer of experts: rows x K each.
bool weights_ok(const LayerWeights &w, int type, int64_t experts, int64_t rows, int64_t K, Range &r, Range &rs) {
    const int esize = type == GEMM_WEIGHTS_SAME ? 2 : 1, per = 16 / esize;
    if (any_over({w.ld}) || w.stride < 0 || w.ld % per != 0 || w.stride % per != 0 || misaligned(w.w, 16)) return false;
    if (!matrix_ok(w.w, rows, K, w.ld, esize, r, experts, w.stride)) return false;
    if (type == GEMM_WEIGHTS_SAME) return true;
    const int64_t blocks = ceil_div(rows, 128), kb = ceil_div(K, 128);
    if (any_over({w.lds}) || w.stride_scale < 0) return false;
    return matrix_ok(w.scale, kb, blocks, kb > 1 ? w.lds : blocks, 4, rs, experts, w.stride_scale);
}

bool ortho_sizes_ok(int64_t M, int64_t N, int64_t batch) {
    return !any_over({M, N, batch}) && !too_big(M, N) && M * N <= MOST_EXTENT / 64 &&
           !too_big(batch, M * N + 4096) && batch * (M * N + 4096) <= MOST_EXTENT / 64;
}

}  // namespace

extern "C" {

size_t gemm_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (!linear_sizes_ok(M, N, K) || M == 0 || N == 0) return 0;
    return linear_workspace(M, N, K);
}

gemm_status_t gemm_linear(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *B,
                          int64_t ldb, gemm_order_t orderB, gemm_input_t in, const void *bias, gemm_activation_t act,
                          float beta, const void *R, int64_t ldr, void *C, int64_t ldc, gemm_output_t typeC, void *Z,
                          int64_t ldz, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    LinearProblem p;
    LinearKernel k;
    const gemm_status_t st =
        linear_plan(forward_problem(M, N, K, alpha, A, lda, B, ldb, orderB, in, bias, act, beta, R, ldr, C, ldc, typeC,
                                    Z, ldz, workspace, workspace_bytes),
                    orderB, p, k);
    return st != GEMM_OK ? st : status_of(launch_linear(k, p, stream));
}

const char *gemm_linear_kernel_name(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                                    const void *B, int64_t ldb, gemm_order_t orderB, gemm_input_t in,
                                    const void *bias, gemm_activation_t act, float beta, const void *R, int64_t ldr,
                                    void *C, int64_t ldc, gemm_output_t typeC, void *Z, int64_t ldz, void *workspace,
                                    size_t workspace_bytes) {
    LinearProblem p;
    LinearKernel k;
    const gemm_status_t st =
        linear_plan(forward_problem(M, N, K, alpha, A, lda, B, ldb, orderB, in, bias, act, beta, R, ldr, C, ldc, typeC,
                                    Z, ldz, workspace, workspace_bytes),
                    orderB, p, k);
    return st != GEMM_OK ? nullptr : linear_kernel_name(k);
}

gemm_status_t gemm_linear_backward(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                                   const void *B, int64_t ldb, gemm_order_t orderB, gemm_input_t in, const void *Z,
                                   int64_t ldz, gemm_activation_t act, void *D, int64_t ldd, gemm_output_t typeD,
                                   float beta, float *dbias, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    LinearProblem p;
    LinearKernel k;
    const gemm_status_t st =
        linear_plan(backward_problem(M, N, K, alpha, A, lda, B, ldb, orderB, in, Z, ldz, act, D, ldd, typeD, beta,
                                     dbias, workspace, workspace_bytes),
                    orderB, p, k);
    return st != GEMM_OK ? st : status_of(launch_linear(k, p, stream));
}

const char *gemm_linear_backward_kernel_name(int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                                             const void *B, int64_t ldb, gemm_order_t orderB, gemm_input_t in,
                                             const void *Z, int64_t ldz, gemm_activation_t act, void *D, int64_t ldd,
                                             gemm_output_t typeD, float beta, float *dbias, void *workspace,
                                             size_t workspace_bytes) {
    LinearProblem p;
    LinearKernel k;
    const gemm_status_t st =
        linear_plan(backward_problem(M, N, K, alpha, A, lda, B, ldb, orderB, in, Z, ldz, act, D, ldd, typeD, beta,
                                     dbias, workspace, workspace_bytes),
                    orderB, p, k);
    return st != GEMM_OK ? nullptr : linear_kernel_name(k);
}

size_t gemm_activation_backward_workspace_size(int64_t M, int64_t N) {
    if (!linear_sizes_ok(M, N, 0) || M == 0 || N == 0) return 0;
    return activation_backward_workspace(M, N);
}

gemm_status_t gemm_activation_backward(int64_t M, int64_t N, const void *A, int64_t lda, gemm_input_t typeA,
                                       const void *Z, int64_t ldz, gemm_input_t typeZ, gemm_activation_t act, void *D,
                                       int64_t ldd, gemm_output_t typeD, float beta, float *dbias, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
    if (!type_ok(typeA) || !type_ok(typeZ) || !type_ok(typeD) || !act_ok(act)) return GEMM_ERR_INVALID_ARG;
    if (any_over({lda}) || !linear_sizes_ok(M, N, 0)) return GEMM_ERR_INVALID_ARG;
    if (D == nullptr && dbias == nullptr) return GEMM_ERR_INVALID_ARG;
    if (N > MOST_N) return GEMM_ERR_UNSUPPORTED;
    if (N == 0) return GEMM_OK;
    if (M == 0 && dbias == nullptr) return GEMM_OK;
    if (M == 0) return misaligned(dbias, 4) ? GEMM_ERR_INVALID_ARG : status_of(launch_no_sums(N, beta, dbias, stream));
    Range ra, rz{0, 0}, rd{0, 0}, rb{0, 0}, rw{0, 0};
    if (!matrix_ok(A, M, N, lda, type_bytes(typeA), ra)) return GEMM_ERR_INVALID_ARG;
    const bool reads_z = act != GEMM_ACT_NONE;
    if (reads_z && (any_over({ldz}) || !matrix_ok(Z, M, N, ldz, type_bytes(typeZ), rz))) return GEMM_ERR_INVALID_ARG;
    if (D != nullptr) {
        if (any_over({ldd}) || !matrix_ok(D, M, N, ldd, type_bytes(typeD), rd)) return GEMM_ERR_INVALID_ARG;
        if (overlap(rd, ra) && !same_matrix(D, ldd, typeD, A, lda, typeA, M)) return GEMM_ERR_INVALID_ARG;
        if (overlap(rd, rz) && !same_matrix(D, ldd, typeD, Z, ldz, typeZ, M)) return GEMM_ERR_INVALID_ARG;
    }
    if (dbias != nullptr) {
        if (misaligned(dbias, 4) || workspace == nullptr || misaligned(workspace, 16) ||
            workspace_bytes < activation_backward_workspace(M, N))
            return GEMM_ERR_INVALID_ARG;
        rb = bytes_at(dbias, N * 4);
        rw = bytes_at(workspace, int64_t(activation_backward_workspace(M, N)));
        if (meets(rb, {ra, rz, rd, rw}) || meets(rw, {ra, rz, rd})) return GEMM_ERR_INVALID_ARG;
    }
    ActivationBackward p{M, N, A, lda, int(typeA), Z, ldz, int(typeZ), int(act), D, ldd, int(typeD), beta, dbias, workspace};
    return status_of(launch_activation_backward(p, stream));
}

size_t gemm_experts_layer_workspace_size(int64_t tokens, int64_t experts, int64_t top_k, int64_t D, int64_t H) {
    if (!layer_sizes_ok(tokens, experts, top_k, D, H) || !layer_limits_ok(tokens, experts, top_k)) return 0;
    if (tokens == 0 || D == 0) return 0;
    return experts_layer_workspace(tokens, experts, top_k, D, H);
}

gemm_status_t gemm_experts_layer(int64_t tokens, int64_t experts, int64_t top_k, int64_t D, int64_t H, const void *X,
                                 int64_t ldx, gemm_input_t in, const int32_t *ids, const float *weights,
                                 gemm_weights_t type, const void *up, int64_t ld_up, int64_t stride_up,
                                 const float *scale_up, int64_t lds_up, int64_t stride_scale_up, const void *down,
                                 int64_t ld_down, int64_t stride_down, const float *scale_down, int64_t lds_down,
                                 int64_t stride_scale_down, gemm_activation_t act, float beta, void *Y, int64_t ldy,
                                 gemm_output_t typeY, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!half_ok(in) || !out_ok(typeY, in) || type < GEMM_WEIGHTS_SAME || type > GEMM_WEIGHTS_E5M2 || !act_ok(act) ||
        act == GEMM_ACT_NONE)
        return GEMM_ERR_INVALID_ARG;
    if (!layer_sizes_ok(tokens, experts, top_k, D, H) || any_over({ldx, ldy})) return GEMM_ERR_INVALID_ARG;
    if (!layer_limits_ok(tokens, experts, top_k)) return GEMM_ERR_UNSUPPORTED;
    if (tokens == 0 || D == 0) return GEMM_OK;
    if (H == 0) return GEMM_ERR_INVALID_ARG;
    Range rx, ru, rsu{0, 0}, rdn, rsd{0, 0}, ry;
    if (ldx % 8 != 0 || misaligned(X, 16) || !matrix_ok(X, tokens, D, ldx, 2, rx)) return GEMM_ERR_INVALID_ARG;
    if (ids == nullptr || weights == nullptr || misaligned(ids, 4) || misaligned(weights, 4)) return GEMM_ERR_INVALID_ARG;
    const LayerWeights wu{up, ld_up, stride_up, scale_up, lds_up, stride_scale_up};
    const LayerWeights wd{down, ld_down, stride_down, scale_down, lds_down, stride_scale_down};
    if (!weights_ok(wu, type, experts, 2 * H, D, ru, rsu) || !weights_ok(wd, type, experts, D, H, rdn, rsd))
        return GEMM_ERR_INVALID_ARG;
    if (!matrix_ok(Y, tokens, D, ldy, type_bytes(typeY), ry)) return GEMM_ERR_INVALID_ARG;
    const size_t need = experts_layer_workspace(tokens, experts, top_k, D, H);
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
    const Range rw = bytes_at(workspace, int64_t(need)), ri = bytes_at(ids, tokens * top_k * 4),
                rg = bytes_at(weights, tokens * top_k * 4);
    if (meets(ry, {rx, ru, rsu, rdn, rsd, rw, ri, rg}) || meets(rw, {rx, ru, rsu, rdn, rsd, ri, rg}))
        return GEMM_ERR_INVALID_ARG;
    // offsets inside a workgroup's rows are 32-bit
    if (ldx > (1 << 23) || ld_up > (1 << 25) || ld_down > (1 << 25) || H > (1 << 17)) return GEMM_ERR_UNSUPPORTED;
    ExpertsLayer p{tokens, experts, top_k, D, H, X, ldx, int(in), ids, weights, int(type), wu, wd, int(act), beta,
                   Y, ldy, int(typeY), workspace};
    return status_of(launch_experts_layer(p, stream));
}

size_t gemm_orthogonalize_workspace_size(int64_t M, int64_t N, int64_t batch) {
    if (!ortho_sizes_ok(M, N, batch) || M == 0 || N == 0 || batch == 0) return 0;
    return orthogonalize_workspace(M, N, batch);
}

gemm_status_t gemm_orthogonalize(int64_t M, int64_t N, const void *G, int64_t ldg, gemm_input_t in, int64_t steps,
                                 const float *coefficients, float eps, float alpha, float beta, void *O, int64_t ldo,
                                 gemm_output_t typeO, int64_t batch, int64_t strideG, int64_t strideO, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!type_ok(in) || !type_ok(typeO) || !(eps >= 0.0f) || std::isinf(eps) || steps < 1) return GEMM_ERR_INVALID_ARG;
    if (!ortho_sizes_ok(M, N, batch) || any_over({ldg, ldo})) return GEMM_ERR_INVALID_ARG;
    if (steps > GEMM_ORTHOGONALIZE_MAX_STEPS) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0 || batch == 0) return GEMM_OK;
    Range rg, ro;
    if (!matrix_ok(G, M, N, ldg, type_bytes(in), rg, batch, strideG) ||
        !matrix_ok(O, M, N, ldo, type_bytes(typeO), ro, batch, strideO))
        return GEMM_ERR_INVALID_ARG;
    if (batch > 1 && strideO < (M - 1) * ldo + N) return GEMM_ERR_INVALID_ARG;
    const size_t need = orthogonalize_workspace(M, N, batch);
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
    const Range rw = bytes_at(workspace, int64_t(need));
    if (meets(ro, {rg, rw}) || overlap(rw, rg)) return GEMM_ERR_INVALID_ARG;
    // a launch has less than 2^32 threads, 256 of them for each block of 64 x 64
    if (M > (1 << 20) || N > (1 << 20) || ceil_div(M, 64) * ceil_div(N, 64) >= (1 << 24)) return GEMM_ERR_UNSUPPORTED;
    Orthogonalize p{M, N, G, ldg, int(in), int(steps), coefficients, eps, alpha, beta, O, ldo, int(typeO),
                    batch, batch > 1 ? strideG : 0, batch > 1 ? strideO : 0, workspace};
    return status_of(launch_orthogonalize(p, stream));
}

const char *gemm_orthogonalize_kernel_name(int64_t M, int64_t N, int64_t batch) {
    if (!ortho_sizes_ok(M, N, batch)) return nullptr;
    return orthogonalize_kernel_name(M, N, batch);
}

}  // extern "C"
