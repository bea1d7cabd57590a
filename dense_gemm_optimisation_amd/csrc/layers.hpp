// The layers' problems as the host layer hands them to the kernels, and their
// launchers.  Every argument has been validated.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

namespace libgemm {

// Lets a kernel have up to `bytes` of dynamic LDS, which beyond 64 KiB it has to
// be allowed, on the device of `stream`; the attribute is set on the current
// device, which need not be that one and stays what it was.
inline hipError_t allow_lds(const void *kernel, int bytes, hipStream_t stream) {
    int device = 0, current = 0;
    hipError_t e = hipStreamGetDevice(stream, &device);
    if (e == hipSuccess) e = hipGetDevice(&current);
    if (e == hipSuccess && device != current) e = hipSetDevice(device);
    if (e != hipSuccess) return e;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    const hipError_t back = device != current ? hipSetDevice(current) : hipSuccess;
    return e != hipSuccess ? e : back;
}

// Types: 0 fp32, 1 bf16, 2 fp16 (gemm_input_t and gemm_output_t alike).
struct LinearProblem {
    int64_t M, N, K;  // K = 0: nothing is multiplied
    float alpha;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    bool b_kmajor;
    int in;
    bool backward;
    int act;
    // forward: bias, beta * R and the stored Z; backward: Z is read
    const void *bias;
    float beta;
    const void *R;
    int64_t ldr;
    void *C;
    int64_t ldc;
    int out;
    void *Z;
    int64_t ldz;
    // backward: column sums
    float *dbias;
    float beta_bias;
    void *workspace;
    size_t workspace_bytes;
    bool packed;  // A and B are copies with rows of whole chunks, filled with zeros
};
enum class LinearKernel { None, Few16, Tile256, Rounds, Tile128, Split, Any, AnySplit, Packed };
const char *linear_kernel_name(LinearKernel k);
LinearKernel linear_choose(const LinearProblem &p);
size_t linear_workspace(int64_t M, int64_t N, int64_t K);
// dbias <- beta * dbias: the sums over no rows.
hipError_t launch_no_sums(int64_t N, float beta, float *dbias, hipStream_t stream);
hipError_t launch_linear(LinearKernel k, const LinearProblem &p, hipStream_t stream);

struct ActivationBackward {
    int64_t M, N;
    const void *A;
    int64_t lda;
    int type_a;
    const void *Z;
    int64_t ldz;
    int type_z;
    int act;
    void *D;
    int64_t ldd;
    int type_d;
    float beta;
    float *dbias;
    void *workspace;
};
size_t activation_backward_workspace(int64_t M, int64_t N);
hipError_t launch_activation_backward(const ActivationBackward &p, hipStream_t stream);

constexpr int LAYER_MAX_TOKENS = 64, LAYER_MAX_EXPERTS = 1024, LAYER_MAX_TOP_K = 32;
struct LayerWeights {
    const void *w;
    int64_t ld, stride;  // elements
    const float *scale;
    int64_t lds, stride_scale;
};
struct ExpertsLayer {
    int64_t tokens, experts, top_k, D, H;
    const void *X;
    int64_t ldx;
    int in;
    const int32_t *ids;
    const float *weights;
    int type;  // 0 X's, 1 E4M3, 2 E5M2
    LayerWeights up, down;
    int act;
    float beta;
    void *Y;
    int64_t ldy;
    int out;
    void *workspace;
};
size_t experts_layer_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t D, int64_t H);
hipError_t launch_experts_layer(const ExpertsLayer &p, hipStream_t stream);

struct Orthogonalize {
    int64_t M, N;
    const void *G;
    int64_t ldg;
    int in;
    int steps;
    const float *coefficients;  // 3 * steps, or nullptr
    float eps, alpha, beta;
    void *O;
    int64_t ldo;
    int out;
    int64_t batch, strideG, strideO;
    void *workspace;
};
const char *orthogonalize_kernel_name(int64_t M, int64_t N, int64_t batch);
size_t orthogonalize_workspace(int64_t M, int64_t N, int64_t batch);
hipError_t launch_orthogonalize(const Orthogonalize &p, hipStream_t stream);

}  // namespace libgemm
