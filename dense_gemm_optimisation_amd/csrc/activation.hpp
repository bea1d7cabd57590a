// Activations of the layers' kernels and their slopes, in fp32.
//
// GELU(x) = x * Phi(x), Phi the standard normal distribution function:
//   Phi(-u) = exp(-u^2 / 2) * q(u), u >= 0, and Phi(u) = 1 - Phi(-u), with
//   q(u) = erfcx(u / sqrt 2) / 2 as t times a polynomial of degree eight in
//   t = 1 / (1 + 0.28 u), fitted to the least largest relative error on
//   u >= 0 by reweighted least squares: 1.7e-7, 5e-7 as evaluated in fp32.  The tail
//   keeps its relative precision, which a slope needs where Phi(x) and
//   x * phi(x) nearly cancel.
// SiLU(x) = x / (1 + exp(-x)).  ReLU(x) = max(x, 0), its slope at 0 is 0.  A NaN
// stays one in all of them and in their slopes.  An infinity takes the limit: a
// factor that has reached 0 times it is 0 (a Z kept in fp16 is infinite from
// 65520 on, and its slope is 1).
#pragma once

#include <hip/hip_runtime.h>

namespace libgemm {
namespace act {

constexpr int NONE = 0, RELU = 1, GELU = 2, SILU = 3;

#if defined(__HIPCC__)
// min(|x|, the largest number): a factor without the infinities that a factor of
// 0 would turn into NaN.  (A NaN's other factor is one too.)
__device__ inline float finite(float x) { return __builtin_amdgcn_fmed3f(fabsf(x), 0.0f, __FLT_MAX__); }

// q(|x|) and e <- exp(-x^2 / 2): Phi(-|x|) is their product.
__device__ inline float normal_tail(float x, float &e) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.28f * fabsf(x));
    float q = 0.0247200172f;
    q = __builtin_fmaf(q, t, -0.0935932765f);
    q = __builtin_fmaf(q, t, 0.0924283286f);
    q = __builtin_fmaf(q, t, -0.00644932837f);
    q = __builtin_fmaf(q, t, 0.0727750677f);
    q = __builtin_fmaf(q, t, 0.0836307803f);
    q = __builtin_fmaf(q, t, 0.103084666f);
    q = __builtin_fmaf(q, t, 0.111699803f);
    q = __builtin_fmaf(q, t, 0.111703858f);
    e = __expf(-0.5f * x * x);
    return q * t;
}

// GELU(x) = max(x, 0) - |x| Phi(-|x|).
__device__ inline float value(int a, float x) {
    if (a == RELU) return x <= 0.0f ? 0.0f : x;
    if (a == GELU) {
        float e;
        const float q = normal_tail(x, e);
        return __builtin_fmaf(-finite(x), q * e, fmaxf(x, 0.0f));
    }
    if (a == SILU) {
        const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-x));
        return __builtin_amdgcn_fmed3f(x, -__FLT_MAX__, __builtin_inff()) * p;
    }
    return x;
}

// Of GELU and SiLU.  GELU'(-u) = exp(-u^2 / 2) (q(u) - u / sqrt(2 pi)), and
// GELU'(u) = 1 - GELU'(-u).
__device__ inline float slope(int a, float x) {
    if (a == GELU) {
        float e;
        const float q = normal_tail(x, e);
        const float s = e * __builtin_fmaf(finite(x), -0.398942280f, q);
        return x >= 0.0f ? 1.0f - s : s;
    }
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-x));
    return p * __builtin_fmaf(__builtin_amdgcn_fmed3f(x, -__FLT_MAX__, __FLT_MAX__), 1.0f - p, 1.0f);
}

// Over N values, the choice made once.
template <int N>
__device__ inline void apply(int a, float (&x)[N]) {
    if (a == NONE) return;
    if (a == RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = value(RELU, x[e]);
    } else if (a == GELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = value(GELU, x[e]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = value(SILU, x[e]);
    }
}
template <int N>
__device__ inline void times_slope(int a, const float (&z)[N], float (&x)[N]) {
    if (a == RELU) {
        // chosen, not multiplied: an infinite or NaN gradient of a value that was cut off is 0
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = z[e] > 0.0f ? x[e] : z[e] <= 0.0f ? 0.0f : z[e];
    } else if (a == GELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= slope(GELU, z[e]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= slope(SILU, z[e]);
    }
}
#endif

}  // namespace act
}  // namespace libgemm
