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
// factor that has reached 0 is not multiplied by it (a Z kept in fp16 is
// infinite from 65520 on, and its slope is 1).
#pragma once

#include <hip/hip_runtime.h>

namespace libgemm {
namespace act {

constexpr int NONE = 0, RELU = 1, GELU = 2, SILU = 3;

#if defined(__HIPCC__)
// e <- exp(-x^2 / 2); Phi(x)
__device__ inline float normal_below(float x, float &e) {
    const float u = fabsf(x);
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.28f * u);
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
    const float tail = q * t * e;
    return x >= 0.0f ? 1.0f - tail : tail;
}

__device__ inline float value(int a, float x) {
    if (a == RELU) return x <= 0.0f ? 0.0f : x;
    if (a == GELU) {
        float e;
        const float below = normal_below(x, e);
        return below == 0.0f ? 0.0f : x * below;
    }
    if (a == SILU) {
        const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-x));
        return p == 0.0f ? 0.0f : x * p;
    }
    return x;
}

// Of GELU and SiLU.
__device__ inline float slope(int a, float x) {
    if (a == GELU) {
        float e;
        const float below = normal_below(x, e);
        return e == 0.0f ? below : __builtin_fmaf(x * 0.398942280f, e, below);
    }
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-x)), q = 1.0f - p;
    return p * q == 0.0f ? p : p * __builtin_fmaf(x, q, 1.0f);
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
