// Quantising to 8-bit floats with one fp32 scale per block: 1 x 128 or
// 128 x 128, along the columns, along the rows, or both from one reading.
//
//   s = max(max |x| / F, 2^-126),  code = nearest_even(x / s)
//
// One workgroup holds a 128 x 128 tile of X in registers, 8 x 8 values per
// thread: thread t has rows 8*(t / 16) .. +7 and columns 8*(t % 16) .. +7, so
// a row's block spans 16 neighbouring lanes and a column's the 16 threads
// t % 16 apart.  Magnitudes are compared as the integers their bits form, which
// orders them and puts NaN above infinity, so neither is lost.
#include "f8_block.hpp"

namespace libgemm {
namespace {

constexpr int TILE = 128;
constexpr uint32_t INF_BITS = 0x7f800000u;

__device__ inline float load_x(const void *x, int64_t at, int type) {
    if (type == 0) return static_cast<const float *>(x)[at];
    const uint16_t b = static_cast<const uint16_t *>(x)[at];
    return type == 1 ? __builtin_bit_cast(float, uint32_t(b) << 16)
                     : static_cast<float>(__builtin_bit_cast(_Float16, b));
}

__device__ inline float scale_of(uint32_t amax, float largest) {
    if (amax >= INF_BITS) return __builtin_nanf("");
    const float s = __builtin_bit_cast(float, amax) / largest;
    return s < 0x1p-126f ? 0x1p-126f : s;
}

// The code of x / s; |x| / s is at most the largest finite value but for the
// rounding of s, which the clamp takes back.
__device__ inline uint32_t code_of(float x, float s, float largest, int e5m2) {
    float v = x / s;
    if (v != v) return 0x7fu;
    v = v > largest ? largest : v < -largest ? -largest : v;
    const int r = e5m2 ? __builtin_amdgcn_cvt_pk_bf8_f32(v, v, 0, false)
                       : __builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false);
    return uint32_t(r) & 0xffu;
}

__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a) {
    __shared__ uint32_t col_max[16][TILE];  // by row group
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    const int64_t b = blockIdx.z;
    const int64_t r0 = int64_t(blockIdx.y) * TILE + 8 * tr, c0 = int64_t(blockIdx.x) * TILE + 8 * tc;
    const float largest = a.e5m2 ? 57344.0f : 448.0f;
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int64_t src = r0 + i;
        bool live = src < a.rows;
        if (live && a.index != nullptr) {
            src = a.index[src];
            live = src >= 0 && src < a.x_rows;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[i][j] = live && c0 + j < a.cols ? load_x(a.x, b * a.sx + src * a.ldx + c0 + j, a.type) : 0.0f;
    }
    uint32_t row[8], col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = col[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = __builtin_bit_cast(uint32_t, x[i][j]) & 0x7fffffffu;
            row[i] = m > row[i] ? m : row[i];
            col[j] = m > col[j] ? m : col[j];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const uint32_t o = __shfl_xor(row[i], d);
            row[i] = o > row[i] ? o : row[i];
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) col_max[tr][8 * tc + j] = col[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        for (int g = 0; g < 16; ++g) {
            const uint32_t o = col_max[g][8 * tc + j];
            col[j] = o > col[j] ? o : col[j];
        }
    if (a.block == TILE) {
        // the whole tile's, from the columns' (each thread has eight of them)
        uint32_t all = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) all = col[j] > all ? col[j] : all;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const uint32_t o = __shfl_xor(all, d);
            all = o > all ? o : all;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = col[i] = all;
    }
    const int64_t rt = int64_t(blockIdx.y), ct = int64_t(blockIdx.x);
    if (a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + i;
            if (r >= a.rows) continue;
            const float s = scale_of(row[i], largest);
            if (tc == 0 && (a.block == 1 || (tr == 0 && i == 0)))
                a.s[b * a.ss + ct * a.lds + (a.block == 1 ? r : rt)] = s;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < a.cols)
                    a.q[b * a.sq + r * a.ldq + c0 + j] = uint8_t(code_of(x[i][j], s, largest, a.e5m2));
        }
    }
    if (a.qt != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + j;
            if (c >= a.cols) continue;
            const float s = scale_of(col[j], largest);
            if (tr == 0 && (a.block == 1 || (tc == 0 && j == 0)))
                a.st[b * a.sst + rt * a.ldst + (a.block == 1 ? c : ct)] = s;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < a.rows)
                    a.qt[b * a.sqt + c * a.ldqt + r0 + i] = uint8_t(code_of(x[i][j], s, largest, a.e5m2));
        }
    }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &q, hipStream_t stream) {
    QuantizeArgs a = q;
    const int64_t gx = (a.cols + TILE - 1) / TILE, gy = (a.rows + TILE - 1) / TILE;
    if (gx > 0x7fffffff || gy > 0xffff || a.batch > 0xffff) return hipErrorInvalidConfiguration;
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quantize_kernel),
                           dim3(unsigned(gx), unsigned(gy), unsigned(a.batch)), dim3(256), args, 0, stream);
}

}  // namespace libgemm
