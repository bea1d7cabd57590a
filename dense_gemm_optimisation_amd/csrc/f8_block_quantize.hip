// Quantising to 8-bit floats with one fp32 scale per block: 1 x 128 or
// 128 x 128, along the columns, along the rows, or both from one reading.
//
//   s = max(max |x| / F, 2^-126),  code = nearest_even(x / s)
//
// Both kernels are bound by memory: X is read once, in 16-byte pieces, and
// each output is written once.
//
// Magnitudes are compared as the integers that their bits form, which orders
// them and puts infinity and NaN on top, so neither is lost; 16-bit types two
// at a time.  The quotient is x * (1/s) with one correction by its exact
// remainder: with a correctly rounded reciprocal that is the correctly
// rounded quotient (Markstein's theorem), in three instructions.  It needs a
// remainder that does not underflow: blocks whose scale is below 2^-60 divide.
#include "f8_block.hpp"

namespace libgemm {
namespace {

constexpr int TILE = 128;
constexpr uint32_t INF_BITS = 0x7f800000u;
constexpr uint32_t NAN_CODES = 0x7f7f7f7fu;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

constexpr int F32 = 0, BF16 = 1, F16 = 2;

// Eight consecutive values of a row as loaded.
template <int TYPE>
struct Eight {
    static constexpr int WORDS = TYPE == F32 ? 8 : 4;
    uint32_t w[WORDS];

    __device__ float value(int j) const {
        if (TYPE == F32) return __builtin_bit_cast(float, w[TYPE == F32 ? j : 0]);
        const uint32_t v = w[j / 2];
        if (TYPE == BF16) return __builtin_bit_cast(float, j % 2 ? v & 0xffff0000u : v << 16);
        return static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(j % 2 ? v >> 16 : v)));
    }
    // The values from element `at` of x on, `n` of them there (the rest 0);
    // whole: the row's eights are 16-byte aligned.
    __device__ void load(const void *x, int64_t at, int64_t n, bool whole) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
        if (whole && n >= 8) {
            const u32x4_t *p = reinterpret_cast<const u32x4_t *>(static_cast<const char *>(x) + at * (TYPE == F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const u32x4_t v = p[i / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i + k] = v[k];
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            if (TYPE == F32) w[TYPE == F32 ? j : 0] = static_cast<const uint32_t *>(x)[at + j];
            else w[j / 2] |= uint32_t(static_cast<const uint16_t *>(x)[at + j]) << (16 * (j % 2));
        }
    }
};

// The larger magnitudes, element by element; a word holds one magnitude of
// fp32 or two of a 16-bit type (their bits without the sign).
template <int TYPE>
__device__ inline uint32_t larger(uint32_t a, uint32_t b) {
    if (TYPE == F32) return a > b ? a : b;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
template <int TYPE>
__device__ inline uint32_t magnitude(uint32_t w) {
    return w & (TYPE == F32 ? 0x7fffffffu : 0x7fff7fffu);
}
// fp32 bits of a 16-bit magnitude (of fp32: itself).
template <int TYPE>
__device__ inline uint32_t widen(uint32_t m) {
    if (TYPE == F32) return m;
    if (TYPE == BF16) return m << 16;
    return __builtin_bit_cast(uint32_t, static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(m))));
}
// Both halves of a word (of fp32: the word).
template <int TYPE>
__device__ inline uint32_t fold(uint32_t m) {
    if (TYPE == F32) return m;
    const uint32_t a = m & 0xffffu, b = m >> 16;
    return a > b ? a : b;
}
// Over the 16 lanes of a row of the data-parallel moves, in all of them.
__device__ inline uint32_t over_16_lanes(uint32_t m) {
    auto step = [&](uint32_t o) { m = o > m ? o : m; };
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x121, 0xf, 0xf, true)));  // row_ror 1
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x122, 0xf, 0xf, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x124, 0xf, 0xf, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x128, 0xf, 0xf, true)));
    return m;
}

// A block's scale and what its quotients need; amax as fp32 bits.
struct Scale {
    float s, r;
    bool nan, tiny;
    __device__ Scale(uint32_t amax, bool e5m2) {
        s = __builtin_bit_cast(float, amax) / (e5m2 ? 57344.0f : 448.0f);
        s = s < 0x1p-126f ? 0x1p-126f : s;
        nan = amax >= INF_BITS;
        tiny = s < 0x1p-60f;
        r = 1.0f / s;
        if (nan) s = __builtin_nanf("");
    }
    __device__ float quotient(float x) const {
        const float q = x * r;
        // (the sign of a zero is x's)
        return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);
    }
};

// The codes of four quotients; their magnitude is at most the largest finite
// value but for the rounding of s, which rounds to that value.
__device__ inline uint32_t codes4(float a, float b, float c, float d, bool e5m2) {
    int w;
    if (e5m2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return uint32_t(w);
}

// The codes of eight values of one block.
__device__ inline u32x2_t codes8(const Scale &k, const float (&x)[8], bool e5m2) {
    float q[8];
    if (__ballot(k.tiny) == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = k.quotient(x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = x[j] / k.s;
    }
    u32x2_t w = {codes4(q[0], q[1], q[2], q[3], e5m2), codes4(q[4], q[5], q[6], q[7], e5m2)};
    if (k.nan) w = u32x2_t{NAN_CODES, NAN_CODES};
    return w;
}

__device__ inline void store8(uint8_t *q, u32x2_t w, int64_t n, bool whole) {
    if (whole && n >= 8) {
        *reinterpret_cast<u32x2_t *>(q) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = uint8_t(w[j / 4] >> (8 * (j % 4)));
}

__device__ inline bool aligned(const void *p, int64_t stride_bytes, int64_t batch_bytes, int to) {
    return ((reinterpret_cast<uintptr_t>(p) | uint64_t(stride_bytes) | uint64_t(batch_bytes)) & (to - 1)) == 0;
}

// The row of X behind row r of the result; false: zeros.
__device__ inline bool source(const QuantizeArgs &a, int64_t r, int64_t &src) {
    src = r;
    if (r >= a.rows) return false;
    if (a.index == nullptr) return true;
    src = a.index[r];
    return src >= 0 && src < a.x_rows;
}

// Along the columns, a scale per row: 16 lanes hold a block, eight values
// each; a workgroup 16*UNITS rows of one block of columns.
template <int TYPE, int UNITS>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeArgs a, int64_t row_groups, int64_t col_blocks) {
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    const int64_t id = blockIdx.x, ct = id % col_blocks, rest = id / col_blocks;
    const int64_t b = rest / row_groups, r0 = (rest - b * row_groups) * (16 * UNITS) + tr;
    const int64_t c0 = ct * TILE + 8 * tc;
    constexpr int ESIZE = TYPE == F32 ? 4 : 2;
    const bool whole = aligned(a.x, a.ldx * ESIZE, a.sx * ESIZE, 16);
    const bool whole_q = aligned(a.q, a.ldq, a.sq, 8);
    Eight<TYPE> x[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        int64_t src;
        const bool live = source(a, r0 + 16 * u, src);
        x[u].load(a.x, b * a.sx + src * a.ldx + c0, live ? a.cols - c0 : 0, whole);
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < Eight<TYPE>::WORDS; ++i) m = larger<TYPE>(m, magnitude<TYPE>(x[u].w[i]));
        const Scale k(widen<TYPE>(over_16_lanes(fold<TYPE>(m))), a.e5m2 != 0);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[u].value(j);
        const u32x2_t w = codes8(k, v, a.e5m2 != 0);
        const int64_t r = r0 + 16 * u;
        if (r >= a.rows) continue;
        if (tc == 0) a.s[b * a.ss + ct * a.lds + r] = k.s;
        store8(a.q + b * a.sq + r * a.ldq + c0, w, a.cols - c0, whole_q);
    }
}

// Any direction and block: one workgroup holds a 128 x 128 tile in registers,
// 8 x 8 values per thread: thread t has rows 8*(t / 16) .. +7 and columns
// 8*(t % 16) .. +7, so a row's block spans 16 neighbouring lanes and a
// column's four lanes of each wave.  Transposed codes go through LDS, 16-byte
// chunk c of column n at c ^ (n / 8) % 8, so that they leave in whole lines.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantizeArgs a, int64_t row_tiles, int64_t col_tiles) {
    constexpr int WORDS = Eight<TYPE>::WORDS;
    __shared__ __attribute__((aligned(16))) uint32_t col_max[4][16 * WORDS];  // by wave
    __shared__ __attribute__((aligned(16))) uint8_t turned[TILE * TILE];
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15, wave = threadIdx.x >> 6;
    const int64_t id = blockIdx.x, ct = id % col_tiles, rest = id / col_tiles;
    const int64_t b = rest / row_tiles, rt = rest - b * row_tiles;
    const int64_t r0 = rt * TILE + 8 * tr, c0 = ct * TILE + 8 * tc;
    const bool e5m2 = a.e5m2 != 0;
    constexpr int ESIZE = TYPE == F32 ? 4 : 2;
    const bool whole = aligned(a.x, a.ldx * ESIZE, a.sx * ESIZE, 16);
    Eight<TYPE> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int64_t src;
        const bool live = source(a, r0 + i, src);
        x[i].load(a.x, b * a.sx + src * a.ldx + c0, live ? a.cols - c0 : 0, whole);
    }
    uint32_t row[8], col[WORDS];
#pragma unroll
    for (int k = 0; k < WORDS; ++k) col[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            const uint32_t w = magnitude<TYPE>(x[i].w[k]);
            m = larger<TYPE>(m, w);
            col[k] = larger<TYPE>(col[k], w);
        }
        row[i] = fold<TYPE>(m);
    }
    if (a.block == 1 && a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = over_16_lanes(row[i]);
    }
    if (a.block == TILE || a.qt != nullptr) {
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            col[k] = larger<TYPE>(col[k], __shfl_xor(col[k], 16));
            col[k] = larger<TYPE>(col[k], __shfl_xor(col[k], 32));
        }
        if ((threadIdx.x & 63) < 16) {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) col_max[wave][tc * WORDS + k] = col[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            col[k] = col_max[0][tc * WORDS + k];
#pragma unroll
            for (int g = 1; g < 4; ++g) col[k] = larger<TYPE>(col[k], col_max[g][tc * WORDS + k]);
        }
    }
    if (a.block == TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) m = larger<TYPE>(m, col[k]);
        m = over_16_lanes(fold<TYPE>(m));
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = m;
    }
    if (a.q != nullptr) {
        const bool whole_q = aligned(a.q, a.ldq, a.sq, 8);
        if (a.block == TILE && threadIdx.x == 0)
            a.s[b * a.ss + ct * a.lds + rt] = Scale(widen<TYPE>(row[0]), e5m2).s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + i;
            const Scale k(widen<TYPE>(row[i]), e5m2);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[i].value(j);
            const u32x2_t w = codes8(k, v, e5m2);
            if (r >= a.rows) continue;
            if (a.block == 1 && tc == 0) a.s[b * a.ss + ct * a.lds + r] = k.s;
            store8(a.q + b * a.sq + r * a.ldq + c0, w, a.cols - c0, whole_q);
        }
    }
    if (a.qt == nullptr) return;
    if (a.block == TILE && threadIdx.x == 0)
        a.st[b * a.sst + rt * a.ldst + ct] = Scale(widen<TYPE>(row[0]), e5m2).s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t m = a.block == TILE ? row[0]
                           : TYPE == F32   ? col[TYPE == F32 ? j : 0]
                                           : (j % 2 ? col[j / 2] >> 16 : col[j / 2] & 0xffffu);
        const Scale k(widen<TYPE>(m), e5m2);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i].value(j);
        const u32x2_t w = codes8(k, v, e5m2);
        *reinterpret_cast<u32x2_t *>(turned + (8 * tc + j) * TILE + (((tr >> 1) ^ (tc & 7)) << 4) + 8 * (tr & 1)) = w;
        if (a.block == 1 && tr == 0 && c0 + j < a.cols) a.st[b * a.sst + rt * a.ldst + c0 + j] = k.s;
    }
    __syncthreads();
    const bool whole_t = aligned(a.qt, a.ldqt, a.sqt, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = i * 32 + int(threadIdx.x >> 3), c = threadIdx.x & 7;
        const int64_t out_c = ct * TILE + n, r = rt * TILE + 16 * c;
        if (out_c >= a.cols || r >= a.rows) continue;
        const u32x4_t w = *reinterpret_cast<const u32x4_t *>(turned + n * TILE + ((c ^ (n >> 3 & 7)) << 4));
        uint8_t *q = a.qt + b * a.sqt + out_c * a.ldqt + r;
        if (whole_t && r + 16 <= a.rows) {
            *reinterpret_cast<u32x4_t *>(q) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (r + e < a.rows) q[e] = uint8_t(w[e / 4] >> (8 * (e % 4)));
        }
    }
}

template <int TYPE>
hipError_t go(const QuantizeArgs &q, hipStream_t stream) {
    QuantizeArgs a = q;
    int64_t cols = (a.cols + TILE - 1) / TILE;
    if (a.qt == nullptr && a.block == 1) {
        // four rows per thread keep enough loads in flight; one while that leaves compute units idle
        const int units = ((a.rows + 63) / 64) * cols * a.batch >= 512 ? 4 : 1;
        int64_t rows = (a.rows + 16 * units - 1) / (16 * units);
        if (rows * cols * a.batch > 0x7fffffff) return hipErrorInvalidConfiguration;
        void *args[] = {&a, &rows, &cols};
        const void *kernel = units == 4 ? reinterpret_cast<const void *>(&quantize_rows_kernel<TYPE, 4>)
                                        : reinterpret_cast<const void *>(&quantize_rows_kernel<TYPE, 1>);
        return hipLaunchKernel(kernel, dim3(unsigned(rows * cols * a.batch)), dim3(256), args, 0, stream);
    }
    int64_t rows = (a.rows + TILE - 1) / TILE;
    if (rows * cols * a.batch > 0x7fffffff) return hipErrorInvalidConfiguration;
    void *args[] = {&a, &rows, &cols};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quantize_tile_kernel<TYPE>),
                           dim3(unsigned(rows * cols * a.batch)), dim3(256), args, 0, stream);
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t stream) {
    if (a.type == F32) return go<F32>(a, stream);
    return a.type == BF16 ? go<BF16>(a, stream) : go<F16>(a, stream);
}

}  // namespace libgemm
