// Quantising to 8-bit floats with one fp32 scale per block: 1 x 128 or
// 128 x 128, along the columns, along the rows, or both from one reading.
//
//   s = max(max |x| / F, 2^-126),  code = nearest_even(x / s)
//
// Both kernels are bound by memory: X is read once, in 16-byte pieces, and
// each output is written once.  8192 x 4096 of bf16 to codes in both
// directions takes 27 us, 4.9 TB/s; a copy of as many bytes 26.
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
    // The values from element `at` of x on; 16-byte aligned.
    __device__ void load(const void *x, int64_t at) {
        const u32x4_t *p = reinterpret_cast<const u32x4_t *>(static_cast<const char *>(x) + at * (TYPE == F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const u32x4_t v = p[i / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[i + k] = v[k];
        }
    }
    // n of them there (the rest 0); whole: 16-byte aligned.
    __device__ void load(const void *x, int64_t at, int64_t n, bool whole) {
        clear();
        if (whole && n >= 8) {
            load(x, at);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            if (TYPE == F32) w[TYPE == F32 ? j : 0] = static_cast<const uint32_t *>(x)[at + j];
            else w[j / 2] |= uint32_t(static_cast<const uint16_t *>(x)[at + j]) << (16 * (j % 2));
        }
    }
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
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

// A block's scale and its reciprocal; amax as fp32 bits.
struct Scale {
    float s, r;
    __device__ Scale(uint32_t amax, bool e5m2) {
        s = __builtin_bit_cast(float, amax) / (e5m2 ? 57344.0f : 448.0f);
        s = s < 0x1p-126f ? 0x1p-126f : s;
        r = 1.0f / s;
        if (amax >= INF_BITS) s = __builtin_nanf("");
    }
};
// Whether the blocks behind the magnitudes need more than quotient():
// NaN or infinity among them, or a scale so small that a remainder underflows.
__device__ inline bool is_special(uint32_t amax, float s) { return amax >= INF_BITS || (amax != 0 && s < 0x1p-60f); }

// x / s for r = 1/s.  (The remainder's sign is chosen so that -0 stays -0.)
__device__ inline float quotient(float x, float s, float r) {
    const float q = x * r;
    return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
}

// v of one lane for all of its 16.
template <int LANE>
__device__ inline float of_lane(float v) {  // row_newbcast
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + LANE, 0xf, 0xf, true));
}

// The scales of N blocks, block i's magnitude in m[i] of all 16 lanes: lane
// i % N makes that of block i, for two divisions per lane take as long as the
// quotients of eight values.  mine: this lane's.
template <int N>  // a power of two
struct Scales {
    float s[N], r[N], mine;
    bool special;  // of any block in the wave
    __device__ Scales(const uint32_t (&m)[N], int lane16, bool e5m2) {
        uint32_t amax = m[0];
#pragma unroll
        for (int i = 1; i < N; ++i) {
            const uint32_t next = m[i];
            amax = (lane16 & (N - 1)) == i ? next : amax;
        }
        const Scale k(amax, e5m2);
        mine = k.s;
        special = __ballot(is_special(amax, k.s)) != 0;
        spread<0>(k);
    }
    template <int I>
    __device__ void spread(const Scale &k) {
        if constexpr (I < N) {
            s[I] = of_lane<I>(k.s);
            r[I] = of_lane<I>(k.r);
            spread<I + 1>(k);
        }
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

// The codes of eight values of one block; special as above.
__device__ inline u32x2_t codes8(float s, float r, bool special, const float (&x)[8], bool e5m2) {
    float q[8];
    if (!special) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = quotient(x[j], s, r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = x[j] / s;
    }
    u32x2_t w = {codes4(q[0], q[1], q[2], q[3], e5m2), codes4(q[4], q[5], q[6], q[7], e5m2)};
    if (special && s != s) w = u32x2_t{NAN_CODES, NAN_CODES};
    return w;
}

template <bool STREAM, typename T>
__device__ inline void store(uint8_t *q, T w) {
    if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<T *>(q));
    else *reinterpret_cast<T *>(q) = w;
}

template <bool STREAM>
__device__ inline void store8(uint8_t *q, u32x2_t w, int64_t n, bool whole) {
    if (whole && n >= 8) {
        store<STREAM>(q, w);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = uint8_t(w[j / 4] >> (8 * (j % 4)));
}

__device__ inline bool aligned(const void *p, int64_t stride_bytes, int64_t batch_bytes, int to) {
    return ((reinterpret_cast<uintptr_t>(p) | uint64_t(stride_bytes) | uint64_t(batch_bytes)) & (to - 1)) == 0;
}

// Columns c0..c0+7 of rows r0 + i*STEP of the result before quantising; rows
// and columns past its end, and rows that the index leaves out, are zeros.
// Where rows are whole aligned eights, a lane that has nothing to read reads
// the first row or columns and forgets them, so that no branch parts the loads.
template <int TYPE, int N, int STEP>
__device__ inline void load_rows(Eight<TYPE> (&x)[N], const QuantizeArgs &a, int64_t b, int64_t r0, int64_t c0) {
    constexpr int ESIZE = TYPE == F32 ? 4 : 2;
    const bool whole = aligned(a.x, a.ldx * ESIZE, a.sx * ESIZE, 16);
    const char *base = static_cast<const char *>(a.x) + b * a.sx * ESIZE;
    int64_t at[N];
    bool live[N];
    if (a.index == nullptr) {
        const int64_t first = (r0 < a.rows ? r0 : 0) * a.ldx;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            live[i] = r0 + i * STEP < a.rows;
            at[i] = first + (live[i] ? i * STEP * a.ldx : 0);
        }
    } else {
        int32_t src[N];
#pragma unroll
        for (int i = 0; i < N; ++i) src[i] = a.index[r0 + i * STEP < a.rows ? r0 + i * STEP : a.rows - 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            live[i] = r0 + i * STEP < a.rows && src[i] >= 0 && src[i] < a.x_rows;
            at[i] = live[i] ? src[i] * a.ldx : 0;
        }
    }
    if (whole && a.cols % 8 == 0 && (a.index == nullptr || a.x_rows > 0)) {
        const int64_t c = c0 < a.cols ? c0 : 0;
        bool gaps = c0 >= a.cols;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i].load(base, at[i] + c);
            gaps |= !live[i];
        }
        if (__ballot(gaps) != 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c0 >= a.cols || !live[i]) x[i].clear();
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i].load(base, at[i] + c0, live[i] ? a.cols - c0 : 0, whole);
    }
}

// Along the columns, a scale per row: 16 lanes hold a block, eight values
// each; a workgroup 16*UNITS rows of one block of columns.
template <int TYPE, int UNITS, bool STREAM>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeArgs a, uint32_t row_groups, uint32_t col_blocks) {
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    const uint32_t rest = blockIdx.x / col_blocks, ct = blockIdx.x - rest * col_blocks, b = rest / row_groups;
    const int64_t r0 = int64_t(rest - b * row_groups) * (16 * UNITS) + tr;
    const int64_t c0 = int64_t(ct) * TILE + 8 * tc;
    const bool whole_q = aligned(a.q, a.ldq, a.sq, 8);
    Eight<TYPE> x[UNITS];
    load_rows<TYPE, UNITS, 16>(x, a, b, r0, c0);
    uint32_t m[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < Eight<TYPE>::WORDS; ++i) w = larger<TYPE>(w, magnitude<TYPE>(x[u].w[i]));
        m[u] = widen<TYPE>(over_16_lanes(fold<TYPE>(w)));
    }
    const Scales<UNITS> k(m, tc, a.e5m2 != 0);
    if (tc < UNITS && r0 + 16 * tc < a.rows) a.s[b * a.ss + ct * a.lds + r0 + 16 * tc] = k.mine;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[u].value(j);
        const u32x2_t w = codes8(k.s[u], k.r[u], k.special, v, a.e5m2 != 0);
        const int64_t r = r0 + 16 * u;
        if (r < a.rows) store8<STREAM>(a.q + b * a.sq + r * a.ldq + c0, w, a.cols - c0, whole_q);
    }
}

// Any direction and block: one workgroup holds a 128 x 128 tile in registers,
// 8 x 8 values per thread: thread t has rows 8*(t / 16) .. +7 and columns
// 8*(t % 16) .. +7, so a row's block spans 16 neighbouring lanes and a
// column's four lanes of each wave.  Transposed codes go through LDS, 16-byte
// chunk c of column n at c ^ (n / 8) % 8, so that they leave in whole lines.
template <int TYPE, bool STREAM>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantizeArgs a, uint32_t row_tiles, uint32_t col_tiles) {
    constexpr int WORDS = Eight<TYPE>::WORDS;
    __shared__ __attribute__((aligned(16))) uint32_t col_max[4][16 * WORDS];  // by wave
    __shared__ __attribute__((aligned(16))) uint8_t turned[TILE * TILE];
    __shared__ __attribute__((aligned(16))) float col_s[TILE], col_r[TILE];
    __shared__ int col_special[2];
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15, wave = threadIdx.x >> 6;
    const uint32_t rest = blockIdx.x / col_tiles;
    const int64_t ct = blockIdx.x - rest * col_tiles, b = rest / row_tiles, rt = rest % row_tiles;
    const int64_t r0 = rt * TILE + 8 * tr, c0 = ct * TILE + 8 * tc;
    const bool e5m2 = a.e5m2 != 0;
    Eight<TYPE> x[8];
    load_rows<TYPE, 8, 1>(x, a, b, r0, c0);
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
    }
    if (a.block == TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
#pragma unroll
            for (int g = 0; g < 4; ++g) m = larger<TYPE>(m, col_max[g][tc * WORDS + k]);
        }
        m = over_16_lanes(fold<TYPE>(m));
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = m;
    } else if (a.qt != nullptr && threadIdx.x < TILE) {  // a column's scale per thread
        const int n = threadIdx.x;
        uint32_t m = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint32_t w = TYPE == F32 ? col_max[g][n] : col_max[g][n / 2] >> (16 * (n % 2)) & 0xffffu;
            m = w > m ? w : m;
        }
        m = widen<TYPE>(m);
        const Scale k(m, e5m2);
        col_s[n] = k.s;
        col_r[n] = k.r;
        const bool special = __ballot(is_special(m, k.s)) != 0;
        if ((n & 63) == 0) col_special[n >> 6] = special;
        if (ct * TILE + n < a.cols) a.st[b * a.sst + rt * a.ldst + ct * TILE + n] = k.s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = widen<TYPE>(row[i]);
    const Scales<8> kr(row, tc, e5m2);
    if (a.q != nullptr) {
        const bool whole_q = aligned(a.q, a.ldq, a.sq, 8);
        uint8_t *q = a.q + b * a.sq + r0 * a.ldq + c0;
        if (a.block == TILE && threadIdx.x == 0) a.s[b * a.ss + ct * a.lds + rt] = kr.mine;
        if (a.block == 1 && tc < 8 && r0 + tc < a.rows) a.s[b * a.ss + ct * a.lds + r0 + tc] = kr.mine;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[i].value(j);
            const u32x2_t w = codes8(kr.s[i], kr.r[i], kr.special, v, e5m2);
            if (r0 + i < a.rows) store8<STREAM>(q + i * a.ldq, w, a.cols - c0, whole_q);
        }
    }
    if (a.qt == nullptr) return;
    if (a.block == TILE) {
        if (threadIdx.x == 0) a.st[b * a.sst + rt * a.ldst + ct] = kr.mine;
    } else {
        __syncthreads();  // the columns' scales are there
    }
    const bool special = a.block == TILE ? kr.special : (col_special[0] | col_special[1]) != 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i].value(j);
        const float s = a.block == TILE ? kr.s[0] : col_s[8 * tc + j], r = a.block == TILE ? kr.r[0] : col_r[8 * tc + j];
        const u32x2_t w = codes8(s, r, special, v, e5m2);
        *reinterpret_cast<u32x2_t *>(turned + (8 * tc + j) * TILE + (((tr >> 1) ^ (tc & 7)) << 4) + 8 * (tr & 1)) = w;
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
            store<STREAM>(q, w);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (r + e < a.rows) q[e] = uint8_t(w[e / 4] >> (8 * (e % 4)));
        }
    }
}

template <int TYPE, bool STREAM>
hipError_t go(const QuantizeArgs &q, hipStream_t stream) {
    QuantizeArgs a = q;
    const int64_t cols = (a.cols + TILE - 1) / TILE;
    // Along the columns alone four rows per thread keep enough loads in
    // flight; one while that leaves compute units idle.
    const bool by_rows = a.qt == nullptr && a.block == 1;
    const int units = ((a.rows + 63) / 64) * cols * a.batch >= 512 ? 4 : 1;
    const int64_t height = by_rows ? 16 * units : TILE, rows = (a.rows + height - 1) / height;
    if (launch_over(double(rows) * cols * a.batch, 256)) return hipErrorInvalidConfiguration;
    uint32_t grid_rows = uint32_t(rows), grid_cols = uint32_t(cols);
    void *args[] = {&a, &grid_rows, &grid_cols};
    const void *kernel = !by_rows    ? reinterpret_cast<const void *>(&quantize_tile_kernel<TYPE, STREAM>)
                         : units > 1 ? reinterpret_cast<const void *>(&quantize_rows_kernel<TYPE, 4, STREAM>)
                                     : reinterpret_cast<const void *>(&quantize_rows_kernel<TYPE, 1, false>);
    return hipLaunchKernel(kernel, dim3(unsigned(rows * cols * a.batch)), dim3(256), args, 0, stream);
}

template <int TYPE>
hipError_t go(const QuantizeArgs &a, hipStream_t stream) {
    // Codes that the second-level caches (32 MB) cannot hold are stored past
    // them: 8192 x 4096 both ways 33 -> 27 us; where the product that reads
    // the codes finds them there, that would cost it 1 us (2048 x 4096).
    const double codes = double(a.rows) * a.cols * a.batch * ((a.q != nullptr) + (a.qt != nullptr));
    return codes > 32 << 20 ? go<TYPE, true>(a, stream) : go<TYPE, false>(a, stream);
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t stream) {
    if (a.type == F32) return go<F32>(a, stream);
    return a.type == BF16 ? go<BF16>(a, stream) : go<F16>(a, stream);
}

}  // namespace libgemm
