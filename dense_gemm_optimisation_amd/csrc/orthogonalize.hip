// Newton-Schulz steps that orthogonalise a matrix (gemm_orthogonalize):
//   A = X X^T,   B = b A + c A^2,   X <- a X + B X,
// X the matrix or its transpose with m <= n, scaled to Frobenius norm 1.
//
// The products run on the fp16 matrix instructions with fp32 sums.  What is kept
// between them and why it is enough:
//   X    two fp16 pieces, hi + lo, 22 bits: a X, whose error would grow with
//        every step in the directions of small singular values, takes both;
//        the products take hi;
//   A, B one fp16 each.
// fp16 holds three more bits than bf16 at the same rate.  Its range is no
// matter: G enters as G * 2^e with an exponent that puts its norm into
// [2^11, 2^12) (exactly, for a 16-bit G), and the rest of the norm is a factor
// of the first step's epilogues; X is kept times 2^12, A times 2^12, B times
// 2^8.  An X of a norm below 1/4 (G's far below eps) is kept times a larger power
// of two, chosen before each update from the norm that it starts from and the
// most that the step's coefficients make of it (next_scale): its digits would
// sink into fp16's subnormals, 2.4e-2 of X at 1e-8 of eps, all of them at 1e-12.
//
// What is rounded is what differs from the mean: with s the mean of A's
// eigenvalues (|X|^2 / m) and E = A - s I, the same polynomial of X X^T is
//   B' = (b + 2 c s) E + c E^2,   X <- (a + b s + c s^2) X + B' X,
// and E is small once the singular values are alike, where a X and B X nearly
// cancel.  It halves the error that E's and B's roundings leave (simulated in
// 64 bits: 128 x 128 1.6e-3 -> 7e-4 of the Frobenius norm, 512 x 512 1.3e-3 ->
// 6e-4).  s is the squares' sum that the step before left; it need not be exact, only the
// same everywhere.
//
// Kernels:
//   small_kernel    a matrix whose pieces fit into one workgroup's LDS and
//                   registers: all steps in one launch, X's master in fp32 registers;
//   norm_kernel, input_kernel, then three product_kernels per step: A and B
//                   are symmetric, so only tiles on and above the diagonal
//                   are computed, and stored twice.  All matrices of the
//                   workspace have rows of a multiple of 8 elements, their
//                   filling zero, so every product runs on direct loads.
#include <math.h>

#include "layers.hpp"
#include "tile16.hpp"

namespace libgemm {
namespace {

using namespace tile16;

constexpr float X_SCALE = 4096.0f;  // 2^12, of X and of A; B's is 2^8
constexpr int PARTS = 256;          // partial sums of squares per matrix

struct OrthoArgs {
    int64_t m, n, ldx, lda;  // m <= n; ldx = n and lda = m rounded up to 8
    int64_t batch;
    uint16_t *x, *next, *lo;  // X's first piece, the next step's, the second piece: m x ldx
    uint16_t *gram, *poly;    // A and B: m x lda
    const float *factor;      // of each matrix: what x and lo are to be multiplied by for 2^12 X
    float *next_factor;       // the same of the next step's, written with A
    const float *norm;        // of each matrix: X's in the first step, else nullptr
    float *shift;             // of each matrix: s of this step
    float *squares;           // of each matrix and tile of the last update: the sum of X's squares
    int64_t tiles_x;          // those tiles
    float a, b, c;
    // the last step's output
    bool last, turned;  // turned: X is G's transpose
    float alpha, beta;
    void *O;
    int64_t ldo, strideO;
    int out;
    int64_t tiles_m, tiles_n;  // of the launch's product; upper: on and above the diagonal
};

// ---------------------------------------------------------------- norm and input
struct InputArgs {
    int64_t M, N, ldg, strideG;
    const void *G;
    int in;
    float eps;
    double *parts;                 // [batch][PARTS]
    float *factor, *shift, *norm;  // [batch]
    uint16_t *x, *lo;
    int64_t ldx, m;
    int64_t blocks, across;  // of 64 x 64, per matrix and across it
};

__device__ inline float value_of(const InputArgs &p, int64_t at) {
    if (p.in == 0) return static_cast<const float *>(p.G)[at];
    const uint16_t v = static_cast<const uint16_t *>(p.G)[at];
    return p.in == 1 ? decode<BF16>(v) : decode<F16>(v);
}

template <int THREADS>
__device__ inline double block_sum(double s, double *scratch) {
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) s += scratch[w];
    return s;
}

// N values of G from element `at` on (fewer than N are there at a row's end).
template <int N>
__device__ inline void values_of(const InputArgs &p, int64_t at, int64_t there, float (&v)[N]) {
    typedef float wide_f __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint16_t wide_h __attribute__((ext_vector_type(N), aligned(2)));
    if (there >= N && p.in == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const wide_f w = *reinterpret_cast<const wide_f *>(static_cast<const float *>(p.G) + at + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i + e] = w[e];
        }
    } else if (there >= N) {
        const wide_h w = *reinterpret_cast<const wide_h *>(static_cast<const uint16_t *>(p.G) + at);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = p.in == 1 ? decode<BF16>(w[e]) : decode<F16>(w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = e < there ? value_of(p, at + e) : 0.0f;
    }
}

// Squares in 64 bits: fp32's would leave its range.  Eight values at a time, eight
// such pieces per lane on their way together (4096 x 4096 in bf16: of four
// rows, 256 lanes, 28 us; so 17 to 19).
constexpr int NORM_THREADS = 512, NORM_PIECES = 8;
__global__ __launch_bounds__(NORM_THREADS) void norm_kernel(InputArgs p) {
    __shared__ double scratch[NORM_THREADS / 64];
    const int64_t batch = blockIdx.x / PARTS, part = blockIdx.x % PARTS, base = batch * p.strideG;
    const uint32_t per_row = uint32_t((p.N + 7) / 8);
    const int64_t pieces = p.M * per_row;
    double s = 0.0;
    for (int64_t i0 = part * NORM_THREADS; i0 < pieces; i0 += int64_t(NORM_PIECES) * PARTS * NORM_THREADS) {
        float v[NORM_PIECES][8];
#pragma unroll
        for (int i = 0; i < NORM_PIECES; ++i) {
            const int64_t at = i0 + int64_t(i) * PARTS * NORM_THREADS + threadIdx.x;
            const int64_t r = at / per_row, c = (at - r * per_row) * 8;
            values_of<8>(p, base + r * p.ldg + c, at < pieces ? p.N - c : 0, v[i]);
        }
#pragma unroll
        for (int i = 0; i < NORM_PIECES; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fma(double(v[i][e]), double(v[i][e]), s);
    }
    s = block_sum<NORM_THREADS>(s, scratch);
    if (threadIdx.x == 0) p.parts[batch * PARTS + part] = s;
}

// 64 x 64 elements of G into X's pieces, turned where M > N.
__global__ __launch_bounds__(256) void input_kernel(InputArgs p) {
    __shared__ double scratch[4];
    __shared__ float tile[64][65];
    const int64_t batch = blockIdx.x / p.blocks;
    const int64_t block = blockIdx.x % p.blocks, down = block / p.across, along = block % p.across;
    const double norm = sqrt(block_sum<256>(p.parts[batch * PARTS + threadIdx.x], scratch));
    // norm * 2^e in [2^11, 2^12); the rest of 2^12 * G / max(norm, eps)
    const bool finite = norm < 1e300;
    const int e = finite && norm > 0.0 ? 11 - ilogb(norm) : 0;
    const double least = norm > p.eps ? norm : p.eps > 0.0f ? double(p.eps) : 1.0;
    const float factor = !finite ? NAN : norm > 0.0 ? float(ldexp(4096.0 / least, -e)) : 0.0f;
    if (block == 0 && threadIdx.x == 0) {
        p.factor[batch] = factor;
        p.shift[batch] = float((norm / least) * (norm / least) / p.m);
        p.norm[batch] = float(norm / least);
    }
    const bool turned = p.M > p.N;
    const int64_t r0 = down * 64, c0 = along * 64;
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6;
    auto put = [&](int64_t r, int64_t c, float v) {
        if (r >= p.m || c >= p.ldx) return;
        const int64_t at = (batch * p.m + r) * p.ldx + c;
        const uint32_t hi = encode<F16>(v);
        p.x[at] = uint16_t(hi);
        p.lo[at] = uint16_t(encode<F16>(v - decode<F16>(hi)));
    };
    for (int i = row; i < 64; i += 4) {
        const int64_t r = r0 + i, c = c0 + col;
        const float v = r < p.M && c < p.N ? ldexpf(value_of(p, batch * p.strideG + r * p.ldg + c), e) : 0.0f;
        if (turned) tile[i][col] = v;
        else put(r, c, v);
    }
    if (!turned) return;
    __syncthreads();
    for (int i = row; i < 64; i += 4) put(c0 + i, r0 + col, tile[col][i]);
}

// ---------------------------------------------------------------- products
enum class Step { Gram, Poly, Update };

// O[at] <- y + beta * O[at]
__device__ inline void put_output(const OrthoArgs &p, int64_t at, float y) {
    if (p.out == 0) {
        float *d = static_cast<float *>(p.O) + at;
        *d = p.beta != 0.0f ? __builtin_fmaf(p.beta, *d, y) : y;
    } else {
        uint16_t *d = static_cast<uint16_t *>(p.O) + at;
        if (p.beta != 0.0f) y = __builtin_fmaf(p.beta, p.out == 1 ? decode<BF16>(*d) : decode<F16>(*d), y);
        *d = uint16_t(p.out == 1 ? encode<BF16>(y) : encode<F16>(y));
    }
}

// The same of four in a row.
__device__ inline void put_output4(const OrthoArgs &p, int64_t at, const float (&y)[4]) {
    typedef float wide_f __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint16_t wide_h __attribute__((ext_vector_type(4), aligned(2)));
    if (p.out == 0) {
        wide_f *d = reinterpret_cast<wide_f *>(static_cast<float *>(p.O) + at);
        wide_f v = {y[0], y[1], y[2], y[3]};
        if (p.beta != 0.0f) {
            const wide_f old = *d;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(p.beta, old[e], v[e]);
        }
        *d = v;
    } else {
        wide_h *d = reinterpret_cast<wide_h *>(static_cast<uint16_t *>(p.O) + at);
        wide_h old = {0, 0, 0, 0}, w;
        if (p.beta != 0.0f) old = *d;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = y[e];
            if (p.beta != 0.0f) v = __builtin_fmaf(p.beta, p.out == 1 ? decode<BF16>(old[e]) : decode<F16>(old[e]), v);
            w[e] = uint16_t(p.out == 1 ? encode<BF16>(v) : encode<F16>(v));
        }
        *d = w;
    }
}

// 2^12 X over what the update of an X of this norm stores: 1 for a norm of 1/4 or
// more; below, the power of two with which no element of the next X, whose norm
// is at most |a| + |b| / 16 + |c| / 256 times this, passes 2^15.
__device__ inline float next_scale(const OrthoArgs &p, float norm) {
    const float most = norm * fmaxf(16.0f, fabsf(p.a) + fabsf(p.b) + fabsf(p.c));
    const int up = most > 0.0f && most < 4.0f ? 2 - ilogbf(most) : 0;
    return ldexpf(1.0f, -(up < 120 ? up : 120));
}

// Tile `id` of the upper triangle of T x T tiles, row by row (in bands of six
// rows, which share more panels on a die, 4096 x 4096 took the same time).
__device__ inline void upper_tile(int64_t id, int64_t T, int64_t &tm, int64_t &tn) {
    int64_t r = 0;
    while (id >= T - r) id -= T - r++;
    tm = r;
    tn = r + id;
}

// Eight values of A less its mean eigenvalue, or of B' from it.
template <Step STEP>
struct Symmetric {
    typedef Raw8 Data;
    const uint16_t *gram;
    uint16_t *out;
    int64_t ld;
    float times, own;  // of the product's sums; of the diagonal (A), of A (B')
    __device__ void load(Data &d, int64_t r, int64_t c, int count) const {
        if (STEP == Step::Poly) d.load(gram + r * ld + c, count);
    }
    __device__ void operator()(int64_t r, int64_t c, int count, float (&v)[8], const Data &d) const {
        if constexpr (STEP == Step::Gram) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = times * v[e] - (r == c + e ? own : 0.0f);
        } else {
            float g[8];
            d.values<F16>(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(times, v[e], own * g[e]);
        }
        store8<F16>(out + r * ld + c, count, v);
    }
};

// Eight values of the next X, or in the last step of O.
struct Updated {
    struct Data {
        Raw8 hi, lo;
    };
    const OrthoArgs &p;
    const uint16_t *x;
    uint16_t *lo, *next;
    int64_t o;
    float factor, own, square;  // factor: of what is stored, or in the last step of 2^12 X
    __device__ void load(Data &d, int64_t r, int64_t c, int count) const {
        d.hi.load(x + r * p.ldx + c, count);
        d.lo.load(lo + r * p.ldx + c, count);
    }
    __device__ void operator()(int64_t r, int64_t c, int count, float (&v)[8], const Data &d) {
        float h[8], l[8];
        d.hi.values<F16>(h);
        d.lo.values<F16>(l);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = factor * __builtin_fmaf(0x1p-8f, v[e], own * (h[e] + l[e]));
        if (!p.last) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                square += v[e] * v[e];
                l[e] = v[e] - decode<F16>(encode<F16>(v[e]));
            }
            store8<F16>(next + r * p.ldx + c, count, v);
            store8<F16>(lo + r * p.ldx + c, count, l);
            return;
        }
        const float s = p.alpha / X_SCALE;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < p.n) put_output(p, o + (p.turned ? (c + e) * p.ldo + r : r * p.ldo + c + e), s * v[e]);
    }
};

template <class Shape, Step STEP>
__global__ __launch_bounds__(Shape::THREADS, Shape::LDS_BYTES > 80 * 1024 ? 1 : 2) void product_kernel(OrthoArgs p) {
    __shared__ __attribute__((aligned(1024))) char smem[Shape::LDS_BYTES];
    LDS char *lds = (LDS char *)smem;
    constexpr bool SYMMETRIC = STEP != Step::Update;
    const int64_t id = xcd_remap(blockIdx.x, gridDim.x, 8), per = gridDim.x / p.batch;
    const int64_t batch = uniform(id / per);
    int64_t tm, tn;
    if (SYMMETRIC) {
        upper_tile(id - batch * per, p.tiles_m, tm, tn);
    } else {
        const TileCoord t = tile_of(TileGrid{p.tiles_m, p.tiles_n, 1, 8, 1}, id - batch * per);
        tm = t.tm;
        tn = t.tn;
    }
    const int64_t m0 = uniform(tm) * Shape::TM, n0 = uniform(tn) * Shape::TN;
    uint16_t *x = p.x + batch * p.m * p.ldx, *gram = p.gram + batch * p.m * p.lda, *poly = p.poly + batch * p.m * p.lda;
    const Operand16 xr{x, p.ldx, p.m}, xc{x, p.ldx, p.ldx}, ar{gram, p.lda, p.m}, br{poly, p.lda, p.m};
    const int64_t K = STEP == Step::Gram ? p.ldx : p.lda;
    const int64_t N = SYMMETRIC ? p.lda : p.ldx;
    // s: read, or added up (by every workgroup alike) from the last update's tiles
    __shared__ float sums[Shape::WAVES];
    float shift = 0.0f;
    const float f = p.factor[batch];
    const bool first_thread = tm == 0 && tn == 0 && threadIdx.x == 0;
    if (STEP != Step::Gram) {
        shift = p.shift[batch];
    } else if (p.norm != nullptr) {
        shift = p.shift[batch];
        if (first_thread) p.next_factor[batch] = next_scale(p, p.norm[batch]);
    } else {
        float q = 0.0f;
        for (int64_t i = threadIdx.x; i < p.tiles_x; i += Shape::THREADS) q += p.squares[batch * p.tiles_x + i];
        for (int d = 1; d < 64; d *= 2) q += __shfl_xor(q, d);
        if ((threadIdx.x & 63) == 0) sums[threadIdx.x / 64] = q;
        __syncthreads();
        for (int w = 0; w < Shape::WAVES; ++w) shift += sums[w];
        // what is stored has a norm that fp32's squares hold; f a power of two
        const float norm = f * (sqrtf(shift) / X_SCALE);
        shift = f * (f * (shift / (X_SCALE * X_SCALE * float(p.m))));
        if (first_thread) {
            p.shift[batch] = shift;
            p.next_factor[batch] = next_scale(p, norm);
        }
    }
    typename Shape::Acc acc;
    // B's filling is columns, X has no rows for them: K = m there
    const int64_t depth = STEP == Step::Update ? p.m : K;
    const int buf = Shape::run(STEP == Step::Gram ? xr : STEP == Step::Poly ? ar : br,
                               STEP == Step::Gram ? xr : STEP == Step::Poly ? ar : xc, depth, m0, n0, 0,
                               (depth + Shape::BK - 1) / Shape::BK, lds, acc);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t mw = m0 + Shape::wave_m(wave) * Shape::WTM, nw = n0 + Shape::wave_n(wave) * Shape::WTN;
    const bool live = mw < p.m && nw < N;
    if (SYMMETRIC && !live) return;
    LDS float *staging = Shape::staging(lds, buf, wave);
    if constexpr (SYMMETRIC) {
        typedef Symmetric<STEP> S;
        const float b = __builtin_fmaf(2.0f * p.c, shift, p.b);
        S put{gram, STEP == Step::Gram ? gram : poly, p.lda, STEP == Step::Gram ? f * f / X_SCALE : p.c * 0x1p-16f,
              STEP == Step::Gram ? X_SCALE * shift : b * 0x1p-4f};
        visit_tile(acc, p.m, N, mw, nw, lane, staging, put);
        // the same values on the other side of the diagonal
        if (n0 > m0) visit_tile_turned(acc, p.m, p.m, mw, nw, lane, staging, put);
    } else {
        const int64_t at = batch * p.m * p.ldx;
        // the quotient of both: f itself may be next to fp32's smallest values
        Updated put{p, x, p.lo + at, p.next + at, batch * p.strideO, p.last ? f : f / p.next_factor[batch],
                    __builtin_fmaf(shift, __builtin_fmaf(shift, p.c, p.b), p.a), 0.0f};
        if (live) visit_tile(acc, p.m, N, mw, nw, lane, staging, put);
        float square = put.square;
        if (p.last) return;
        for (int d = 1; d < 64; d *= 2) square += __shfl_xor(square, d);
        if (lane == 0) sums[wave] = square;
        __syncthreads();
        if (threadIdx.x != 0) return;
        for (int w = 1; w < Shape::WAVES; ++w) square += sums[w];
        p.squares[batch * per + tm * p.tiles_n + tn] = square;
    }
}

// ---------------------------------------------------------------- in one workgroup
// Blocks of 32 x 32: at most 4 x 4 of A, dealt to 16 waves, and 48 of X.
constexpr int SMALL_WAVES = 16, SMALL_SIDE = 128, SMALL_BLOCKS = 3;  // X's blocks per wave
constexpr int SMALL_LDS = 150 * 1024;                              // beside what is declared
struct SmallArgs {
    InputArgs in;
    OrthoArgs p;
    int steps;
    float coefficients[3 * 32];
    int pitch_x, pitch_a;  // bytes per row of X and of A, 16 more than a multiple of 64
    int blocks_m, blocks_n;
};

// Fragments of 32 rows for 16 k from k0: K-contiguous rows, and k rows read
// transposed.  A row is 16 bytes longer than a multiple of 64, so neighbouring
// rows start in different banks.
__device__ inline u32x4 frag_rows(const LDS char *base, int pitch, int row0, int k0, int lane) {
    return *reinterpret_cast<const LDS u32x4 *>(base + (row0 + (lane & 31)) * pitch + (k0 + 8 * (lane >> 5)) * 2);
}
__device__ inline u32x4 frag_columns(const LDS char *base, int pitch, int col0, int k0, int lane) {
    const int g = lane >> 5, h = (lane >> 4) & 1, ii = lane & 15;
    u32x4 out;
#pragma unroll
    for (int e2 = 0; e2 < 2; ++e2) {
        const LDS s16x4 *at = reinterpret_cast<const LDS s16x4 *>(
            base + (k0 + g * 8 + e2 * 4 + (ii >> 2)) * pitch + (col0 + h * 16 + 4 * (ii & 3)) * 2);
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<LDS s16x4 *>(at)));
        out[2 * e2] = v[0];
        out[2 * e2 + 1] = v[1];
    }
    return out;
}
__device__ inline void put4(LDS char *at, const float (&v)[4]) {
    u32x2 w;
    w[0] = encode<F16>(v[0]) | encode<F16>(v[1]) << 16;
    w[1] = encode<F16>(v[2]) | encode<F16>(v[3]) << 16;
    *reinterpret_cast<LDS u32x2 *>(at) = w;
}

// BLOCKS: of X per wave at most.  Bound by the latency of three dependent products a
// step (16 matrices of 128 x 128, five steps: 31 us; 40 with every block of A and B
// computed and G read twice).
template <int BLOCKS>
__global__ __launch_bounds__(SMALL_WAVES * 64) void small_kernel(SmallArgs a) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ double scratch[SMALL_WAVES];
    __shared__ float sums[SMALL_WAVES];
    const InputArgs &in = a.in;
    const OrthoArgs &p = a.p;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t batch = blockIdx.x;
    const int m = int(p.m), n = int(p.n), mp = a.blocks_m * 32, np = a.blocks_n * 32;
    LDS char *x = (LDS char *)smem, *gram = x + mp * a.pitch_x, *poly = gram + mp * a.pitch_a;
    // a lane's part of block i: row l % 32, columns 8q + 4 (l / 32) + 0..3
    const int r_in = lane & 31, c_in = 4 * (lane >> 5), blocks = a.blocks_m * a.blocks_n;
    f32x16 X[BLOCKS];
    auto store_x = [&](int i, int block) {
        LDS char *at = x + (block / a.blocks_n * 32 + r_in) * a.pitch_x + (block % a.blocks_n * 32 + c_in) * 2;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float v[4] = {X[i][4 * u], X[i][4 * u + 1], X[i][4 * u + 2], X[i][4 * u + 3]};
            put4(at + 16 * u, v);
        }
    };
    // G as it is, and its norm in 64 bits
    double q = 0.0;
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const int block = wave + i * SMALL_WAVES;
        const int r = block / a.blocks_n * 32 + r_in, c = block % a.blocks_n * 32 + c_in;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = c + 8 * u;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (block < blocks && r < m && col < n) {
                if (!p.turned) {
                    values_of<4>(in, batch * in.strideG + r * in.ldg + col, n - col, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < n) v[e] = value_of(in, batch * in.strideG + (col + e) * in.ldg + r);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) X[i][4 * u + e] = v[e];
        }
    }
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
        for (int u = 0; u < 16; ++u) q = __builtin_fma(double(X[i][u]), double(X[i][u]), q);
    for (int d = 1; d < 64; d *= 2) q += __shfl_xor(q, d);
    if (lane == 0) scratch[wave] = q;
    __syncthreads();
    q = 0.0;
    for (int w = 0; w < SMALL_WAVES; ++w) q += scratch[w];
    const double norm = sqrt(q), least = norm > in.eps ? norm : in.eps > 0.0f ? double(in.eps) : 1.0;
    const float factor = norm < 1e300 ? 1.0f : NAN;
    float shift = float((norm / least) * (norm / least) / m);
    // a 0 times NaN is NaN, but the filling's stays out of every sum
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const int block = wave + i * SMALL_WAVES;
        if (block >= blocks) continue;
        const int r = block / a.blocks_n * 32 + r_in, c = block % a.blocks_n * 32 + c_in;
#pragma unroll
        for (int u = 0; u < 16; ++u)
            X[i][u] = r < m && c + 8 * (u / 4) + u % 4 < n ? factor * float(double(X[i][u]) * (X_SCALE / least)) : 0.0f;
        store_x(i, block);
    }
    __syncthreads();
    // A and B: a block on or above the diagonal per wave, stored twice
    const bool has = wave < a.blocks_m * (a.blocks_m + 1) / 2;
    int bi = 0, bj = wave;
    while (has && bj >= a.blocks_m - bi) bj -= a.blocks_m - bi++;
    bj = 32 * (bi + bj), bi *= 32;
    // columns c_in + 8 u .. + 3 of its row r_in
    auto put_symmetric = [&](LDS char *to, int u, const float (&v)[4]) {
        put4(to + (bi + r_in) * a.pitch_a + (bj + c_in + 8 * u) * 2, v);
        if (bi == bj) return;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<LDS uint16_t *>(to + (bj + c_in + 8 * u + e) * a.pitch_a + (bi + r_in) * 2) = uint16_t(encode<F16>(v[e]));
    };
    for (int step = 0; step < a.steps; ++step) {
        const float ca = a.coefficients[3 * step], cb = a.coefficients[3 * step + 1], cc = a.coefficients[3 * step + 2];
        if (has) {
            f32x16 acc = {};
#pragma unroll 4
            for (int k = 0; k < np; k += 16)
                acc = mfma32<F16>(frag_rows(x, a.pitch_x, bj, k, lane), frag_rows(x, a.pitch_x, bi, k, lane), acc);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = acc[4 * u + e] / X_SCALE;
                    // the filling stays zero
                    if (bi + r_in == bj + c_in + 8 * u + e && bi + r_in < m) v[e] -= X_SCALE * shift;
                }
                put_symmetric(gram, u, v);
            }
        }
        __syncthreads();
        const float b = __builtin_fmaf(2.0f * cc, shift, cb);
        if (has) {
            f32x16 acc = {};
#pragma unroll 4
            for (int k = 0; k < mp; k += 16)
                acc = mfma32<F16>(frag_rows(gram, a.pitch_a, bj, k, lane), frag_rows(gram, a.pitch_a, bi, k, lane), acc);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = (bi + r_in) * a.pitch_a + (bj + c_in + 8 * u) * 2;
                const u32x2 g = *reinterpret_cast<const LDS u32x2 *>(gram + at);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __builtin_fmaf(cc * 0x1p-16f, acc[4 * u + e], b * 0x1p-4f * decode<F16>(g[e / 2] >> (16 * (e % 2)) & 0xffffu));
                put_symmetric(poly, u, v);
            }
        }
        __syncthreads();
        const float own = __builtin_fmaf(shift, __builtin_fmaf(shift, cc, cb), ca);
        float square = 0.0f;
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i) {
            const int block = wave + i * SMALL_WAVES;
            if (block >= blocks) continue;
            const int xi = block / a.blocks_n * 32, xj = block % a.blocks_n * 32;
            f32x16 acc = {};
#pragma unroll 4
            for (int k = 0; k < mp; k += 16)
                acc = mfma32<F16>(frag_columns(x, a.pitch_x, xj, k, lane), frag_rows(poly, a.pitch_a, xi, k, lane), acc);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                X[i][u] = __builtin_fmaf(0x1p-8f, acc[u], own * X[i][u]);
                square += X[i][u] * X[i][u];
            }
        }
        for (int d = 1; d < 64; d *= 2) square += __shfl_xor(square, d);
        if (lane == 0) sums[wave] = square;
        __syncthreads();  // X has been read by every wave
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
            if (wave + i * SMALL_WAVES < blocks) store_x(i, wave + i * SMALL_WAVES);
        shift = 0.0f;
        for (int w = 0; w < SMALL_WAVES; ++w) shift += sums[w];
        shift /= X_SCALE * X_SCALE * float(m);
        __syncthreads();
    }
    const float s = p.alpha / X_SCALE;
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const int block = wave + i * SMALL_WAVES;
        if (block >= blocks) continue;
        const int r = block / a.blocks_n * 32 + r_in, c = block % a.blocks_n * 32 + c_in;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = c + 8 * u;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = s * X[i][4 * u + e];
            if (r >= m) continue;
            if (!p.turned && col + 3 < n) {
                put_output4(p, batch * p.strideO + r * p.ldo + col, y);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < n) put_output(p, batch * p.strideO + (p.turned ? (col + e) * p.ldo + r : r * p.ldo + col + e), y[e]);
        }
    }
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_to(int64_t n, int64_t m) { return ceil_div(n, m) * m; }

struct Layout {
    int64_t m, n, ldx, lda;
    size_t parts, factor[2], norm, shift, squares, x, next, lo, gram, poly, bytes;
};
Layout layout_of(int64_t M, int64_t N, int64_t batch) {
    Layout l{};
    l.m = M < N ? M : N;
    l.n = M < N ? N : M;
    l.ldx = round_to(l.n, 8);
    l.lda = round_to(l.m, 8);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += size_t(round_to(bytes, 256));
        return here;
    };
    l.parts = take(batch * PARTS * 8);
    l.factor[0] = take(batch * 4);
    l.factor[1] = take(batch * 4);
    l.norm = take(batch * 4);
    l.shift = take(batch * 4);
    l.squares = take(batch * ceil_div(l.m, 128) * ceil_div(l.n, 128) * 4);
    l.x = take(batch * l.m * l.ldx * 2);
    l.next = take(batch * l.m * l.ldx * 2);
    l.lo = take(batch * l.m * l.ldx * 2);
    l.gram = take(batch * l.m * l.lda * 2);
    l.poly = take(batch * l.m * l.lda * 2);
    l.bytes = at;
    return l;
}

// What small_kernel needs of LDS; 0 where the matrix does not fit.
size_t small_lds(int64_t m, int64_t n) {
    const int64_t bm = ceil_div(m, 32), bn = ceil_div(n, 32);
    if (m > SMALL_SIDE || bm * bn > SMALL_BLOCKS * SMALL_WAVES) return 0;
    const int64_t bytes = bm * 32 * ((bn * 64 + 16) + 2 * (bm * 64 + 16));
    return bytes <= SMALL_LDS ? size_t(bytes) : 0;
}

template <int BLOCKS>
hipError_t launch_small(const SmallArgs &a, size_t lds, hipStream_t stream) {
    if (lds > 64 * 1024) {
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(&small_kernel<BLOCKS>), SMALL_LDS, stream);
        if (e != hipSuccess) return e;
    }
    small_kernel<BLOCKS><<<dim3(unsigned(a.p.batch)), dim3(SMALL_WAVES * 64), lds, stream>>>(a);
    return hipGetLastError();
}

// Tiles of 256, 192 (symmetric products) or 128, whichever takes the least time
// by whole rounds of workgroups: one of 256 or 192 per compute unit, two of 128.
// 4096 x 4096: A and B of 192 (253 tiles) 98 and 102 us, of 256 (136) 111 and 114,
// of 128 (528) 111 and 115; X of 256 (256 tiles) 146, of 128 160.
// What fits into one round of one 128 tile per unit takes a ring of four stages
// instead of two (1000 x 2049: A 26 us for 32, X 20 for 21); symmetric products
// that leave half the units idle then take 64 tiles (A 15 us for 26, B 11 for 18).
enum class Size { Large, Middle, Small, Few, Least };
Size size_of(int64_t m, int64_t n, int64_t batch, bool symmetric) {
    auto tiles = [&](int64_t side) {
        const int64_t r = ceil_div(m, side), c = ceil_div(n, side);
        return batch * (symmetric ? r * (r + 1) / 2 : r * c);
    };
    if (symmetric && tiles(128) <= 128) return Size::Least;
    if (tiles(128) <= 256) return Size::Few;
    const int64_t large = ceil_div(tiles(256), 256) * 64, small = ceil_div(tiles(128), 512) * 40;
    const int64_t middle = symmetric ? ceil_div(tiles(192), 256) * 42 : INT64_MAX;
    if (middle < large && middle < small) return Size::Middle;
    return large <= small ? Size::Large : Size::Small;
}
int64_t side_of(Size s) { return s == Size::Large ? 256 : s == Size::Middle ? 192 : s == Size::Least ? 64 : 128; }

template <class Shape, Step STEP>
hipError_t launch_shape(OrthoArgs &a, int64_t tiles, hipStream_t stream) {
    product_kernel<Shape, STEP><<<dim3(unsigned(tiles)), dim3(Shape::THREADS), 0, stream>>>(a);
    return hipGetLastError();
}

template <Step STEP>
hipError_t launch_product(OrthoArgs &a, hipStream_t stream) {
    constexpr bool SYMMETRIC = STEP != Step::Update;
    using Large = Tile<F16, 256, 256, 2, 4, true, SYMMETRIC, true>;
    using Middle = Tile<F16, 192, 192, 2, 2, true, true, true, 64, 3>;
    using Small = Tile<F16, 128, 128, 2, 2, true, SYMMETRIC, true>;
    using Few = Tile<F16, 128, 128, 2, 2, true, SYMMETRIC, true, 64, 4>;
    using Least = Tile<F16, 64, 64, 2, 2, true, true, true, 64, 4>;
    const int64_t cols = SYMMETRIC ? a.m : a.n;
    const Size size = size_of(a.m, cols, a.batch, SYMMETRIC);
    a.tiles_m = ceil_div(a.m, side_of(size));
    a.tiles_n = ceil_div(cols, side_of(size));
    if (!SYMMETRIC) a.tiles_x = a.tiles_m * a.tiles_n;
    const int64_t tiles = a.batch * (SYMMETRIC ? a.tiles_m * (a.tiles_m + 1) / 2 : a.tiles_m * a.tiles_n);
    if (size == Size::Large) return launch_shape<Large, STEP>(a, tiles, stream);
    if (size == Size::Small) return launch_shape<Small, STEP>(a, tiles, stream);
    if (size == Size::Few) return launch_shape<Few, STEP>(a, tiles, stream);
    if constexpr (SYMMETRIC)
        return size == Size::Middle ? launch_shape<Middle, STEP>(a, tiles, stream) : launch_shape<Least, STEP>(a, tiles, stream);
    return hipSuccess;
}

}  // namespace

// Matrices at a time, one batch after another in the same workspace: a launch has
// less than 2^32 threads, of 256 for 64 x 64 elements, of 512 for a part of a norm.
static int64_t most_batch(int64_t M, int64_t N) {
    const int64_t blocks = ceil_div(M, 64) * ceil_div(N + 7, 64), most = (int64_t(1) << 23) / blocks;
    return most < 1 ? 1 : most < 16384 ? most : 16384;
}

const char *orthogonalize_kernel_name(int64_t M, int64_t N, int64_t batch) {
    if (M == 0 || N == 0 || batch == 0) return "";
    const int64_t most = most_batch(M, N);
    if (batch > most) batch = most;
    if (small_lds(M < N ? M : N, M < N ? N : M) != 0) return "orthogonalize_small";
    switch (size_of(M < N ? M : N, M < N ? N : M, batch, false)) {
        case Size::Large: return "orthogonalize_mfma_256";
        case Size::Few: return "orthogonalize_mfma_128_few";
        default: return "orthogonalize_mfma_128";
    }
}

size_t orthogonalize_workspace(int64_t M, int64_t N, int64_t batch) {
    const int64_t most = most_batch(M, N);
    return layout_of(M, N, batch < most ? batch : most).bytes;
}

static hipError_t launch_batch(const Orthogonalize &p, hipStream_t stream) {
    const Layout l = layout_of(p.M, p.N, p.batch);
    char *w = static_cast<char *>(p.workspace);
    auto half = [&](size_t at) { return reinterpret_cast<uint16_t *>(w + at); };
    auto floats = [&](size_t at) { return reinterpret_cast<float *>(w + at); };
    float *factor[2] = {floats(l.factor[0]), floats(l.factor[1])};
    InputArgs in{p.M, p.N, p.ldg, p.strideG, p.G, p.in, p.eps, reinterpret_cast<double *>(w + l.parts), factor[0],
                 floats(l.shift), floats(l.norm), half(l.x), half(l.lo), l.ldx, l.m};
    const bool turned = p.M > p.N;
    OrthoArgs a{};
    a.m = l.m;
    a.n = l.n;
    a.ldx = l.ldx;
    a.lda = l.lda;
    a.batch = p.batch;
    a.shift = in.shift;
    a.squares = floats(l.squares);
    a.x = half(l.x);
    a.next = half(l.next);
    a.lo = half(l.lo);
    a.gram = half(l.gram);
    a.poly = half(l.poly);
    a.turned = turned;
    a.alpha = p.alpha;
    a.beta = p.beta;
    a.O = p.O;
    a.ldo = p.ldo;
    a.strideO = p.strideO;
    a.out = p.out;
    auto coefficient = [&](int s, int i) {
        constexpr float usual[3] = {3.4445f, -4.7750f, 2.0315f};
        return p.coefficients != nullptr ? p.coefficients[3 * s + i] : usual[i];
    };
    if (const size_t lds = small_lds(l.m, l.n)) {
        SmallArgs sm{in, a, p.steps, {}, 0, 0, int(ceil_div(l.m, 32)), int(ceil_div(l.n, 32))};
        for (int s = 0; s < 3 * p.steps; ++s) sm.coefficients[s] = coefficient(s / 3, s % 3);
        sm.pitch_x = sm.blocks_n * 64 + 16;
        sm.pitch_a = sm.blocks_m * 64 + 16;
        const int blocks = sm.blocks_m * sm.blocks_n;
        if (blocks <= SMALL_WAVES) return launch_small<1>(sm, lds, stream);
        if (blocks <= 2 * SMALL_WAVES) return launch_small<2>(sm, lds, stream);
        return launch_small<SMALL_BLOCKS>(sm, lds, stream);
    }
    // the tiles of G also cover the filling of X's rows
    const int64_t rows = ceil_div(turned ? l.ldx : p.M, 64), cols = ceil_div(turned ? p.N : l.ldx, 64);
    in.blocks = rows * cols;
    in.across = cols;
    norm_kernel<<<dim3(unsigned(PARTS * p.batch)), dim3(NORM_THREADS), 0, stream>>>(in);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    input_kernel<<<dim3(unsigned(in.blocks * p.batch)), dim3(256), 0, stream>>>(in);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    for (int s = 0; s < p.steps; ++s) {
        a.factor = factor[s % 2];
        a.next_factor = factor[(s + 1) % 2];
        a.norm = s == 0 ? in.norm : nullptr;
        a.last = s == p.steps - 1;
        a.a = coefficient(s, 0);
        a.b = coefficient(s, 1);
        a.c = coefficient(s, 2);
        e = launch_product<Step::Gram>(a, stream);
        if (e == hipSuccess) e = launch_product<Step::Poly>(a, stream);
        if (e == hipSuccess) e = launch_product<Step::Update>(a, stream);
        if (e != hipSuccess) return e;
        uint16_t *t = a.x;
        a.x = a.next;
        a.next = t;
    }
    return hipSuccess;
}

hipError_t launch_orthogonalize(const Orthogonalize &p, hipStream_t stream) {
    const int64_t most = most_batch(p.M, p.N);
    for (int64_t first = 0; first < p.batch; first += most) {
        Orthogonalize q = p;
        q.batch = p.batch - first < most ? p.batch - first : most;
        q.G = static_cast<const char *>(p.G) + first * p.strideG * (p.in == 0 ? 4 : 2);
        q.O = static_cast<char *>(p.O) + first * p.strideO * (p.out == 0 ? 4 : 2);
        const hipError_t e = launch_batch(q, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace libgemm
