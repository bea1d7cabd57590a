// The product with bias, activation and residual in its epilogue
// (gemm_linear), the product with an activation's slope and column sums in
// its epilogue (gemm_linear_backward), and the latter without a product
// (gemm_activation_backward).
//
// Kernels, by the work there is (linear_choose):
//   tile 256 / 128   256 x 256 tiles of eight waves, 128 x 128 tiles of four,
//                    two workgroups per compute unit (tile16.hpp).  The epilogue reads and
//                    writes whole rows of 64 columns and costs what its bytes
//                    cost;
//   rounds           the 256 x 256 tiles where the last of several rounds is less
//                    than half full: its tiles are cut into slices of K;
//   split            the 128 x 128 tiles with K cut into slices, each slice's
//                    sums in the workspace, joined in order by finish_kernel,
//                    which also has the epilogue: few tiles, long K;
//   few              up to 16 rows against a K-contiguous B: 16 columns per
//                    workgroup, K dealt to eight waves, each with a ring of its
//                    own in LDS; bound by reading B;
//   any              the 128 x 128 tiles with panels through registers, for
//                    operands of any alignment; larger problems copy such
//                    operands into the workspace first (pack.hip).
// Column sums: each wave (or finish workgroup) leaves the sums over its rows
// in the workspace, and sums_kernel adds them in order: no atomics, the same
// result on every run.
#include "activation.hpp"
#include "gemm_problem.hpp"
#include "layers.hpp"
#include "tile16.hpp"

namespace libgemm {
namespace {

using namespace tile16;

struct LinearArgs {
    int64_t M, N, K;
    float alpha, beta, beta_bias;
    Operand16 a, b;
    const uint16_t *bias;
    const void *R;
    void *C;
    uint16_t *Z;
    int64_t ldr, ldc, ldz;
    int act;
    bool c_same;     // C (and R) have the inputs' type, else fp32
    TileGrid grid;   // batch: slices of K
    int64_t first, tiles;  // of the grid, those that a launch has
    float *sums;     // backward: column sums by rows of blocks, N each,
    float *dbias;    // or, where one block has all rows, the result itself
    float *partial;  // split: [slice][M][ldp]; the last tiles': [slice][tile][256][256]
    int64_t ldp;
    int slices;
};

// The values of one lane's eight columns, which stay the same while it goes
// down the rows.
template <class T, bool BACKWARD>
struct Finish {
    const LinearArgs &p;
    float column[8];  // forward: the bias; backward: the sums so far

    __device__ Finish(const LinearArgs &args, int64_t n) : p(args) {
#pragma unroll
        for (int e = 0; e < 8; ++e) column[e] = 0.0f;
        if (!BACKWARD && p.bias != nullptr && n < p.N)
            load8<T>(p.bias + n, p.N - n < 8 ? int(p.N - n) : 8, column);
    }
    // What row m's columns n .. n + count - 1 read: Z, or a 16-bit residual.
    typedef Raw8 Data;
    __device__ void load(Data &d, int64_t m, int64_t n, int count) const {
        if (BACKWARD && p.act != act::NONE) d.load(p.Z + m * p.ldz + n, count);
        if (!BACKWARD && p.beta != 0.0f && p.c_same) d.load(static_cast<const uint16_t *>(p.R) + m * p.ldr + n, count);
    }
    // x: the products' sums of those columns
    __device__ void operator()(int64_t m, int64_t n, int count, float (&x)[8], const Data &d) {
        if constexpr (BACKWARD) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= p.alpha;
            if (p.act != act::NONE) {
                float z[8];
                d.values<T>(z);
                act::times_slope(p.act, z, x);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) column[e] += x[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(p.alpha, x[e], column[e]);
            if (p.Z != nullptr) store8<T>(p.Z + m * p.ldz + n, count, x);
            act::apply(p.act, x);
            if (p.beta != 0.0f) {
                float r[8];
                if (p.c_same) d.values<T>(r);
                else load8f(static_cast<const float *>(p.R) + m * p.ldr + n, count, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(p.beta, r[e], x[e]);
            }
        }
        store8_as<T>(p.C, m * p.ldc + n, p.c_same, count, x);
    }
    // The lanes with this lane's columns (those a multiple of `lanes` apart)
    // add up; the first of them writes row `block` of the sums.
    __device__ void write_sums(int64_t block, int64_t n, int lanes, int lane) {
        if (!BACKWARD || p.sums == nullptr) return;
        for (int d = lanes; d < 64; d *= 2)
#pragma unroll
            for (int e = 0; e < 8; ++e) column[e] += __shfl_xor(column[e], d);
        if (lane < lanes && n < p.N) store_sums(block, n, p.N - n < 8 ? int(p.N - n) : 8, column);
    }
    __device__ void store_sums(int64_t block, int64_t n, int count, float (&v)[8]) const {
        if (p.dbias == nullptr) {
            store8f(p.sums + block * p.N + n, count, v);
            return;
        }
        if (p.beta_bias != 0.0f) {
            float old[8];
            load8f(p.dbias + n, count, old);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(p.beta_bias, old[e], v[e]);
        }
        store8f(p.dbias + n, count, v);
    }
};

// ---------------------------------------------------------------- tiles
// 4096 x 16384 x 4096 in bf16 with GELU and Z kept: 500 to 520 us, 1.07 PFLOP/s,
// where the loop alone takes 465 (loads, LDS reads and power together bound it:
// 454 without reading fragments, 374 without refills, 406 on zeros) and a library's
// plain product 401.  The rest is the rounds' epilogues: 268 MB stored, GELU.
template <class T, class Shape, bool BACKWARD>
__global__ __launch_bounds__(Shape::THREADS, Shape::THREADS == 512 ? 1 : 2) void tile_kernel(LinearArgs p) {
    __shared__ __attribute__((aligned(1024))) char smem[Shape::LDS_BYTES];
    LDS char *lds = (LDS char *)smem;
    const TileCoord t = tile_of(p.grid, p.first + xcd_remap(blockIdx.x, p.tiles, 8));
    const int64_t m0 = uniform(t.tm) * Shape::TM, n0 = uniform(t.tn) * Shape::TN;
    typename Shape::Acc acc;
    const int buf = Shape::run(p.a, p.b, p.K, m0, n0, 0, (p.K + Shape::BK - 1) / Shape::BK, lds, acc);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t mw = m0 + Shape::wave_m(wave) * Shape::WTM, nw = n0 + Shape::wave_n(wave) * Shape::WTN;
    if (mw >= p.M || nw >= p.N) return;
    constexpr int LANES = Shape::WTN / 8;
    const int64_t n = nw + (lane % LANES) * 8;
    Finish<T, BACKWARD> finish(p, n);
    visit_tile(acc, p.M, p.N, mw, nw, lane, Shape::staging(lds, buf, wave), finish);
    finish.write_sums(mw / Shape::WTM, n, LANES, lane);
}

// What a slice of K leaves in the workspace: its sums, element (m, n) at out[m * ld + n].
struct Partial {
    typedef Nothing Data;
    float *out;
    int64_t ld;
    __device__ void load(Data &, int64_t, int64_t, int) const {}
    __device__ void operator()(int64_t m, int64_t n, int count, const float (&x)[8], const Data &) const {
        store8f(out + m * ld + n, count, x);
    }
};

// One slice of K of a tile.
template <class Shape>
__global__ __launch_bounds__(Shape::THREADS, 2) void split_kernel(LinearArgs p) {
    __shared__ __attribute__((aligned(1024))) char smem[Shape::LDS_BYTES];
    LDS char *lds = (LDS char *)smem;
    const TileCoord t = tile_of(p.grid, blockIdx.x);
    const int64_t m0 = uniform(t.tm) * Shape::TM, n0 = uniform(t.tn) * Shape::TN, z = uniform(t.batch);
    const int64_t stages = (p.K + Shape::BK - 1) / Shape::BK;
    typename Shape::Acc acc;
    const int buf = Shape::run(p.a, p.b, p.K, m0, n0, stages * z / p.slices, stages * (z + 1) / p.slices, lds, acc);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t mw = m0 + Shape::wave_m(wave) * Shape::WTM, nw = n0 + Shape::wave_n(wave) * Shape::WTN;
    if (mw >= p.M || nw >= p.N) return;
    visit_tile(acc, p.M, p.N, mw, nw, lane, Shape::staging(lds, buf, wave), Partial{p.partial + z * p.M * p.ldp, p.ldp});
}

// One slice of K of one of the tiles from p.first on.
template <class Shape>
__global__ __launch_bounds__(Shape::THREADS, 1) void last_kernel(LinearArgs p) {
    __shared__ __attribute__((aligned(1024))) char smem[Shape::LDS_BYTES];
    LDS char *lds = (LDS char *)smem;
    const int64_t tile = blockIdx.x / p.slices, z = blockIdx.x % p.slices;
    const TileCoord t = tile_of(p.grid, p.first + tile);
    const int64_t m0 = uniform(t.tm) * Shape::TM, n0 = uniform(t.tn) * Shape::TN;
    const int64_t stages = (p.K + Shape::BK - 1) / Shape::BK;
    typename Shape::Acc acc;
    const int buf = Shape::run(p.a, p.b, p.K, m0, n0, stages * z / p.slices, stages * (z + 1) / p.slices, lds, acc);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t mw = m0 + Shape::wave_m(wave) * Shape::WTM, nw = n0 + Shape::wave_n(wave) * Shape::WTN;
    if (mw >= p.M || nw >= p.N) return;
    float *out = p.partial + (z * p.tiles + tile) * (Shape::TM * Shape::TN);
    visit_tile(acc, p.M, p.N, mw, nw, lane, Shape::staging(lds, buf, wave), Partial{out - (m0 * Shape::TN + n0), Shape::TN});
}

// The sums of a workgroup's waves over 64 columns, eight per lane, as row
// `block` of the sums; n0 is the first column.
template <int WAVES, class T, bool BACKWARD>
__device__ inline void join_sums(Finish<T, BACKWARD> &finish, float (&waves)[WAVES][64], int64_t block, int64_t n0) {
    if (!BACKWARD || finish.p.sums == nullptr) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = 8; d < 64; d *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) finish.column[e] += __shfl_xor(finish.column[e], d);
    if (lane < 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) waves[wave][lane * 8 + e] = finish.column[e];
    __syncthreads();
    const int64_t n = n0 + lane * 8;
    if (wave != 0 || lane >= 8 || n >= finish.p.N) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = waves[0][lane * 8 + e];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v[e] += waves[w][lane * 8 + e];
    }
    finish.store_sums(block, n, finish.p.N - n < 8 ? int(finish.p.N - n) : 8, v);
}

// Joins their slices: 64 columns of 128 rows per workgroup.
template <class T, class Shape, bool BACKWARD>
__global__ __launch_bounds__(256) void last_finish_kernel(LinearArgs p) {
    __shared__ float waves[4][64];
    const TileCoord t = tile_of(p.grid, p.first + blockIdx.z);
    const int64_t m0 = t.tm * Shape::TM + blockIdx.y * Shape::WTM, n0 = t.tn * Shape::TN;
    if (m0 >= p.M || n0 + blockIdx.x * 64 >= p.N) return;
    const int64_t n = n0 + blockIdx.x * 64 + (threadIdx.x % 8) * 8;
    const int count = p.N - n < 8 ? int(p.N - n) : 8;
    const float *base = p.partial + blockIdx.z * (Shape::TM * Shape::TN);
    Finish<T, BACKWARD> finish(p, n);
    // four rows of each lane at a time: their loads all go out first
    constexpr int ROWS = Shape::WTM / 32;
    const float *at = base + (blockIdx.y * Shape::WTM + threadIdx.x / 8) * Shape::TN + (n - n0);
    auto live = [&](int i) { return m0 + i * 32 + threadIdx.x / 8 < p.M && count > 0; };
    float x[ROWS][8], part[ROWS][8];
    Raw8 data[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (!live(i)) continue;
        finish.load(data[i], m0 + i * 32 + threadIdx.x / 8, n, count);
        load8f(at + i * 32 * Shape::TN, 8, x[i]);  // whole: the workspace's rows are
    }
    for (int s = 1; s < p.slices; ++s) {
        const float *next = at + s * p.tiles * (Shape::TM * Shape::TN);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (live(i)) load8f(next + i * 32 * Shape::TN, 8, part[i]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] += part[i][e];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (live(i)) finish(m0 + i * 32 + threadIdx.x / 8, n, count, x[i], data[i]);
    join_sums(finish, waves, m0 / Shape::WTM, n0 + blockIdx.x * 64);
}

// Joins the slices: 64 columns by FINISH_ROWS rows per workgroup of four waves, or
// by all rows per workgroup of eight.
constexpr int FINISH_ROWS = 32;
template <class T, bool BACKWARD, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void finish_kernel(LinearArgs p) {
    __shared__ float waves[WAVES][64];
    const int64_t n = int64_t(blockIdx.x) * 64 + (threadIdx.x % 8) * 8;
    const int count = p.N - n < 8 ? int(p.N - n) : 8;
    Finish<T, BACKWARD> finish(p, n);
    const int64_t end = WAVES == 4 && (int64_t(blockIdx.y) + 1) * FINISH_ROWS < p.M ? (int64_t(blockIdx.y) + 1) * FINISH_ROWS : p.M;
    if (count > 0)
        for (int64_t m = int64_t(blockIdx.y) * FINISH_ROWS + threadIdx.x / 8; m < end; m += WAVES * 8) {
            float x[8], part[8];
            const float *at = p.partial + m * p.ldp + n;
            Raw8 data;
            finish.load(data, m, n, count);
            load8f(at, 8, x);  // whole: the workspace's rows are
            for (int s = 1; s < p.slices; ++s) {
                load8f(at + s * p.M * p.ldp, 8, part);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] += part[e];
            }
            finish(m, n, count, x, data);
        }
    join_sums(finish, waves, blockIdx.y, int64_t(blockIdx.x) * 64);
}

// ---------------------------------------------------------------- few rows
template <class T>
__device__ inline f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c);
template <>
__device__ inline f32x4 mfma16<BF16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ inline f32x4 mfma16<F16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// At most ROWS (4, 8 or 16) rows by 16 columns, K dealt to eight waves in runs of 128.
// A wave keeps the next runs of both operands on their way into its own
// LDS: a direct load takes four rows of 256 bytes, while loads in the matrix
// instruction's own order would ask for one 16-byte piece of 16 rows after
// another and keep the address unit busy three times as long.  16-byte chunk
// c of row r lies at c ^ r, so the 16 rows of a read fall in different banks.
// Operands swapped: lane l has column 4*(l / 16) + r of row l % 16 in
// register r.  Bound by reading B: 16 x 4096 x 16384 28 us, 4.8 TB/s (32 from call
// to call).
template <class T, bool BACKWARD, int ROWS>
__global__ __launch_bounds__(512, 1) void few_kernel(LinearArgs p) {
    constexpr int WAVES = 8, RUN = 128, STEPS = RUN / 32;
    constexpr int STAGE = (16 + ROWS) * 256, RING = ROWS == 16 ? 2 : ROWS == 8 ? 3 : 4, PER = 4 + ROWS / 4;
    __shared__ __attribute__((aligned(1024))) char smem[WAVES * RING * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = int64_t(blockIdx.x) * 16;
    const int row = lane & 15, q = lane >> 4;
    LDS char *lds = (LDS char *)smem + wave * (RING * STAGE);
    const char *pa = reinterpret_cast<const char *>(p.a.p), *pb = reinterpret_cast<const char *>(p.b.p + n0 * p.b.ld);
    uint32_t va[ROWS / 4], vb[4];
    int ca[4];  // this lane's chunk of each row group
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 4 * j + q, c = row ^ r;
        ca[j] = c * 8;
        vb[j] = n0 + r < p.N ? uint32_t(r * p.b.ld * 2 + c * 16) : OOB;
        if (j < ROWS / 4) va[j] = r < p.M ? uint32_t(r * p.a.ld * 2 + c * 16) : OOB;
    }
    const int64_t runs = (p.K + RUN - 1) / RUN, mine = (runs - wave + WAVES - 1) / WAVES;
    auto issue = [&](int64_t n) {
        const int64_t k0 = (wave + n * WAVES) * RUN, left = p.K - k0;
        const u32x4 rb = dma::raw_buffer(static_cast<uint64_t>(uniform(reinterpret_cast<int64_t>(pb + 2 * k0))), 0x7fffffff);
        const u32x4 ra = dma::raw_buffer(static_cast<uint64_t>(uniform(reinterpret_cast<int64_t>(pa + 2 * k0))), 0x7fffffff);
        const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + uint32_t(n % RING) * STAGE;
#pragma unroll
        for (int j = 0; j < 4; ++j) direct_load16(rb, to + j * 1024, ca[j] < left ? vb[j] : OOB);
#pragma unroll
        for (int j = 0; j < ROWS / 4; ++j) direct_load16(ra, to + 4096 + j * 1024, ca[j] < left ? va[j] : OOB);
    };
    f32x4 acc = {0, 0, 0, 0};
    for (int n = 0; n < RING; ++n)
        if (n < mine) issue(n);
    for (int64_t n = 0; n < mine; ++n) {
        const int64_t later = mine - 1 - n;
        if (RING > 3 && later >= 3) wait_vmcnt<(RING > 3 ? 3 : 0) * PER>();
        else if (RING > 2 && later >= 2) wait_vmcnt<(RING > 2 ? 2 : 0) * PER>();
        else if (later >= 1) wait_vmcnt<PER>();
        else wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        const LDS char *stage = lds + int(n % RING) * STAGE;
        u32x4 a[STEPS], b[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int ra = row % ROWS;  // columns past the rows are not stored
            b[s] = *reinterpret_cast<const LDS u32x4 *>(stage + row * 256 + (((4 * s + q) ^ row) << 4));
            a[s] = *reinterpret_cast<const LDS u32x4 *>(stage + 4096 + ra * 256 + (((4 * s + q) ^ ra) << 4));
        }
        wait_lgkmcnt0();
        asm volatile("" ::: "memory");
        if (n + RING < mine) issue(n + RING);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) acc = mfma16<T>(b[s], a[s], acc);
    }
    LDS f32x4 *part = reinterpret_cast<LDS f32x4 *>((LDS char *)smem);
    __syncthreads();  // every wave has read its runs
    part[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        const f32x4 o = part[w * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += o[e];
    }
    // two lanes' four columns to one lane's eight: lanes 0 .. 31 finish
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int from = (lane & 15) + 32 * (lane >> 4 & 1);
        x[e] = __shfl(acc[e], from);
        x[4 + e] = __shfl(acc[e], from + 16);
    }
    const int64_t n = n0 + 8 * (lane >> 4 & 1);
    const int count = p.N - n < 8 ? int(p.N - n) : 8;
    Finish<T, BACKWARD> finish(p, n);
    if (lane < 32 && row < p.M && count > 0) {
        Raw8 data;
        finish.load(data, row, n, count);
        finish(row, n, count, x, data);
    }
    if (!BACKWARD || p.sums == nullptr) return;
    for (int d = 1; d < 16; d *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) finish.column[e] += __shfl_xor(finish.column[e], d);
    if (lane < 32 && row == 0 && count > 0) finish.store_sums(0, n, count, finish.column);
}

// ---------------------------------------------------------------- column sums
// dbias[j] = the sum of rows of sums[.][j], in order, + beta * dbias[j]; 32
// columns per workgroup, eight threads to a column.
__global__ __launch_bounds__(256) void sums_kernel(const float *sums, int64_t rows, int64_t N, float beta,
                                                   float *dbias) {
    __shared__ float part[8][32];
    const int c = threadIdx.x % 32, g = threadIdx.x / 32;
    const int64_t j = int64_t(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (j < N) {
        int64_t r = g;
        for (; r + 56 < rows; r += 64) {  // eight loads under way
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = sums[(r + 8 * i) * N + j];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; r < rows; r += 8) s += sums[r * N + j];
    }
    part[g][c] = s;
    __syncthreads();
    if (g != 0 || j >= N) return;
    for (int i = 1; i < 8; ++i) s += part[i][c];
    dbias[j] = beta != 0.0f ? __builtin_fmaf(beta, dbias[j], s) : s;
}

hipError_t launch_sums(const float *sums, int64_t rows, int64_t N, float beta, float *dbias, hipStream_t stream) {
    sums_kernel<<<dim3(unsigned((N + 31) / 32)), dim3(256), 0, stream>>>(sums, rows, N, beta, dbias);
    return hipGetLastError();
}

// ---------------------------------------------------------------- without a product
// 64 columns by AB_ROWS rows per workgroup of four waves; a thread has eight
// columns and every 32nd row.  Up to AB_ALL rows, a workgroup of sixteen waves
// takes them all and writes the column sums' result (129 x 4097: 5.0 us for 5.6
// and 2.5 in two launches).  Bound by memory: 8192 x 4096 in bf16 43 us, 4.7 TB/s.
constexpr int AB_ROWS = 128, AB_ALL = 512;
struct ActivationArgs {
    ActivationBackward p;
    float *sums;
    int64_t rows;  // per workgroup
};
template <int TYPE>
__device__ inline void load8_type(const void *x, int64_t at, int n, float (&v)[8]) {
    if constexpr (TYPE == 0) load8f(static_cast<const float *>(x) + at, n, v);
    else if constexpr (TYPE == 1) load8<BF16>(static_cast<const uint16_t *>(x) + at, n, v);
    else load8<F16>(static_cast<const uint16_t *>(x) + at, n, v);
}
template <int TA, int TZ, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void activation_kernel(ActivationArgs a) {
    const ActivationBackward &p = a.p;
    __shared__ float waves[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = int64_t(blockIdx.x) * 64 + (threadIdx.x % 8) * 8;
    const int count = p.N - n < 8 ? int(p.N - n) : 8;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    const int64_t end = (int64_t(blockIdx.y) + 1) * a.rows < p.M ? (int64_t(blockIdx.y) + 1) * a.rows : p.M;
    if (count > 0)
        for (int64_t m = int64_t(blockIdx.y) * a.rows + threadIdx.x / 8; m < end; m += WAVES * 8) {
            float x[8], z[8];
            load8_type<TA>(p.A, m * p.lda + n, count, x);
            if (p.act != act::NONE) {
                load8_type<TZ>(p.Z, m * p.ldz + n, count, z);
                act::times_slope(p.act, z, x);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += x[e];
            if (p.D != nullptr) {
                const int64_t at = m * p.ldd + n;
                if (p.type_d == 0) store8f(static_cast<float *>(p.D) + at, count, x);
                else if (p.type_d == 1) store8<BF16>(static_cast<uint16_t *>(p.D) + at, count, x);
                else store8<F16>(static_cast<uint16_t *>(p.D) + at, count, x);
            }
        }
    if (a.sums == nullptr) return;
    for (int d = 8; d < 64; d *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], d);
    if (lane < 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) waves[wave][lane * 8 + e] = sum[e];
    __syncthreads();
    const int64_t j = int64_t(blockIdx.x) * 64 + lane;
    if (wave != 0 || j >= p.N) return;
    float s = waves[0][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += waves[w][lane];
    if (WAVES == 4) a.sums[blockIdx.y * p.N + j] = s;
    else p.dbias[j] = p.beta != 0.0f ? __builtin_fmaf(p.beta, p.dbias[j], s) : s;
}

// ---------------------------------------------------------------- launches
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Slices of K for `tiles` tiles of 128 x 128: two workgroups for each of 256
// compute units, four stages each at least; two, where less than a quarter of them
// had work (fp16, odd leading dimensions: 250 x 1000 x 515, 16 tiles, 15 us for
// 16; but 1000 x 1001 x 1001, 64 tiles, 27 for 23).
int split_slices(int64_t tiles, int64_t K) {
    const int64_t stages = ceil_div(K, 64), want = 512 / tiles, few = 64 / tiles;
    const int64_t s = want < stages / 4 ? want : stages / 4;
    const int64_t more = few < stages / 2 ? few : stages / 2;
    return int(s > more ? s : more > 1 ? more : 1);
}
// K from which slices pay for a second launch and the sums' way through memory.
// bf16, us in slices and not: 4 tiles, K 256 7.6 and 7.5, 512 8.3 and 9.3; 32
// tiles, 512 10.5 and 10.6, 1024 12 and 15; 64 tiles, 1024 20 and 16, 2048 25 and
// 25, 4096 26 and 43; 128 tiles, 2048 29 and 25, 4096 34 and 44; 256 tiles, 512
// 30 and 12, 2048 34 and 27, 4096 51 and 58, 16384 153 and 218.  Panels through
// registers take longer a step: 16 tiles, 256 9.2 and 10; 64 tiles, 512 17 and
// 16, 1024 22 and 26; 128 tiles, 1024 27 and 26, 2048 30 and 44; 256 tiles, 1024 32
// and 26, 2048 42 and 45.
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t split_from(int64_t tiles, bool direct) {
    if (!direct) return least(16 * tiles, 2048);
    return tiles < 16 ? 512 : least(32 * tiles, 4096);
}
int64_t tiles_of(int64_t M, int64_t N, int64_t t) { return ceil_div(M, t) * ceil_div(N, t); }
// Slices of K for the tiles of 256 x 256 that whole rounds of 256 leave over; 1
// where they stay one more round.  A round takes its time however few tiles it
// has: 4095 x 4097 x 1001 (272 tiles) 88 us in two rounds, 51 + 15 + 9 us as a
// round, the slices of 16 tiles and their joining.
int last_slices(int64_t M, int64_t N, int64_t K) {
    const int64_t total = tiles_of(M, N, 256), last = total % 256;
    if (total < 256 || last == 0) return 1;
    const int64_t most = ceil_div(K, 64) / 4, want = 256 / last, s = want < most ? want : most;
    return int(s < 1 ? 1 : s);
}
int64_t round8(int64_t n) { return ceil_div(n, 8) * 8; }
size_t partial_bytes(int64_t M, int64_t N, int slices) { return size_t(slices) * M * round8(N) * 4; }
// Column sums take a row for each 32 rows at least (finish_kernel).
size_t sums_bytes(int64_t M, int64_t N) { return size_t(ceil_div(ceil_div(M, FINISH_ROWS) * N, 64) * 256); }

size_t last_bytes(int64_t M, int64_t N, int slices) { return size_t(tiles_of(M, N, 256) % 256) * slices * 256 * 256 * 4; }

// A launch has less than 2^32 threads: so many tiles, so many columns of 16 per
// workgroup of 512.
constexpr int64_t MOST_TILES = int64_t(1) << 22, MOST_COLUMNS = int64_t(1) << 26;
template <class Shape, class T, bool BACKWARD>
hipError_t run_tiles(LinearArgs &a, int64_t count, hipStream_t stream) {
    for (a.first = 0; a.first < count; a.first += MOST_TILES) {
        a.tiles = count - a.first < MOST_TILES ? count - a.first : MOST_TILES;
        tile_kernel<T, Shape, BACKWARD><<<dim3(unsigned(a.tiles)), dim3(Shape::THREADS), 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <class Shape, class T, bool BACKWARD>
hipError_t run_tile(LinearArgs &a, hipStream_t stream) {
    a.grid = TileGrid{ceil_div(a.M, Shape::TM), ceil_div(a.N, Shape::TN), 1, 8, 1};
    return run_tiles<Shape, T, BACKWARD>(a, a.grid.count(), stream);
}
// Whole rounds of 256 tiles, then the rest in slices of K.
template <class Shape, class T, bool BACKWARD>
hipError_t run_rounds(LinearArgs &a, hipStream_t stream) {
    a.grid = TileGrid{ceil_div(a.M, Shape::TM), ceil_div(a.N, Shape::TN), 1, 8, 1};
    const int64_t total = a.grid.count(), whole = total / 256 * 256;
    hipError_t e = run_tiles<Shape, T, BACKWARD>(a, whole, stream);
    if (e != hipSuccess) return e;
    a.first = whole;
    a.tiles = total - whole;
    last_kernel<Shape><<<dim3(unsigned(a.tiles * a.slices)), dim3(Shape::THREADS), 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    last_finish_kernel<T, Shape, BACKWARD>
        <<<dim3(Shape::TN / 64, Shape::TM / Shape::WTM, unsigned(a.tiles)), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}
template <class Shape, class T, bool BACKWARD>
hipError_t run_split(LinearArgs &a, hipStream_t stream) {
    a.grid = TileGrid{ceil_div(a.M, Shape::TM), ceil_div(a.N, Shape::TN), a.slices, 8, 8};
    split_kernel<Shape><<<dim3(unsigned(a.grid.count())), dim3(Shape::THREADS), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned columns = unsigned(ceil_div(a.N, 64));
    if constexpr (BACKWARD) {
        if (a.dbias != nullptr) {
            finish_kernel<T, true, 8><<<dim3(columns), dim3(512), 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    finish_kernel<T, BACKWARD, 4><<<dim3(columns, unsigned(ceil_div(a.M, FINISH_ROWS))), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, bool BACKWARD, bool BKM>
hipError_t run_kernel(LinearKernel k, LinearArgs &a, hipStream_t stream) {
    using T256 = Tile<T, 256, 256, 2, 4, true, BKM, true>;
    using T128 = Tile<T, 128, 128, 2, 2, true, BKM, true>;
    using Any = Tile<T, 128, 128, 2, 2, true, BKM, false>;
    switch (k) {
        case LinearKernel::Tile256: return run_tile<T256, T, BACKWARD>(a, stream);
        case LinearKernel::Rounds: return run_rounds<T256, T, BACKWARD>(a, stream);
        case LinearKernel::Tile128: return run_tile<T128, T, BACKWARD>(a, stream);
        case LinearKernel::Any: return run_tile<Any, T, BACKWARD>(a, stream);
        case LinearKernel::Split: return run_split<T128, T, BACKWARD>(a, stream);
        case LinearKernel::AnySplit: return run_split<Any, T, BACKWARD>(a, stream);
        case LinearKernel::Few16:
            if (a.M <= 4) few_kernel<T, BACKWARD, 4><<<dim3(unsigned(ceil_div(a.N, 16))), dim3(512), 0, stream>>>(a);
            else if (a.M <= 8) few_kernel<T, BACKWARD, 8><<<dim3(unsigned(ceil_div(a.N, 16))), dim3(512), 0, stream>>>(a);
            else few_kernel<T, BACKWARD, 16><<<dim3(unsigned(ceil_div(a.N, 16))), dim3(512), 0, stream>>>(a);
            return hipGetLastError();
        default: return hipSuccess;
    }
}

// Up to so many rows, a workgroup of finish_kernel takes them all for its columns
// and writes the column sums' result, which saves a launch; for more rows it takes
// longer than that (250 x 1000 in four slices of K: 8.5 us, 4.1 + 2.4 in two).
constexpr int64_t ONE_BLOCK = 64;
int64_t sums_rows(LinearKernel k, int64_t M) {
    switch (k) {
        case LinearKernel::Few16: return 1;
        case LinearKernel::Tile256:
        case LinearKernel::Rounds: return ceil_div(M, 128);
        case LinearKernel::Split:
        case LinearKernel::AnySplit: return M <= ONE_BLOCK ? 1 : ceil_div(M, FINISH_ROWS);
        default: return ceil_div(M, 64);
    }
}

bool whole_chunks(const void *x, int64_t ld, int64_t inner) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld % 8 == 0 && inner % 8 == 0 && ld <= MOST_LD;
}

// Copies of operands that direct loads do not take, with rows of whole lines.
int64_t round64(int64_t n) { return ceil_div(n, 64) * 64; }
PackSpec pack_a(const LinearProblem &p) { return {p.A, p.M, p.K, p.lda, 0, 1, p.M, round64(p.K), 2}; }
PackSpec pack_b(const LinearProblem &p) {
    const int64_t outer = p.b_kmajor ? p.N : p.K, inner = p.b_kmajor ? p.K : p.N;
    return {p.B, outer, inner, p.ldb, 0, 1, outer, round64(inner), 2};
}
// Elements of an operand and of a copy: their offsets stay below 2^31 bytes.
constexpr int64_t PACK_MOST = (int64_t(1) << 30) - 64;
bool can_pack(const PackSpec &s) {
    const int64_t ld = s.ld > s.inner_p ? s.ld : s.inner_p;
    return s.outer <= PACK_MOST && ld <= MOST_LD && s.outer * ld <= PACK_MOST;
}
// Copying pays where eight tiles or more read each operand and K is not short:
// fp16, operands with odd leading dimensions, a row-major B, copied and not:
// 2049 x 2049 x 2049 54 and 71 us, 4095 x 16385 x 4097 657 and 952, but 1000 x
// 1001 x 1001 26 and 24, 4095 x 4097 x 65 48 and 40.  Fewer rows gain little (250 x
// 4097 x 4095 42 and 45) for a workspace that holds all of B.
bool worth_packing(int64_t M, int64_t N, int64_t K) { return M >= 1024 && N >= 1024 && K >= 512; }
// What the kernels take beside copies.
size_t own_bytes(int64_t M, int64_t N, int64_t K) {
    const int slices = split_slices(tiles_of(M, N, 128), K), last = last_slices(M, N, K);
    const bool split = slices > 1 && K >= split_from(tiles_of(M, N, 128), false);
    return sums_bytes(M, N) + (split ? partial_bytes(M, N, slices) : 0) + (last > 1 ? last_bytes(M, N, last) : 0);
}
// What copies of both operands take where a row of either may not be whole chunks
// (rows that are usually start on them).
size_t pack_bytes(int64_t M, int64_t N, int64_t K) {
    if (!worth_packing(M, N, K) || (K % 8 == 0 && N % 8 == 0)) return 0;
    if (M > PACK_MOST / 512 || N > PACK_MOST / 512 || K > PACK_MOST / 512) return 0;
    const int64_t a = M * round64(K), b = N * round64(K) > K * round64(N) ? N * round64(K) : K * round64(N);
    return a > PACK_MOST || b > PACK_MOST ? 0 : size_t(a + b) * 2;
}

}  // namespace

const char *linear_kernel_name(LinearKernel k) {
    switch (k) {
        case LinearKernel::Few16: return "linear_few_16";
        case LinearKernel::Tile256: return "linear_mfma_256";
        case LinearKernel::Rounds: return "linear_mfma_256_rounds";
        case LinearKernel::Tile128: return "linear_mfma_128";
        case LinearKernel::Split: return "linear_mfma_128_split";
        case LinearKernel::Any: return "linear_mfma_any";
        case LinearKernel::AnySplit: return "linear_mfma_any_split";
        case LinearKernel::Packed: return "linear_packed";
        default: return "";
    }
}

hipError_t launch_no_sums(int64_t N, float beta, float *dbias, hipStream_t stream) {
    return launch_sums(nullptr, 0, N, beta, dbias, stream);
}

size_t linear_workspace(int64_t M, int64_t N, int64_t K) { return own_bytes(M, N, K) + pack_bytes(M, N, K) + 16; }

// The problem on copies of the operands that need one, at the workspace's end;
// false where they do not fit into it.
static bool packed_problem(const LinearProblem &p, LinearProblem &q, PackSpec specs[2], void *dst[2], int &n) {
    n = 0;
    if (!worth_packing(p.M, p.N, p.K) || p.workspace == nullptr) return false;
    q = p;
    size_t left = p.workspace_bytes / 16 * 16;
    auto copy = [&](const PackSpec &s, const void *&x, int64_t &ld) {
        const size_t need = size_t(packed_bytes(s));
        if (!can_pack(s) || need > left) return false;
        left -= need;
        specs[n] = s;
        dst[n++] = static_cast<char *>(p.workspace) + left;
        x = static_cast<char *>(p.workspace) + left;
        ld = s.inner_p;
        return true;
    };
    if (!whole_chunks(p.A, p.lda, p.K) && !copy(pack_a(p), q.A, q.lda)) return false;
    if (!whole_chunks(p.B, p.ldb, p.b_kmajor ? p.K : p.N) && !copy(pack_b(p), q.B, q.ldb)) return false;
    q.workspace_bytes = left;
    q.packed = true;
    return left >= own_bytes(p.M, p.N, p.K);
}

LinearKernel linear_choose(const LinearProblem &p) {
    if (p.M == 0 || p.N == 0) return LinearKernel::None;
    const bool direct = p.packed || (p.K > 0 && whole_chunks(p.A, p.lda, p.K) && whole_chunks(p.B, p.ldb, p.b_kmajor ? p.K : p.N));
    // 16 rows so, and 17 in slices of tiles: 4096 x 1024 4.5 and 10 us, 4096 x 4096 9.6
    // and 17.5, 4096 x 16384 32 and 41
    if (direct && p.b_kmajor && p.M <= 16 && p.N <= MOST_COLUMNS) return LinearKernel::Few16;
    if (!direct) {
        LinearProblem q;
        PackSpec specs[2];
        void *dst[2];
        int n;
        if (packed_problem(p, q, specs, dst, n)) return LinearKernel::Packed;
    }
    const int64_t t128 = tiles_of(p.M, p.N, 128);
    const int slices = p.K > 0 ? split_slices(t128, p.K) : 1;
    const bool split = slices > 1 && p.K >= split_from(t128, direct) && p.workspace != nullptr &&
                       p.workspace_bytes >= sums_bytes(p.M, p.N) + partial_bytes(p.M, p.N, slices);
    if (!direct) return split ? LinearKernel::AnySplit : LinearKernel::Any;
    if (split) return LinearKernel::Split;
    const int last = last_slices(p.M, p.N, p.K);
    if (last > 1 && p.workspace != nullptr && p.workspace_bytes >= sums_bytes(p.M, p.N) + last_bytes(p.M, p.N, last))
        return LinearKernel::Rounds;
    // 128 x 128 tiles while one round takes them all, two to a compute unit (bf16, K
    // 4096: 2560 x 2560, 400 tiles, 63 us, of 256 88; 3328 x 3328, 676 tiles, 105, of
    // 256 93; 4096 x 4096 137 and 116)
    return t128 <= 512 ? LinearKernel::Tile128 : LinearKernel::Tile256;
}

hipError_t launch_linear(LinearKernel k, const LinearProblem &p, hipStream_t stream) {
    if (k == LinearKernel::None)
        return p.dbias != nullptr && p.N > 0 ? launch_no_sums(p.N, p.beta_bias, p.dbias, stream) : hipSuccess;
    if (k == LinearKernel::Packed) {
        LinearProblem q;
        PackSpec specs[2];
        void *dst[2];
        int n;
        if (!packed_problem(p, q, specs, dst, n)) return hipErrorInvalidValue;
        const hipError_t e = n == 2 ? launch_pack2(specs[0], dst[0], specs[1], dst[1], stream) : launch_pack(specs[0], dst[0], stream);
        return e != hipSuccess ? e : launch_linear(linear_choose(q), q, stream);
    }
    LinearArgs a{};
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.alpha = p.alpha;
    a.beta = p.beta;
    a.a = Operand16{static_cast<const uint16_t *>(p.A), p.lda, p.M};
    a.b = Operand16{static_cast<const uint16_t *>(p.B), p.ldb, p.N};
    a.bias = static_cast<const uint16_t *>(p.bias);
    a.R = p.R;
    a.C = p.C;
    a.Z = static_cast<uint16_t *>(p.Z);
    a.ldr = p.ldr;
    a.ldc = p.ldc;
    a.ldz = p.ldz;
    a.act = p.act;
    a.c_same = p.out != 0;
    a.sums = p.dbias != nullptr ? static_cast<float *>(p.workspace) : nullptr;
    a.dbias = sums_rows(k, p.M) == 1 ? p.dbias : nullptr;
    a.beta_bias = p.beta_bias;
    a.ldp = round8(p.N);
    if (k == LinearKernel::Split || k == LinearKernel::AnySplit) a.slices = split_slices(tiles_of(p.M, p.N, 128), p.K);
    if (k == LinearKernel::Rounds) a.slices = last_slices(p.M, p.N, p.K);
    if (a.slices > 1)
        a.partial = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + sums_bytes(p.M, p.N));
    hipError_t e;
    if (p.in == 1) {
        if (p.backward) e = p.b_kmajor ? run_kernel<BF16, true, true>(k, a, stream) : run_kernel<BF16, true, false>(k, a, stream);
        else e = p.b_kmajor ? run_kernel<BF16, false, true>(k, a, stream) : run_kernel<BF16, false, false>(k, a, stream);
    } else {
        if (p.backward) e = p.b_kmajor ? run_kernel<F16, true, true>(k, a, stream) : run_kernel<F16, true, false>(k, a, stream);
        else e = p.b_kmajor ? run_kernel<F16, false, true>(k, a, stream) : run_kernel<F16, false, false>(k, a, stream);
    }
    if (e != hipSuccess || p.dbias == nullptr || a.dbias != nullptr) return e;
    return launch_sums(a.sums, sums_rows(k, p.M), p.N, p.beta_bias, p.dbias, stream);
}

size_t activation_backward_workspace(int64_t M, int64_t N) { return size_t(ceil_div(M, AB_ROWS)) * N * 4 + 16; }

hipError_t launch_activation_backward(const ActivationBackward &p, hipStream_t stream) {
    const bool all = p.dbias != nullptr && p.M <= AB_ALL && p.N <= MOST_COLUMNS;
    // a grid has at most 65535 rows of workgroups
    const int64_t rows = all ? p.M : AB_ROWS * ceil_div(p.M, AB_ROWS * int64_t(65535)), blocks = ceil_div(p.M, rows);
    ActivationArgs a{p, p.dbias != nullptr ? static_cast<float *>(p.workspace) : nullptr, rows};
    const unsigned columns = unsigned(ceil_div(p.N, 64));
    auto run = [&](auto few, auto many) {
        if (all) few<<<dim3(columns), dim3(1024), 0, stream>>>(a);
        else many<<<dim3(columns, unsigned(blocks)), dim3(256), 0, stream>>>(a);
    };
    switch (p.type_a * 3 + (p.act == act::NONE ? p.type_a : p.type_z)) {
        case 0: run(activation_kernel<0, 0, 16>, activation_kernel<0, 0, 4>); break;
        case 1: run(activation_kernel<0, 1, 16>, activation_kernel<0, 1, 4>); break;
        case 2: run(activation_kernel<0, 2, 16>, activation_kernel<0, 2, 4>); break;
        case 3: run(activation_kernel<1, 0, 16>, activation_kernel<1, 0, 4>); break;
        case 4: run(activation_kernel<1, 1, 16>, activation_kernel<1, 1, 4>); break;
        case 5: run(activation_kernel<1, 2, 16>, activation_kernel<1, 2, 4>); break;
        case 6: run(activation_kernel<2, 0, 16>, activation_kernel<2, 0, 4>); break;
        case 7: run(activation_kernel<2, 1, 16>, activation_kernel<2, 1, 4>); break;
        default: run(activation_kernel<2, 2, 16>, activation_kernel<2, 2, 4>); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.dbias == nullptr || all) return e;
    return launch_sums(a.sums, blocks, p.N, p.beta, p.dbias, stream);
}

}  // namespace libgemm
