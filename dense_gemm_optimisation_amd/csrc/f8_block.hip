// Products of 8-bit floats with one fp32 scale per 128 of the contracted
// dimension, for each row or for each 128 rows of an operand; whole, over
// segments of A's rows with a B each, or over segments of the contracted
// dimension with a C each.
//
//   C(i, j) = alpha * sum_kb sA(kb, i) sB(kb, j) P_kb(i, j) + beta C(i, j),
//   P_kb(i, j) = sum of A(i, k) B(j, k) over the 128 k of block kb
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 (its own scales 2^0, its accumulator
// input 0) forms P_kb of a 16 x 16 block; the vector ALUs add it, times the
// two scales, to the fp32 accumulators.  The operands are swapped (B's
// fragment first), so a lane's four values are consecutive columns of one
// row of C: with a scale per 128 rows of B all four share one factor.
#include "dma_tile.hpp"
#include "f8_block.hpp"

#ifndef LIBGEMM_BLOCK_PART
#define LIBGEMM_BLOCK_PART -1
#endif
#define LIBGEMM_BLOCK_HAS(part) (LIBGEMM_BLOCK_PART < 0 || LIBGEMM_BLOCK_PART == (part))

namespace libgemm {

// The tile kernel for formats FA, FB (0 E4M3, 1 E5M2), defined in the part of
// those formats.
template <int FA, int FB>
hipError_t block_tile_formats(const BlockProblem &p, hipStream_t stream);

namespace {

using dma::OOB;
using dma::direct_load16;
using dma::direct_load4;
using dma::uniform;
using dma::wait_vmcnt;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int UNIT = 0x7F7F7F7F;  // E8M0 2^0 in every byte

struct BlockArgs {
    BlockProblem p;
    TileGrid grid;
};

// 16-byte chunk c of a panel's 128-byte row r sits at c ^ swz(r): the 16 rows
// one fragment read touches at one chunk fall in distinct banks.
__device__ inline int swz(int row) { return (row ^ (row >> 3)) & 7; }

// ROWS rows of an operand, 128 k deep, in LDS: direct loads of 1 KiB (8 rows)
// fill it.
template <int ROWS, int WAVES>
struct Panel {
    static constexpr int BYTES = ROWS * 128;
    static constexpr int PER_WAVE = ROWS / 8 / WAVES;
    static_assert(PER_WAVE >= 1 && ROWS % (8 * WAVES) == 0, "panel split over waves");
    uint32_t voff[PER_WAVE];
    int k[PER_WAVE];  // this lane's first k within a stage
    int64_t base;
    int64_t bytes;

    // Rows r0 .. r0 + nrows - 1 (nrows <= ROWS valid) from byte k0 of each row on, K of them.
    __device__ void init(const uint8_t *x, int64_t ld, int64_t r0, int64_t nrows, int64_t k0,
                         int64_t K, int wave, int lane) {
        base = uniform(reinterpret_cast<int64_t>(x) + r0 * ld + k0);
        bytes = uniform((nrows - 1) * ld + ((K + 15) & ~int64_t(15)));
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int row = (wave * PER_WAVE + i) * 8 + (lane >> 3);
            const int c = (lane & 7) ^ swz(row);
            k[i] = c * 16;
            voff[i] = row < nrows ? uint32_t(row * ld + c * 16) : OOB;
        }
    }

    // All of this wave's loads for the stage at k = 128*stage, kleft = K - 128*stage > 0.
    __device__ void issue(LDS char *dst, int64_t stage, int64_t kleft, int wave) const {
        const u32x4 rs = dma::raw_buffer(static_cast<uint64_t>(base + 128 * stage),
                                         static_cast<uint32_t>(bytes - 128 * stage));
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst));
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i)
            direct_load16(rs, at + (wave * PER_WAVE + i) * 1024, k[i] < kleft ? voff[i] : OOB);
    }

    // The lane's 32 bytes of row row0 + lane % 16: chunks lane/16 and 4 + lane/16.  Both
    // operands take the same k in the same place, so which k that is does not matter.
    __device__ static i32x8 frag(const LDS char *panel, int row0, int lane) {
        const int row = row0 + (lane & 15), c = lane >> 4;
        const LDS char *r = panel + row * 128;
        const u32x4 lo = *reinterpret_cast<const LDS u32x4 *>(r + ((c ^ swz(row)) << 4));
        const u32x4 hi = *reinterpret_cast<const LDS u32x4 *>(r + (((c + 4) ^ swz(row)) << 4));
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                     int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    }
};

// Segment `e` of the offsets, cut to [0, limit).
__device__ inline void segment_of(const int32_t *offsets, int64_t e, int64_t limit, int64_t &lo,
                                  int64_t &hi) {
    auto cut = [&](int64_t v) { return v < 0 ? int64_t(0) : v > limit ? limit : v; };
    lo = cut(offsets[e]);
    hi = cut(offsets[e + 1]);
    if (hi < lo) hi = lo;
}

// The segment that holds tile row `tm` when every segment of the rows starts
// a tile of its own, and the tile's first row; false when there are fewer
// tiles.  Each wave finds it alone, 64 segments at a time.
__device__ inline bool find_segment(const BlockProblem &p, int64_t tm, int BM, int lane, int64_t &e,
                                    int64_t &m0, int64_t &end) {
    int64_t before = 0;
    for (int64_t e0 = 0; e0 < p.batch; e0 += 64) {
        int64_t lo = 0, hi = 0;
        if (e0 + lane < p.batch) segment_of(p.offsets, e0 + lane, p.M, lo, hi);
        const int tiles = int((hi - lo + BM - 1) / BM);
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const uint64_t past = __ballot(before + sum > tm);
        if (past) {
            const int l = __builtin_ctzll(past);
            e = uniform(e0 + l);
            const int64_t first = before + __shfl(sum, l) - __shfl(tiles, l);
            m0 = uniform(__shfl(lo, l) + (tm - first) * BM);
            end = uniform(__shfl(hi, l));
            return true;
        }
        before += __shfl(sum, 63);
    }
    return false;
}

template <int OUT>
__device__ inline void store_one(const BlockProblem &p, int64_t at, float v) {
    if (OUT == 0) {
        float *c = static_cast<float *>(p.C) + at;
        *c = p.beta != 0.0f ? __builtin_fmaf(p.beta, *c, v) : v;
    } else {
        uint16_t *c = static_cast<uint16_t *>(p.C) + at;
        if (p.beta != 0.0f) {
            const float old = OUT == 1 ? __builtin_bit_cast(float, uint32_t(*c) << 16)
                                       : static_cast<float>(__builtin_bit_cast(_Float16, *c));
            v = __builtin_fmaf(p.beta, old, v);
        }
        *c = OUT == 1 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v))
                      : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
}

// One workgroup per BM x BN tile, WAVES_M x WAVES_N waves of FM x FN blocks.
template <int FA, int FB, bool PER_COLUMN, int WAVES_M, int WAVES_N, int FM, int FN>
__global__ __launch_bounds__(WAVES_M *WAVES_N * 64) void block_tile_kernel(BlockArgs a) {
    constexpr int WAVES = WAVES_M * WAVES_N;
    constexpr int WTM = FM * 16, WTN = FN * 16, BM = WAVES_M * WTM, BN = WAVES_N * WTN;
    static_assert(128 % WTN == 0, "a wave's columns lie in one block of 128");
    using PA = Panel<BM, WAVES>;
    using PB = Panel<BN, WAVES>;
    __shared__ __attribute__((aligned(1024))) char smem[PA::BYTES + PB::BYTES + (BM + BN) * 4];
    LDS char *lds = (LDS char *)smem;
    LDS char *lds_b = lds + PA::BYTES;
    LDS float *sc = reinterpret_cast<LDS float *>(lds_b + PB::BYTES);
    const BlockProblem &p = a.p;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;

    const TileCoord t = tile_of(a.grid, blockIdx.x);
    int64_t e = uniform(t.batch), m0 = uniform(t.tm) * BM, m_end = p.M, k_lo = 0, k_hi = p.K;
    const int64_t n0 = uniform(t.tn) * BN;
    if (p.segments == Segments::Rows && !find_segment(p, uniform(t.tm), BM, lane, e, m0, m_end)) return;
    if (p.segments == Segments::Contracted) {
        segment_of(p.offsets, e, p.K, k_lo, k_hi);
        k_lo = uniform(k_lo) & ~int64_t(127);
        k_hi = uniform(k_hi);
    }
    const int64_t K = k_hi - k_lo, kb0 = k_lo / 128;
    const int64_t ea = p.segments == Segments::None ? e : 0;
    const int64_t eb = p.segments == Segments::Contracted ? 0 : e;
    const int64_t ec = p.segments == Segments::Rows ? 0 : e;
    const int64_t mrows = m_end - m0 < BM ? m_end - m0 : BM, nrows = p.N - n0 < BN ? p.N - n0 : BN;

    PA pa;
    PB pb;
    pa.init(p.a.x + ea * p.a.stride, p.a.ld, m0, mrows, k_lo, K, wave, lane);
    pb.init(p.b.x + eb * p.b.stride, p.b.ld, n0, nrows, k_lo, K, wave, lane);

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int64_t steps = (K + 127) / 128;
    for (int64_t s = 0; s < steps; ++s) {
        const int64_t kleft = K - 128 * s;
        pa.issue(lds, s, kleft, wave);
        pb.issue(lds_b, s, kleft, wave);
        // the scales of the panel rows: row m0 + i of A, n0 + i of B
        for (int i = tid; i < BM + BN; i += WAVES * 64) {
            const bool on_a = i < BM;
            const BlockOperand &o = on_a ? p.a : p.b;
            const int r = on_a ? i : i - BM;
            const float *src = o.s + (on_a ? ea : eb) * o.sstride + (kb0 + s) * o.lds;
            sc[i] = r < (on_a ? mrows : nrows) ? src[((on_a ? m0 : n0) + r) >> o.shift] : 0.0f;
        }
        wait_vmcnt<0>();
        __syncthreads();
        if (kleft < 128 && (K & 15) != 0) {
            // the chunk that holds the end of K: its bytes from there on are not the operand's
            const int c = int(kleft >> 4), from = int(kleft & 15);
            for (int r = tid; r < BM + BN; r += WAVES * 64) {
                LDS char *row = r < BM ? lds + r * 128 : lds_b + (r - BM) * 128;
                const int rr = r < BM ? r : r - BM;
                for (int b = from; b < 16; ++b) row[((c ^ swz(rr)) << 4) + b] = 0;
            }
            __syncthreads();
        }
        i32x8 fb[FN];
        f32x4 sb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            fb[j] = PB::frag(lds_b, wn * WTN + j * 16, lane);
            sb[j] = *reinterpret_cast<const LDS f32x4 *>(sc + BM + wn * WTN + j * 16 + 4 * (lane >> 4));
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const i32x8 fa = PA::frag(lds, wm * WTM + i * 16, lane);
            const float sa = sc[wm * WTM + i * 16 + (lane & 15)];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fb[j], fa, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, UNIT, 0, UNIT);
                if (PER_COLUMN) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][r] = __builtin_fmaf(part[r], sa * sb[j][r], acc[i][j][r]);
                } else {
                    const float f = sa * sb[0][0];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(part[r], f, acc[i][j][r]);
                }
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + wm * WTM + i * 16 + (lane & 15);
        if (m >= m_end) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + wn * WTN + j * 16 + 4 * (lane >> 4) + r;
                if (n >= p.N) continue;
                const int64_t at = ec * p.sC + m * p.ldc + n;
                const float v = p.alpha * acc[i][j][r];
                if (p.out == 0) store_one<0>(p, at, v);
                else if (p.out == 1) store_one<1>(p, at, v);
                else store_one<2>(p, at, v);
            }
    }
}

template <int FA, int FB, bool PER_COLUMN>
hipError_t tile_go(const BlockProblem &p, hipStream_t stream) {
    constexpr int WM = 2, WN = 2, FM = 4, FN = 4, BM = WM * FM * 16, BN = WN * FN * 16;
    BlockArgs a{};
    a.p = p;
    int64_t tiles_m = (p.M + BM - 1) / BM;
    if (p.segments == Segments::Rows) {  // every segment that is not empty starts a tile
        const int64_t more = p.batch < p.M ? p.batch : p.M;
        tiles_m = p.M / BM + more < p.M ? p.M / BM + more : p.M;
    }
    a.grid = TileGrid{tiles_m, (p.N + BN - 1) / BN, p.segments == Segments::Rows ? 1 : p.batch, 8, 8};
    if (a.grid.count() > 0x7fffffff) return hipErrorInvalidConfiguration;
    void *args[] = {&a};
    return hipLaunchKernel(
        reinterpret_cast<const void *>(&block_tile_kernel<FA, FB, PER_COLUMN, WM, WN, FM, FN>),
        dim3(static_cast<unsigned>(a.grid.count())), dim3(WM * WN * 64), args, 0, stream);
}

}  // namespace

#define LIBGEMM_BLOCK_FORMATS(part, FA, FB)                                               \
    template <>                                                                           \
    hipError_t block_tile_formats<FA, FB>(const BlockProblem &p, hipStream_t stream) {    \
        return p.b.shift == 0 ? tile_go<FA, FB, true>(p, stream)                          \
                              : tile_go<FA, FB, false>(p, stream);                        \
    }
#if LIBGEMM_BLOCK_HAS(0)
LIBGEMM_BLOCK_FORMATS(0, 0, 0)
#endif
#if LIBGEMM_BLOCK_HAS(1)
LIBGEMM_BLOCK_FORMATS(1, 0, 1)
#endif
#if LIBGEMM_BLOCK_HAS(2)
LIBGEMM_BLOCK_FORMATS(2, 1, 0)
#endif
#if LIBGEMM_BLOCK_HAS(3)
LIBGEMM_BLOCK_FORMATS(3, 1, 1)
#endif

#if LIBGEMM_BLOCK_PART <= 0
BlockKernel block_choose(const BlockProblem &p, bool tiles_only) {
    (void)tiles_only;
    if (p.M == 0 || p.N == 0 || p.batch == 0) return BlockKernel::None;
    return BlockKernel::Tile;
}

const char *block_kernel_name(BlockKernel k) {
    switch (k) {
    case BlockKernel::None: return "";
    case BlockKernel::Tile: return "f8block_mfma";
    }
    return "";
}

hipError_t launch_block(BlockKernel k, const BlockProblem &p, hipStream_t stream) {
    if (k == BlockKernel::None) return hipSuccess;
    if (p.a.e5m2) return p.b.e5m2 ? block_tile_formats<1, 1>(p, stream) : block_tile_formats<1, 0>(p, stream);
    return p.b.e5m2 ? block_tile_formats<0, 1>(p, stream) : block_tile_formats<0, 0>(p, stream);
}
#endif

}  // namespace libgemm
