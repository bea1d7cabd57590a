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
#include <type_traits>

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
hipError_t block_tile_formats(BlockKernel k, const BlockProblem &p, hipStream_t stream);

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

// 16-byte chunk c of a panel's 128-byte row r sits at c ^ swz(r).  The 16 rows
// one fragment read touches at one chunk differ in (r % 2, swz(r)): they fall
// in distinct 16-byte groups of the 256 bytes the banks span.  It does not
// change from one 16-row block to the next, so a lane's address is the same
// for all blocks but for a constant.
__device__ inline int swz(int row) { return (row >> 1) & 7; }

// ROWS rows of an operand, 128 k deep, in LDS: direct loads of 1 KiB (8 rows)
// fill it.
template <int ROWS, int WAVES>
struct Panel {
    static constexpr int BYTES = ROWS * 128;
    static constexpr int PER_WAVE = ROWS / 8 / WAVES;
    static_assert(PER_WAVE >= 1 && ROWS % (8 * WAVES) == 0, "panel split over waves");
    uint32_t voff[PER_WAVE];
    int64_t base;
    uint32_t bytes;

    // This lane's first k, within a stage, in load i.
    __device__ static int lane_k(int i, int wave, int lane) {
        return ((lane & 7) ^ swz((wave * PER_WAVE + i) * 8 + (lane >> 3))) * 16;
    }

    // Rows r0 .. r0 + nrows - 1 (nrows <= ROWS valid) from byte k0 of each row
    // on, K of them (ld < 2^22: a tile's rows lie within 2^30 bytes).
    __device__ void init(const uint8_t *x, int64_t ld, int64_t r0, int nrows, int64_t k0, int K, int wave, int lane) {
        base = uniform(reinterpret_cast<int64_t>(x) + r0 * ld + k0);
        const uint32_t pitch = uint32_t(ld);
        bytes = uint32_t(uniform(int64_t(uint32_t(nrows - 1) * pitch + ((uint32_t(K) + 15) & ~15u))));
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int row = (wave * PER_WAVE + i) * 8 + (lane >> 3);
            voff[i] = row < nrows ? uint32_t(row) * pitch + lane_k(i, wave, lane) : OOB;
        }
    }

    // The stage at k = 128*stage; nothing of it is read where `live` is not set.
    __device__ u32x4 stage(int stage, bool live) const {
        return dma::raw_buffer(static_cast<uint64_t>(base + 128 * stage), live ? bytes - 128u * stage : 0u);
    }
    // Load i of this wave's for the stage rs with kleft = K - 128*stage; what
    // lies past K reads as zero but for the rest of K's last chunk.
    __device__ void load(u32x4 rs, uint32_t at, int i, int kleft, int wave, int lane) const {
        direct_load16(rs, at + (wave * PER_WAVE + i) * 1024, lane_k(i, wave, lane) < kleft ? voff[i] : OOB);
    }
};

// The lane's 32 bytes of row row0 + lane % 16 (row0 a multiple of 16): chunks
// lane/16 and 4 + lane/16.  Both operands take the same k in the same place,
// so which k that is does not matter.  `at` is lane_chunk(lane).
__device__ inline int lane_chunk(int lane) {
    return (lane & 15) * 128 + (((lane >> 4) ^ swz(lane & 15)) << 4);
}
__device__ inline i32x8 frag(const LDS char *panel, int row0, int at) {
    const u32x4 lo = *reinterpret_cast<const LDS u32x4 *>(panel + row0 * 128 + at);
    const u32x4 hi = *reinterpret_cast<const LDS u32x4 *>(panel + row0 * 128 + (at ^ 64));
    return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                 int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
}

// Segment `e` of the offsets, cut to [0, limit).
__device__ inline void segment_of(const int32_t *offsets, int64_t e, int64_t limit, int64_t &lo,
                                  int64_t &hi) {
    auto cut = [&](int64_t v) { return v < 0 ? int64_t(0) : v > limit ? limit : v; };
    lo = cut(offsets[e]);
    hi = cut(offsets[e + 1]);
    if (hi < lo) hi = lo;
}

// 64 segments of rows from e0 on, one per lane, and their tiles when every
// segment starts a tile of its own: sum counts those of the lanes up to this.
struct SegmentTiles {
    int64_t lo, hi;
    int tiles, sum;
    __device__ SegmentTiles(const BlockProblem &p, int64_t e0, int BM, int lane) {
        lo = hi = 0;
        if (e0 + lane < p.batch) segment_of(p.offsets, e0 + lane, p.M, lo, hi);
        sum = tiles = int((hi - lo + BM - 1) / BM);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
    }
    __device__ int64_t total() const { return __shfl(sum, 63); }
};

// All segments' tiles (at most `most`); first: the first 64 segments.
__device__ inline uint32_t tile_rows(const BlockProblem &p, const SegmentTiles &first, int64_t most, int BM, int lane) {
    int64_t n = first.total();
    for (int64_t e0 = 64; e0 < p.batch; e0 += 64) n += SegmentTiles(p, e0, BM, lane).total();
    return uint32_t(uniform(n < most ? n : most));
}

// The segment that holds tile row `tm`, and the tile's first row; false when
// there are fewer tiles.  Each wave finds it alone.
__device__ inline bool find_segment(const BlockProblem &p, SegmentTiles s, int64_t tm, int BM, int lane, int64_t &e,
                                    int64_t &m0, int64_t &end) {
    int64_t before = 0;
    for (int64_t e0 = 0; e0 < p.batch; e0 += 64) {
        if (e0 > 0) s = SegmentTiles(p, e0, BM, lane);
        const uint64_t past = __ballot(before + s.sum > tm);
        if (past) {
            const int l = __builtin_ctzll(past);
            e = uniform(e0 + l);
            const int64_t first = before + __shfl(s.sum, l) - __shfl(s.tiles, l);
            m0 = uniform(__shfl(s.lo, l) + (tm - first) * BM);
            end = uniform(__shfl(s.hi, l));
            return true;
        }
        before += s.total();
    }
    return false;
}

// The n-th longest of at most 64 segments (of equal ones the first): the long
// ones' tiles start first, so that the short ones fill the end of the launch.
__device__ inline int64_t by_length(const BlockProblem &p, int64_t n, int lane) {
    int64_t lo = 0, hi = -1;  // lanes without a segment come last
    if (lane < p.batch) segment_of(p.offsets, lane, p.K, lo, hi);
    const int length = int(hi - lo);
    int ahead = 0;
    for (int i = 0; i < int(p.batch); ++i) {
        const int other = __builtin_amdgcn_readlane(length, i);
        ahead += other > length || (other == length && i < lane);
    }
    return uniform(int64_t(__builtin_ctzll(__ballot(lane < p.batch && ahead == int(n)))));
}

typedef uint32_t u32x2_ea __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_ea __attribute__((ext_vector_type(4), aligned(2)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// Two values rounded to bf16 (OUT 1) or fp16 (2), the first in the low half.
template <int OUT>
__device__ inline uint32_t pack2(float x, float y) {
    const f32x2 v = {x, y};
    return OUT == 1 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2))
                    : __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// W consecutive columns (4, or 8 of a 16-bit type) of a row of C at element
// `at` of `base`, the first `n` of them inside C (n >= W: all): v + beta * C,
// rounded.  Rows of C start at any element: the accesses are element-aligned
// only.
template <int OUT, int W>
__device__ inline void store_columns(const BlockProblem &p, char *base, int64_t at, const float *v, int n) {
    auto old = [](uint32_t b) {
        return OUT == 1 ? __builtin_bit_cast(float, b << 16)
                        : static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(b)));
    };
    auto bits = [](float x) {
        return uint32_t(OUT == 1 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(x))
                                 : __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)));
    };
    if constexpr (OUT == 0) {
        static_assert(W == 4, "16 bytes");
        float *c = reinterpret_cast<float *>(base) + at;
        if (n >= W) {
            f32x4 x = {v[0], v[1], v[2], v[3]};
            if (p.beta != 0.0f) {
                const f32x4 o = *reinterpret_cast<const dmatile::f32x4_ea *>(c);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(p.beta, o[r], x[r]);
            }
            *reinterpret_cast<dmatile::f32x4_ea *>(c) = x;
        } else {
            for (int r = 0; r < W - 1; ++r)
                if (r < n) c[r] = p.beta != 0.0f ? __builtin_fmaf(p.beta, c[r], v[r]) : v[r];
        }
    } else {
        using V = std::conditional_t<W == 8, u32x4_ea, u32x2_ea>;
        uint16_t *c = reinterpret_cast<uint16_t *>(base) + at;
        if (n >= W) {
            V x;
            if (p.beta != 0.0f) {
                const V o = *reinterpret_cast<const V *>(c);
#pragma unroll
                for (int r = 0; r < W / 2; ++r)
                    x[r] = pack2<OUT>(__builtin_fmaf(p.beta, old(o[r] & 0xffffu), v[2 * r]),
                                      __builtin_fmaf(p.beta, old(o[r] >> 16), v[2 * r + 1]));
            } else {
#pragma unroll
                for (int r = 0; r < W / 2; ++r) x[r] = pack2<OUT>(v[2 * r], v[2 * r + 1]);
            }
            *reinterpret_cast<V *>(c) = x;
        } else {
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                if (r < n) c[r] = uint16_t(bits(p.beta != 0.0f ? __builtin_fmaf(p.beta, old(c[r]), v[r]) : v[r]));
        }
    }
}

// ROWS rows of a wave's tile (16*FN columns) that it staged in LDS, row by
// row: 16-byte chunk q of row r at q ^ (r % 16), so that neither the columns'
// writes nor the rows' reads meet in a bank.  A store covers whole rows of
// the strip.  c: C's element (0, 0) of the tile, which has mrows x ncols
// elements; the strip is at (m, n) of it.
// plain: the tile lies whole within C and beta is 0, so that the rows are
// stored one after another without a look at either (the general way spends
// four times as long on addresses and predicates as on the stores).
template <int OUT, int FN, int ROWS>
__device__ inline void store_strip(const BlockProblem &p, const LDS float *strip, char *c, int m, int mrows,
                                   int n, int ncols, bool plain, int lane) {
    constexpr int W = OUT == 0 ? 4 : 8;          // columns per lane
    constexpr int LANES = FN * 16 / W;           // per row
    constexpr int STEP = 64 / LANES;             // rows per store
    n += W * (lane % LANES);
    float v[ROWS / STEP][W];
#pragma unroll
    for (int i = 0; i < ROWS / STEP; ++i) {
        const int r = i * STEP + lane / LANES;
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
            const int q = (lane % LANES) * (W / 4) + h;
            const f32x4 x = *reinterpret_cast<const LDS f32x4 *>(strip + r * FN * 16 + ((q ^ r) & (FN * 4 - 1)) * 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][4 * h + k] = x[k];
        }
    }
    if (plain) {
        constexpr int ESIZE = OUT == 0 ? 4 : 2;
        char *at = c + ((m + lane / LANES) * p.ldc + n) * ESIZE;
#pragma unroll
        for (int i = 0; i < ROWS / STEP; ++i) {
            if constexpr (OUT == 0) {
                *reinterpret_cast<dmatile::f32x4_ea *>(at) = f32x4{v[i][0], v[i][1], v[i][2], v[i][3]};
            } else {
                u32x4_ea w;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack2<OUT>(v[i][2 * k], v[i][2 * k + 1]);
                *reinterpret_cast<u32x4_ea *>(at) = w;
            }
            at += STEP * p.ldc * ESIZE;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < ROWS / STEP; ++i) {
        const int r = m + i * STEP + lane / LANES;
        if (r < mrows && n < ncols) store_columns<OUT, W>(p, c, r * p.ldc + n, v[i], ncols - n);
    }
}

// The output tile of workgroup wg, as tile_of numbers them, in 32 bits (the
// grid has fewer than 2^31 tiles), and its quarter; false past the last tile
// of the part, of `rows` tile rows.
__device__ inline bool coordinates(const TileGrid &g, TilePart part, uint32_t rows, uint32_t wg, uint32_t &batch,
                                   uint32_t &tm, uint32_t &tn, uint32_t &quarter) {
    const uint32_t cols = uint32_t(g.tiles_n), group = uint32_t(g.group_m);
    // The dispatcher deals workgroups to the 8 dies in turn: those of one die
    // take neighbouring tiles, of the whole grid or (g.xcds 0) of every slice
    // alike: slices of unlike lengths would keep the dies busy for unlike
    // times.
    const uint32_t slice = rows * cols, of = g.xcds == 0 ? wg / slice : 0;
    uint32_t total = g.xcds == 0 ? slice : slice * uint32_t(g.batch), before = 0;
    if (part == TilePart::Rest) {
        before = total - total % ROUND;
        total = 4 * (total % ROUND);
    } else if (part == TilePart::Rounds) {
        total -= total % ROUND;
    }
    const uint32_t q = total / 8, odd = total % 8;
    wg -= of * slice;
    const uint32_t x = wg % 8;
    uint32_t id = (x < odd ? x * (q + 1) : odd * (q + 1) + (x - odd) * q) + wg / 8;
    if (wg / 8 >= q + (x < odd ? 1 : 0)) return false;
    quarter = id % 4;
    if (part == TilePart::Rest) id = before + id / 4;
    batch = g.xcds == 0 ? of : id / slice;
    const uint32_t local = g.xcds == 0 ? id : id - batch * slice;
    const uint32_t n = local / (group * cols), first = n * group;
    const uint32_t high = rows - first < group ? rows - first : group;  // the last group may be short
    const uint32_t r = local - n * (group * cols);
    tn = r / high;
    tm = first + (r - tn * high);
    return true;
}

// One workgroup per BM x BN tile, WAVES_M x WAVES_N waves of FM x FN blocks.
//
// Two LDS stages of 128 k, filled by direct loads.  B's fragments stay in
// registers for a stage, A's rotate through two; the last row's instructions
// run after the barrier that ends a stage, while the next stage's first
// fragments are read, and the freed stage is refilled there.  A block's sum
// is added to its accumulators LAG instructions after it was started, so that
// neither pipe waits for the other.
// TEAMS 2: two such groups of waves, each with its own stages, take the blocks
// of k in turn; at the end each adds the other's sums of half of the rows to
// its own and stores them.
//
// Why 256 x 256 of eight waves of 128 x 64: a stage is 64 KiB read from the
// second-level cache and 192 KiB from LDS for 2^23 multiply-adds, half of what
// 128 x 128 tiles read (4096^3 62 us, with those 91).  4096 x 4096 by K of 1024
// to 8192, one tile per compute unit, takes 10.7 us and 1.67 per step of k with
// one factor per row, 10.2 and 1.97 with one per value; the matrix instructions
// alone are 0.85 at 2.4 GHz.  On random values the socket's power limit sets
// the clock (2.0 to 2.1 GHz, 2.2 PFLOP/s at 4096^3); on zeros it is 12.7 and
// 1.33, 12.0 and 1.61, of which a quarter goes without the refill.  Of the part
// that K does not change, coordinates and addresses are 1.5, the first stage
// 1.2 to 5, C about 3, the rest the launch.
template <int FA, int FB, bool PER_COLUMN, int WAVES_M, int WAVES_N, int FM, int FN, int TEAMS>
__global__ __launch_bounds__(TEAMS *WAVES_M *WAVES_N * 64) void block_tile_kernel(BlockArgs a) {
    constexpr int WAVES = WAVES_M * WAVES_N;  // of a team
    constexpr int WTM = FM * 16, WTN = FN * 16, BM = WAVES_M * WTM, BN = WAVES_N * WTN;
    static_assert(128 % WTN == 0, "a wave's columns lie in one block of 128");
    static_assert(FM % 2 == 0, "A's fragments alternate between two slots");
    static_assert(TEAMS == 1 || TEAMS == 2, "one adds the other's sums");
    using PA = Panel<BM, WAVES>;
    using PB = Panel<BN, WAVES>;
    constexpr int AT_B = PA::BYTES, AT_S = AT_B + PB::BYTES;  // within a stage
    constexpr int STAGE = AT_S + (BM + BN) * 4;
    constexpr int SLOADS = (BM + BN) / 64;  // scale loads of 64 rows, one per wave or less
    static_assert(SLOADS <= WAVES, "at most one scale load per wave");
    constexpr int LAG = 3;
    __shared__ __attribute__((aligned(1024))) char smem[TEAMS * 2 * STAGE];
    const BlockProblem &p = a.p;
    const int team = TEAMS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (WAVES * 64));
    LDS char *lds = (LDS char *)smem + team * 2 * STAGE;
    const int tid = threadIdx.x - team * WAVES * 64, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;

    // With segments of rows the grid has as many tile rows as there can be: the
    // dies share those that there are.
    static_assert(BM == BN && (BM == 128 || BM == 256), "tiles of 256, or quarters of them");
    const bool quarters = BM == 128 && p.part == TilePart::Rest;
    const int side = quarters ? 2 * BM : BM;
    uint32_t te, tm, tn, quarter;
    int64_t e, m0, m_end = p.M, k_lo = 0, k_hi = p.K;
    if (p.segments == Segments::Rows) {
        const SegmentTiles first(p, 0, BM, lane);
        const uint32_t rows = tile_rows(p, first, a.grid.tiles_m, BM, lane);
        if (!coordinates(a.grid, TilePart::All, rows, blockIdx.x, te, tm, tn, quarter)) return;
        if (!find_segment(p, first, uniform(tm), BM, lane, e, m0, m_end)) return;
    } else {
        if (!coordinates(a.grid, p.part, uint32_t(a.grid.tiles_m), blockIdx.x, te, tm, tn, quarter)) return;
        e = uniform(te);
        m0 = uniform(tm) * side;
    }
    int64_t n0 = uniform(tn) * side;
    if (quarters) {
        m0 += uniform(quarter >> 1) * BM;
        n0 += uniform(quarter & 1) * BN;
        if (m0 >= p.M || n0 >= p.N) return;
    }
    if (p.segments == Segments::Contracted) {
        if (p.batch <= 64) e = by_length(p, e, lane);
        segment_of(p.offsets, e, p.K, k_lo, k_hi);
        k_lo = uniform(k_lo);
        k_hi = uniform(k_hi);
        k_lo = k_hi > k_lo ? k_lo & ~int64_t(127) : k_hi;  // (an empty segment may start anywhere)
    }
    const int K = int(uniform(k_hi - k_lo));  // at most ld < 2^22
    const int64_t ea = p.segments == Segments::None ? e : 0;
    const int64_t eb = p.segments == Segments::Contracted ? 0 : e;
    const int64_t ec = p.segments == Segments::Rows ? 0 : e;
    const int mrows = int(m_end - m0 < BM ? m_end - m0 : BM), nrows = int(p.N - n0 < BN ? p.N - n0 : BN);

    PA pa;
    PB pb;
    pa.init(p.a.x + ea * p.a.stride, p.a.ld, m0, mrows, k_lo, K, wave, lane);
    pb.init(p.b.x + eb * p.b.stride, p.b.ld, n0, nrows, k_lo, K, wave, lane);

    // Scales: wave w loads those of 64 panel rows (A's first, then B's), one
    // per lane; panel row r of the tile has the scale (r0 + r) >> shift of its
    // operand's row of scales.
    const bool s_on_a = wave < BM / 64;
    const int s_row = (s_on_a ? wave : wave - BM / 64) * 64 + lane;
    const int s_shift = s_on_a ? p.a.shift : p.b.shift;
    const int64_t s_r0 = s_on_a ? m0 : n0;
    const int s_rows = s_on_a ? mrows : nrows;
    const int64_t s_first = s_r0 >> s_shift;
    const uint32_t s_voff =
        s_row < s_rows ? uint32_t((((s_r0 + s_row) >> s_shift) - s_first) * 4) : OOB;
    const int64_t s_ld = (s_on_a ? p.a.lds : p.b.lds) * 4;
    const int64_t s_base = uniform(
        reinterpret_cast<int64_t>((s_on_a ? p.a.s + ea * p.a.sstride : p.b.s + eb * p.b.sstride) + s_first) +
        (k_lo >> 7) * s_ld);
    const uint32_t s_bytes =
        uint32_t(uniform((((s_r0 + s_rows - 1) >> s_shift) - s_first + 1) * 4));

    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    const int blocks = (K + 127) / 128, steps = (blocks + TEAMS - 1) / TEAMS;
    // The stage that is being loaded.  Its loads (A's, B's, the scales) go out
    // a few at a time between matrix instructions: all at once they fill the
    // memory pipe's queue and hold up the matrix pipe.
    constexpr int LOADS = PA::PER_WAVE + PB::PER_WAVE + 1, EARLY = FN, LOADS_PER_ROW = 2;
    struct Loading {
        u32x4 a, b, s;
        int kleft;
    };
    auto loading = [&](int step) {  // past the last block: loads that read nothing and store zeros
        const int s = step * TEAMS + team;
        const bool live = s < blocks;
        const int kleft = K - 128 * s;
        return Loading{pa.stage(s, live), pb.stage(s, live),
                       dma::raw_buffer(static_cast<uint64_t>(s_base + s * s_ld), live ? s_bytes : 0u),
                       kleft < 128 ? kleft : 128};
    };
    auto load = [&](const Loading &l, int buf, int q) {
        const uint32_t at = lds0 + buf * STAGE;
        if (q < PA::PER_WAVE) pa.load(l.a, at, q, l.kleft, wave, lane);
        else if (q < LOADS - 1) pb.load(l.b, at + AT_B, q - PA::PER_WAVE, l.kleft, wave, lane);
        else if (SLOADS == WAVES || wave < SLOADS) direct_load4(l.s, at + AT_S + wave * 256, s_voff);
    };
    // The chunk that holds the end of K, in the stage of buffer buf: its bytes
    // from K on are not the operand's.  (Of the teams the one that has that block.)
    auto clear_tail = [&](int buf) {
        const int kleft = K & 127, c = kleft >> 4;
        const bool mine = TEAMS == 1 || (steps - 1) * TEAMS + team == blocks - 1;
        for (int r = mine ? tid : BM + BN; r < BM + BN; r += WAVES * 64) {
            const int rr = r < BM ? r : r - BM;
            LDS char *chunk = lds + buf * STAGE + r * 128 + ((c ^ swz(rr)) << 4);
            for (int b = kleft & 15; b < 16; ++b) chunk[b] = 0;
        }
        __syncthreads();
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int at = lane_chunk(lane);
    i32x8 fb[FN], fa[2];
    f32x4 part[LAG + 1];
    float sa[FM];
    f32x4 sb[PER_COLUMN ? FN : 1];  // one factor, in [0][0], when the columns share a scale
    auto read_a = [&](int buf, int i) {
        fa[i & 1] = frag(lds + buf * STAGE, wm * WTM + i * 16, at);
    };
    auto read_b = [&](int buf, int j) {
        fb[j] = frag(lds + buf * STAGE + AT_B, wn * WTN + j * 16, at);
    };
    float nsa[FM], nfactor = 0.0f;  // the next stage's, as stored
    auto read_scales = [&](int buf) {
        const LDS float *s = reinterpret_cast<const LDS float *>(lds + buf * STAGE + AT_S);
#pragma unroll
        for (int i = 0; i < FM; ++i) nsa[i] = s[wm * WTM + i * 16 + (lane & 15)];
        if (!PER_COLUMN) nfactor = s[BM + wn * WTN];
    };
    auto take_scales = [&](int buf) {
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = PER_COLUMN ? nsa[i] : nsa[i] * nfactor;
        if (PER_COLUMN) {  // read here: there are no registers for two stages' columns
            const LDS float *s = reinterpret_cast<const LDS float *>(lds + buf * STAGE + AT_S);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sb[j] = *reinterpret_cast<const LDS f32x4 *>(s + BM + wn * WTN + j * 16 + 4 * (lane >> 4));
        }
    };
    auto start = [&](int n) {
        part[n % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            fb[n % FN], fa[(n / FN) & 1], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, UNIT, 0, UNIT);
    };
    // The empty statement takes the sums as operands: without it the compiler
    // moves a whole stage's instructions past the barrier, to where its sums
    // are next read, and keeps every fragment of the stage until there.
    auto add = [&](int n) {
        const int i = n / FN, j = n % FN;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float f = PER_COLUMN ? sa[i] * sb[PER_COLUMN ? j : 0][r] : sa[i];
            acc[i][j][r] = __builtin_fmaf(part[n % (LAG + 1)][r], f, acc[i][j][r]);
        }
        asm volatile("" : "+v"(acc[i][j]));
    };
    // Rows 0 .. FM - 2 of stage s, in buffer buf, with the next stage's loads from EARLY on.
    auto rows = [&](int s, int buf) {
        const Loading l = loading(s + 1);
        take_scales(buf);
#pragma unroll
        for (int n = 0; n < (FM - 1) * FN; ++n) {
            if (n % FN == 0) {
                read_a(buf, n / FN + 1);
#pragma unroll
                for (int q = EARLY + n / FN * LOADS_PER_ROW; q < EARLY + (n / FN + 1) * LOADS_PER_ROW; ++q)
                    if (q < LOADS) load(l, buf ^ 1, q);
            }
            start(n);
            if (n >= LAG) add(n - LAG);
            if (n % FN == FN - 1) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (j < 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, PER_COLUMN ? 8 : 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    static_assert(EARLY + (FM - 1) * LOADS_PER_ROW >= LOADS, "every load has its place");
    auto finish = [&]() {
#pragma unroll
        for (int n = FM * FN - LAG; n < FM * FN; ++n) add(n);
    };

    if (steps > 0) {
        const Loading l0 = loading(0), l1 = loading(1);
#pragma unroll
        for (int q = 0; q < LOADS; ++q) load(l0, 0, q);
#pragma unroll
        for (int q = 0; q < EARLY; ++q) load(l1, 1, q);
        wait_vmcnt<EARLY>();
        __syncthreads();
        if (steps == 1 && (K & 15) != 0) clear_tail(0);
#pragma unroll
        for (int j = 0; j < FN; ++j) read_b(0, j);
        read_a(0, 0);
        read_scales(0);
    }
    int buf = 0;
    for (int s = 0; s + 1 < steps; ++s) {
        rows(s, buf);
        wait_vmcnt<0>();
        dma::wait_lgkmcnt0();
        __syncthreads();
        if (s + 2 == steps && (K & 15) != 0) clear_tail(buf ^ 1);
        read_a(buf ^ 1, 0);
        read_scales(buf ^ 1);
        const Loading l = loading(s + 2);
#pragma unroll
        for (int n = (FM - 1) * FN; n < FM * FN; ++n) {
            start(n);
            read_b(buf ^ 1, n % FN);
            load(l, buf, n % FN);
            add(n - LAG);
        }
        finish();
        buf ^= 1;
    }
    if (steps > 0) {
        rows(steps - 1, buf);
#pragma unroll
        for (int n = (FM - 1) * FN; n < FM * FN; ++n) {
            start(n);
            add(n - LAG);
        }
        finish();
        // the loads past the last stage have put zeros into the buffer that C goes through
        wait_vmcnt<0>();
        __syncthreads();
    }

    // The buffer after the last stage's: nothing reads or fills it any more.
    constexpr int PAIR = 2;  // strips of 16 rows that leave together
    static_assert(WAVES * PAIR * 16 * WTN * 4 <= STAGE, "a pair of strips per wave fits a stage");
    LDS float *strip = reinterpret_cast<LDS float *>(lds + (buf ^ 1) * STAGE) + wave * PAIR * 16 * WTN;
    if constexpr (TEAMS == 2) {
        constexpr int HALF = FM / 2;
        LDS f32x4 *sums = reinterpret_cast<LDS f32x4 *>(lds + buf * STAGE) + tid;  // this team's of the other's rows
        LDS f32x4 *others = reinterpret_cast<LDS f32x4 *>((LDS char *)smem + (team ^ 1) * 2 * STAGE + buf * STAGE) + tid;
        static_assert(HALF * FN * WAVES * 64 * 16 <= STAGE, "half of the sums fit a stage");
#pragma unroll
        for (int i = 0; i < HALF; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) sums[(i * FN + j) * WAVES * 64] = team == 0 ? acc[HALF + i][j] : acc[i][j];
        dma::wait_lgkmcnt0();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < HALF; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = (team == 0 ? acc[i][j] : acc[HALF + i][j]) + others[(i * FN + j) * WAVES * 64];
    }
    constexpr int ROWS = FM / TEAMS;  // of blocks that this team stores
    // An empty segment has no terms: beta * C, whatever alpha is.  (Asking for K
    // here in every launch costs 4096^3 0.6 of 62 us; elsewhere the host sets alpha.)
    const float alpha = p.segments == Segments::Contracted && steps == 0 ? 0.0f : p.alpha;
    const bool plain = mrows == BM && nrows == BN && p.beta == 0.0f;
    char *c = static_cast<char *>(p.C) + (ec * p.sC + m0 * p.ldc + n0) * (p.out == 0 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < ROWS; i += PAIR) {
        const int r = lane & 15;
#pragma unroll
        for (int k = 0; k < PAIR; ++k)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int q = j * 4 + (lane >> 4);
                *reinterpret_cast<LDS f32x4 *>(strip + (k * 16 + r) * WTN + ((q ^ r) & (FN * 4 - 1)) * 4) =
                    alpha * acc[i + k][j];
            }
        const int m = wm * WTM + (team * ROWS + i) * 16, n = wn * WTN;
        if (p.out == 0) store_strip<0, FN, PAIR * 16>(p, strip, c, m, mrows, n, nrows, plain, lane);
        else if (p.out == 1) store_strip<1, FN, PAIR * 16>(p, strip, c, m, mrows, n, nrows, plain, lane);
        else store_strip<2, FN, PAIR * 16>(p, strip, c, m, mrows, n, nrows, plain, lane);
    }
}

// ---- few rows

// The first `valid` (any integer) of a chunk's 16 bytes, the others 0.
__device__ inline u32x4 first_bytes(u32x4 v, int valid) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int n = valid - 4 * w;
        v[w] = n >= 4 ? v[w] : n <= 0 ? 0u : v[w] & ((1u << (8 * n)) - 1);
    }
    return v;
}

constexpr int FEW_WAVES = 8;

// For few rows of C: 16 columns by 16*FM rows per workgroup, B and A read
// straight into registers, the blocks of K dealt to the waves in turn, UNROLL
// of them in flight per wave.  The waves' sums are added in order through
// LDS.  Bound by reading B: with 16 columns a chip-wide launch needs only 4096
// columns, and 128-byte pieces of 16 rows keep whole lines.  128 rows dealt at
// random to 64 experts of 2048 x 4096, about 55 of which have any, take 95 to
// 104 us, 4.5 to 4.9 TB/s; 16x4096x4096 7.8 us, of which 3.4 are reading.
template <int FA, int FB, bool PER_COLUMN, int FM, int UNROLL>
__global__ __launch_bounds__(FEW_WAVES * 64) void block_few_kernel(BlockArgs a) {
    __shared__ f32x4 sums[FEW_WAVES][FM * 64];
    const BlockProblem &p = a.p;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (the parts of the same columns, which read the same B, follow each other at a distance)
    const uint32_t groups = uint32_t(p.batch * a.grid.tiles_n), part = blockIdx.x / groups, group = blockIdx.x - part * groups;
    const int64_t e = uniform(group / uint32_t(a.grid.tiles_n));
    const int64_t n0 = uniform(int64_t(group) - e * a.grid.tiles_n) * 16;
    const bool rows_cut = p.segments == Segments::Rows;
    int64_t m_lo = 0, m_hi = p.M;
    if (rows_cut) {
        segment_of(p.offsets, e, p.M, m_lo, m_hi);
        m_lo = uniform(m_lo);
        m_hi = uniform(m_hi);
    }
    const int64_t ea = rows_cut ? 0 : e, ec = rows_cut ? 0 : e;
    const int64_t kbs = (p.K + 127) / 128;
    const int c = lane >> 4;  // this lane's chunks of a block: c and 4 + c
    const int64_t n = n0 + (lane & 15) < p.N ? n0 + (lane & 15) : p.N - 1;  // rows past the end read the last
    const uint8_t *b = p.b.x + e * p.b.stride + n * p.b.ld;
    const float *sb = p.b.s + e * p.b.sstride;
    auto chunk = [&](const uint8_t *row, int64_t kb, int which) {
        // a chunk past the end of K reads the block's first instead, and is cleared below
        const int at = 16 * (c + 4 * which);
        return *reinterpret_cast<const u32x4 *>(row + 128 * kb + (128 * kb + at < p.K ? at : 0));
    };
    auto joined = [&](u32x4 lo, u32x4 hi, int64_t kb) {
        if (128 * kb + 128 > p.K) {
            lo = first_bytes(lo, int(p.K - 128 * kb) - 16 * c);
            hi = first_bytes(hi, int(p.K - 128 * kb) - 16 * (c + 4));
        }
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                     int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };
    const int64_t m_first = m_lo + int64_t(part) * 16 * FM;
    for (int64_t m0 = m_first; m0 < m_hi; m0 += a.grid.tiles_m * 16 * FM) {
        const uint8_t *ar[FM];
        int64_t am[FM];
        f32x4 acc[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int64_t m = m0 + 16 * i + (lane & 15);
            am[i] = m < m_hi ? m : m_hi - 1;
            ar[i] = p.a.x + ea * p.a.stride + am[i] * p.a.ld;
            acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int64_t k0 = wave; k0 < kbs; k0 += FEW_WAVES * UNROLL) {
            u32x4 bv[UNROLL][2], av[UNROLL][FM][2];
            float sa[UNROLL][FM];
            f32x4 sv[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t kb = k0 + u * FEW_WAVES < kbs ? k0 + u * FEW_WAVES : kbs - 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) bv[u][h] = chunk(b, kb, h);
                if (PER_COLUMN) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int64_t nr = n0 + 4 * c + r;
                        sv[u][r] = sb[kb * p.b.lds + (nr < p.N ? nr : p.N - 1)];
                    }
                } else {
                    sv[u][0] = sb[kb * p.b.lds + (n0 >> 7)];
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) av[u][i][h] = chunk(ar[i], kb, h);
                    sa[u][i] = p.a.s[ea * p.a.sstride + kb * p.a.lds + (am[i] >> p.a.shift)];
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t kb = k0 + u * FEW_WAVES;
                if (kb >= kbs) break;
                const i32x8 fb = joined(bv[u][0], bv[u][1], kb);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fb, joined(av[u][i][0], av[u][i][1], kb), f32x4{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, UNIT,
                        0, UNIT);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][r] = __builtin_fmaf(part[r], sa[u][i] * sv[u][PER_COLUMN ? r : 0], acc[i][r]);
                }
            }
        }
        if (m0 > m_first) __syncthreads();  // the last rows' sums have been read
#pragma unroll
        for (int i = 0; i < FM; ++i) sums[wave][i * 64 + lane] = acc[i];
        __syncthreads();
        if (tid < FM * 64) {
            f32x4 v = sums[0][tid];
#pragma unroll
            for (int w = 1; w < FEW_WAVES; ++w) v += sums[w][tid];
            const int64_t m = m0 + 16 * (tid >> 6) + (tid & 15), col = n0 + 4 * (tid >> 4 & 3);
            if (m < m_hi && col < p.N) {
                const int64_t at = ec * p.sC + (p.c_turned ? col * p.ldc + m : m * p.ldc + col);
                const int left = p.N - col < 4 ? int(p.N - col) : 4;
                v *= p.alpha;
                const float x[4] = {v[0], v[1], v[2], v[3]};
                auto store = [&](int64_t to, const float *y, int n) {
                    if (p.out == 0) store_columns<0, 4>(p, static_cast<char *>(p.C), to, y, n);
                    else if (p.out == 1) store_columns<1, 4>(p, static_cast<char *>(p.C), to, y, n);
                    else store_columns<2, 4>(p, static_cast<char *>(p.C), to, y, n);
                };
                if (!p.c_turned) {
                    store(at, x, left);
                } else {
                    for (int r = 0; r < left; ++r) store(at + r * p.ldc, x + r, 1);
                }
            }
        }
    }
}

// The rows of C that share a B: all of them, or about a busy expert's.
int64_t rows_of(const BlockProblem &p) {
    return p.segments == Segments::Rows ? 2 * ((p.M + p.batch - 1) / p.batch) : p.M;
}

template <int FA, int FB, bool PER_COLUMN, int FM, int UNROLL>
hipError_t few_go(const BlockProblem &p, hipStream_t stream) {
    BlockArgs a{};
    a.p = p;
    a.grid.tiles_n = (p.N + 15) / 16;
    a.grid.tiles_m = (rows_of(p) + 16 * FM - 1) / (16 * FM);  // (an expert with more rows takes several turns)
    if (launch_over(double(a.grid.tiles_n) * a.grid.tiles_m * p.batch, FEW_WAVES * 64)) return hipErrorInvalidConfiguration;
    const int64_t count = a.grid.tiles_n * a.grid.tiles_m * p.batch;
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&block_few_kernel<FA, FB, PER_COLUMN, FM, UNROLL>),
                           dim3(static_cast<unsigned>(count)), dim3(FEW_WAVES * 64), args, 0, stream);
}

template <int FA, int FB, bool PER_COLUMN, int WM, int WN, int FM, int FN, int TEAMS>
hipError_t tile_go(const BlockProblem &p, hipStream_t stream) {
    constexpr int BM = WM * FM * 16;  // tiles are square
    BlockArgs a{};
    a.p = p;
    const int64_t side = p.part == TilePart::Rest ? 256 : BM;
    int64_t tiles_m = (p.M + side - 1) / side;
    if (p.segments == Segments::Rows) {  // every segment that is not empty starts a tile
        const int64_t more = p.batch < p.M ? p.batch : p.M;
        tiles_m = p.M / side + more < p.M ? p.M / side + more : p.M;
    }
    a.grid = TileGrid{tiles_m, (p.N + side - 1) / side, p.segments == Segments::Rows ? 1 : p.batch, 8,
                      p.segments == Segments::Contracted ? 0 : 8};
    // (also of the quarters' four times `rest`, which is below ROUND)
    if (launch_over(double(a.grid.tiles_m) * a.grid.tiles_n * a.grid.batch, TEAMS * WM * WN * 64))
        return hipErrorInvalidConfiguration;
    void *args[] = {&a};
    const int64_t rest = p.part == TilePart::All ? 0 : a.grid.count() % ROUND;
    const int64_t count = p.part == TilePart::Rest ? 4 * rest : a.grid.count() - rest;
    return hipLaunchKernel(
        reinterpret_cast<const void *>(&block_tile_kernel<FA, FB, PER_COLUMN, WM, WN, FM, FN, TEAMS>),
        dim3(static_cast<unsigned>(count)), dim3(TEAMS * WM * WN * 64), args, 0, stream);
}

template <int FA, int FB, bool PER_COLUMN>
hipError_t tile_size(BlockKernel k, const BlockProblem &p, hipStream_t stream) {
    if (k == BlockKernel::Few16) return few_go<FA, FB, PER_COLUMN, 1, 4>(p, stream);
    if (k == BlockKernel::Few32) return few_go<FA, FB, PER_COLUMN, 2, 4>(p, stream);
    if (k == BlockKernel::Few64) return few_go<FA, FB, PER_COLUMN, 4, 2>(p, stream);
    if (k == BlockKernel::Tile256) return tile_go<FA, FB, PER_COLUMN, 2, 4, 8, 4, 1>(p, stream);
    if (k == BlockKernel::Tile128) return tile_go<FA, FB, PER_COLUMN, 2, 2, 4, 4, 1>(p, stream);
    return tile_go<FA, FB, PER_COLUMN, 2, 2, 4, 4, 2>(p, stream);
}

}  // namespace

#define LIBGEMM_BLOCK_FORMATS(part, FA, FB)                                               \
    template <>                                                                           \
    hipError_t block_tile_formats<FA, FB>(BlockKernel k, const BlockProblem &p,           \
                                          hipStream_t stream) {                           \
        return p.b.shift == 0 ? tile_size<FA, FB, true>(k, p, stream)                     \
                              : tile_size<FA, FB, false>(k, p, stream);                   \
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
namespace {

// Tiles of `side` x `side` of a problem.  With segments of rows an estimate
// for lengths that differ by half: one per expert where they are short, else
// half a tile more for each.
int64_t tiles_of(const BlockProblem &p, int64_t M, int64_t N, int64_t side) {
    const int64_t cols = (N + side - 1) / side;
    if (p.segments != Segments::Rows) return (M + side - 1) / side * cols * p.batch;
    const double n = double(p.batch < M ? p.batch : M), rows = double(M) / side + 0.5 * n;
    const double tiles = (4.0 * M <= side * n ? n : rows > 1.06 * n ? rows : 1.06 * n) * cols;
    return int64_t(tiles < 1e15 ? tiles : 1e15);
}
int64_t rounds_of(int64_t tiles, int64_t at_once) { return (tiles + at_once - 1) / at_once; }

// Rows or columns past the last whole 256 that are few enough for the few-rows kernel.
int64_t edge_of(int64_t n) { return n > 256 && n % 256 <= 64 ? n % 256 : 0; }

// Rows and columns of C that leave the 256 x 256 tiles and run by themselves:
// a tile that holds few of them takes as long as a whole one, so where they
// cost a wave of 256 tiles (13 us and more) the few-rows kernel is cheaper
// (about 5 us for each of the two edges).
void edges_of(const BlockProblem &p, int64_t &rows, int64_t &cols) {
    rows = cols = 0;
    if (p.segments != Segments::None) return;
    auto waves = [&](int64_t M, int64_t N) { return rounds_of(tiles_of(p, M, N, 256), 256); };
    // (an edge that one launch does not take stays in the tiles)
    auto edge = [&](int64_t n, int64_t other) {
        return launch_over(double((other + 15) / 16) * p.batch, FEW_WAVES * 64) ? 0 : edge_of(n);
    };
    const int64_t er = edge(p.M, p.N), ec = edge(p.N, p.M), whole = waves(p.M, p.N);
    if (waves(p.M, p.N - ec) < whole) cols = ec;
    else if (waves(p.M - er, p.N) < whole) rows = er;
    else if (waves(p.M - er, p.N - ec) < whole) rows = er, cols = ec;
}

hipError_t launch_formats(BlockKernel k, const BlockProblem &p, hipStream_t stream) {
    if (p.a.e5m2) return p.b.e5m2 ? block_tile_formats<1, 1>(k, p, stream) : block_tile_formats<1, 0>(k, p, stream);
    return p.b.e5m2 ? block_tile_formats<0, 1>(k, p, stream) : block_tile_formats<0, 0>(k, p, stream);
}

BlockKernel few_for(int64_t rows) {
    return rows <= 16 ? BlockKernel::Few16 : rows <= 32 ? BlockKernel::Few32 : BlockKernel::Few64;
}

BlockOperand from_row(BlockOperand o, int64_t row) {  // row: a multiple of 128
    o.x += row * o.ld;
    o.s += row >> o.shift;
    return o;
}

}  // namespace

// The kernel for a problem, by what was measured (us).
// Few rows.  The few-rows kernel reads B at the rate of memory, but again for
// each of its parts of 16, 32 or 64 rows, and its workgroups hold a compute
// unit each: it wants the lowest parts that all run at once.  Against 128 x
// 128 tiles of two teams: 64x4096x4096 14 and 19, 256x512x5376 16 and 23,
// 64x8192x4096 25 and 22, 128x4096x4096 25 and 19.  At 16 rows it gains with
// more workgroups as well, where they are long: 16x12288x4096 16 and 22,
// 16x16384x4096 21 and 23, 16x32768x2048 33 and 21; at 8, which are mostly
// waiting for memory, always (64 experts of 2048x4096: 4 rows each 111 and
// 142, 8 rows each 127 and 133, 12 rows each 157 and 134).
// Tiles.  128 x 128 of two teams hold a compute unit each, as 256 x 256 do;
// of one team two share one.  Teams, two and one: 512x4096x4096 23 and 33,
// 1536x1536x7552 39 and 54; where there are more than 256 tiles
// 512x16384x4096 46 and 43.  A round of 256 tiles of 256 x 256 takes 5/4 of the
// time of one of 512 tiles of 128 x 128: of K = 4096, 128 tiles of 256 50 where
// 512 of 128 take 45, 192 of 256 51 where 768 of 128 take 69; 64 experts of
// 2048x4096 at 64 rows each 143 and 177, of 1024x2048 at 128 rows each 57 and 44.
// Up to a quarter of a round past whole rounds runs in quarters of tiles, by
// two teams, after them: 4608x4096x4096 102 and 84, 9216x4096x8192 301 and 267,
// 4608x4096x1024 34.6 and 32.1; half a round would not gain (6144x4096x4096 103
// and 110), nor would most segments of rows, whose rest the host does not know.
BlockKernel block_choose(const BlockProblem &p, bool general, bool split) {
    if (p.M == 0 || p.N == 0 || p.batch == 0) return BlockKernel::None;
    if (general) return BlockKernel::Tile256;
    if (split && p.segments != Segments::Contracted) {
        const int64_t rows = rows_of(p);
        const double groups = double(p.batch) * ((p.N + 15) / 16);  // of 16 columns, a workgroup each
        for (int64_t height : {16, 32, 64})
            if (groups * ((rows + height - 1) / height) <= 256) return few_for(height);
        if ((rows <= 16 && groups <= (p.K >= 4096 ? 1024 : 512)) || (rows <= 8 && p.K >= 4096)) return BlockKernel::Few16;
        if (rows <= 32 && groups <= 512) return BlockKernel::Few32;
    }
    const int64_t tiles = tiles_of(p, p.M, p.N, 128);
    if (split && tiles <= 256 && p.K > 128) return BlockKernel::Tile128Two;
    int64_t er = 0, ec = 0;
    if (split) edges_of(p, er, ec);
    const int64_t large = tiles_of(p, p.M, p.N, 256), rest = large % ROUND;
    const int64_t whole = 10 * rounds_of(tiles_of(p, p.M - er, p.N - ec, 256), 256) + 2 * (er > 0) + 2 * (ec > 0);
    const int64_t small = 8 * rounds_of(tiles, 512), split_off = 10 * (large / ROUND) + 7;
    if (split && p.segments == Segments::None && p.K >= 1024 && rest > 0 && rest <= ROUND / 4 && large > ROUND &&
        split_off < (whole < small ? whole : small))
        return BlockKernel::Tile256Rest;
    if (small < whole) return BlockKernel::Tile128;
    return er + ec > 0 ? BlockKernel::Tile256Edge : BlockKernel::Tile256;
}

const char *block_kernel_name(BlockKernel k) {
    switch (k) {
    case BlockKernel::None: return "";
    case BlockKernel::Tile256: return "f8block_mfma_256";
    case BlockKernel::Tile256Edge: return "f8block_mfma_256_edge";
    case BlockKernel::Tile256Rest: return "f8block_mfma_256_rest";
    case BlockKernel::Few16: return "f8block_few_16";
    case BlockKernel::Few32: return "f8block_few_32";
    case BlockKernel::Few64: return "f8block_few_64";
    case BlockKernel::Tile128: return "f8block_mfma_128";
    case BlockKernel::Tile128Two: return "f8block_mfma_128_two";
    }
    return "";
}

hipError_t launch_block(BlockKernel k, const BlockProblem &p, hipStream_t stream) {
    if (k == BlockKernel::None) return hipSuccess;
    BlockProblem q = p;
    if (k == BlockKernel::Tile256Rest) {
        q.part = TilePart::Rounds;
        const hipError_t e = launch_formats(BlockKernel::Tile256, q, stream);
        if (e != hipSuccess) return e;
        q.part = TilePart::Rest;
        return launch_formats(BlockKernel::Tile128Two, q, stream);
    }
    if (k != BlockKernel::Tile256Edge) return launch_formats(k, p, stream);
    int64_t er, ec;
    edges_of(p, er, ec);
    const int64_t M = p.M - er, N = p.N - ec, esize = p.out == 0 ? 4 : 2;
    q.M = M;
    q.N = N;
    hipError_t e = launch_formats(BlockKernel::Tile256, q, stream);
    if (e == hipSuccess && er > 0) {  // the last rows, of the tiles' columns
        q.M = er;
        if (p.K > 0) q.a = from_row(p.a, M);
        q.C = static_cast<char *>(p.C) + M * p.ldc * esize;
        e = launch_formats(few_for(er), q, stream);
    }
    if (e == hipSuccess && ec > 0) {  // the last columns, of all rows: as rows of the transpose
        q = p;
        q.M = ec;
        q.N = p.M;
        q.a = p.K > 0 ? from_row(p.b, N) : p.b;
        q.b = p.a;
        q.C = static_cast<char *>(p.C) + N * esize;
        q.c_turned = true;
        e = launch_formats(few_for(ec), q, stream);
    }
    return e;
}
#endif

}  // namespace libgemm
