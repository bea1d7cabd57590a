// The tile pipeline of the layers' 16-bit kernels (linear.hip and
// orthogonalize.hip): a BM x BN tile of op(A) * op(B) on the CDNA4 matrix
// cores, into fp32 accumulators, and a walk over the finished tile in whole
// pieces of rows for an epilogue.
//
// A ring of LDS stages of 64 k, refilled behind one barrier per stage, and
// fragments double-buffered in registers, over panels of any number of rows.  DIRECT panels are filled by direct
// global -> LDS loads and need whole 16-byte chunks; the others go through
// registers and take any alignment and extent.  Both leave the same layout:
//   K-contiguous panel: [rows][64 k], 128 bytes per row, 16-byte chunk c of
//     row r at c ^ ((r ^ (r >> 3)) & 7);
//   row-contiguous panel: [64 k][rows], chunk c of k row r XORed so that the
//     k rows one transposing read touches fall in different 64-byte banks.
// Addresses inside a tile are 32-bit offsets from the tile's own base, so an
// operand may be of any size.
#pragma once

#include <type_traits>

#include "dma_tile.hpp"

namespace libgemm {
namespace tile16 {

using namespace dmatile;

struct BF16 {};
struct F16 {};

template <class T>
__device__ inline f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c);
template <>
__device__ inline f32x16 mfma32<BF16>(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ inline f32x16 mfma32<F16>(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 16-bit values to fp32 and back (to nearest even).
template <class T>
__device__ inline float decode(uint32_t b);
template <>
__device__ inline float decode<BF16>(uint32_t b) { return __builtin_bit_cast(float, b << 16); }
template <>
__device__ inline float decode<F16>(uint32_t b) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
}
template <class T>
__device__ inline uint32_t encode(float x);
template <>
__device__ inline uint32_t encode<BF16>(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
template <>
__device__ inline uint32_t encode<F16>(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// n (1 .. 8) consecutive values from p, at element alignment; the others 0.
template <class T>
__device__ inline void load8(const uint16_t *p, int n, float (&x)[8]) {
    if (n == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4_ea *>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = decode<T>(v[e / 2] >> (16 * (e % 2)) & 0xffffu);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? decode<T>(p[e]) : 0.0f;
    }
}
__device__ inline void load8f(const float *p, int n, float (&x)[8]) {
    if (n == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = *reinterpret_cast<const f32x4_ea *>(p + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * h + e] = v[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? p[e] : 0.0f;
    }
}
template <class T>
__device__ inline u32x4 pack8(const float (&x)[8]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = encode<T>(x[2 * e]) | (encode<T>(x[2 * e + 1]) << 16);
    return w;
}
template <class T>
__device__ inline void store8(uint16_t *p, int n, const float (&x)[8]) {
    const u32x4 w = pack8<T>(x);
    if (n == 8) {
        *reinterpret_cast<u32x4_ea *>(p) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2)));
    }
}
__device__ inline void store8f(float *p, int n, const float (&x)[8]) {
    if (n == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = {x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
            *reinterpret_cast<f32x4_ea *>(p + 4 * h) = v;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = x[e];
    }
}
// In a type known only when running: T where `same`, else fp32.
template <class T>
__device__ inline void store8_as(void *p, int64_t at, bool same, int n, const float (&x)[8]) {
    if (same) store8<T>(static_cast<uint16_t *>(p) + at, n, x);
    else store8f(static_cast<float *>(p) + at, n, x);
}

// The same loads, kept as they come until they are needed.
struct Raw8 {
    u32x4 v;
    __device__ void load(const uint16_t *p, int n) {
        if (n == 8) {
            v = *reinterpret_cast<const u32x4_ea *>(p);
        } else {
            v = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) v[e / 2] |= uint32_t(p[e]) << (16 * (e % 2));
        }
    }
    // 16-bit values
    template <class T>
    __device__ void values(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = decode<T>(v[e / 2] >> (16 * (e % 2)) & 0xffffu);
    }
};
// Element `it` of four, without an array in memory.
template <class D>
__device__ inline D pick(const D (&d)[4], int it) {
    D r = d[0];
    constexpr int WORDS = sizeof(D) / 4;
    uint32_t *to = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(&d[i]);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) to[w] = it == i ? from[w] : to[w];
    }
    return r;
}
struct Nothing {
    uint32_t unused;
};

// Leading dimensions (elements) whose tiles' offsets stay below 2^31 bytes:
// 256 rows of a K-contiguous panel, 64 of the other.
constexpr int64_t MOST_LD = int64_t(1) << 21;

// An operand of R rows contracted over K: element (r, k) at p[r*ld + k]
// (K-contiguous) or p[k*ld + r].
struct Operand16 {
    const uint16_t *p;
    int64_t ld, R;
};

template <bool KMAJOR, int ROWS, int WAVES, int BK>
struct Panel {
    static constexpr int CHK = BK / 8;  // chunks per row, K-contiguous
    static constexpr int BYTES = ROWS * BK * 2;
    static constexpr int PER_WAVE = BYTES / 1024 / WAVES;  // 1 KiB pieces per wave per stage
    static constexpr int CHR = ROWS / 8;                   // chunks per k row, row-contiguous
    static_assert(PER_WAVE * WAVES * 1024 == BYTES, "panel split over waves");
    static_assert(KMAJOR || ROWS == 128 || ROWS == 256, "the layout's swizzle");
    uint32_t voff[PER_WAVE];  // byte offset of this lane's chunk from the stage's base
    int kl[PER_WAVE];         // its k within the stage
    int rl[PER_WAVE];         // its first row, from r0
    const uint16_t *base;     // row r0 at k = 0
    int64_t bytes, step;      // from base to the operand's end; per stage
    int64_t ld, left;         // rows from r0

    static __device__ int swz_rows(int krow) { return ROWS == 256 ? swz_mn(krow) : (krow & 3) << 2; }

    __device__ void init(const Operand16 &x, int64_t K, int64_t r0, int wave, int lane) {
        ld = x.ld;
        left = x.R - r0;
        base = x.p + (KMAJOR ? r0 * ld : r0);
        // whole chunks: a last one may hold filling past K or R
        bytes = 2 * (KMAJOR ? (left - 1) * ld + (K + 7) / 8 * 8 : (K - 1) * ld + (left + 7) / 8 * 8);
        step = KMAJOR ? 2 * BK : 2 * BK * ld;
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int blk = wave * PER_WAVE + i;
            if (KMAJOR) {
                const int row = blk * (64 / CHK) + lane / CHK;
                const int c = (lane % CHK) ^ swz_k<CHK>(row);
                kl[i] = c * 8;
                rl[i] = row;
                voff[i] = row < left ? uint32_t((row * ld + c * 8) * 2) : OOB;
            } else {
                const int krow = blk * (64 / CHR) + lane / CHR;
                const int c = (lane % CHR) ^ swz_rows(krow);
                kl[i] = krow;
                rl[i] = c * 8;
                voff[i] = c * 8 < left ? uint32_t((krow * ld + c * 8) * 2) : OOB;
            }
        }
    }

    // ---- direct loads
    __device__ u32x4 rsrc(int64_t stage) const {
        const int64_t off = uniform(stage * step);
        const int64_t rest = uniform(bytes) - off;
        return dma::raw_buffer(static_cast<uint64_t>(uniform(reinterpret_cast<int64_t>(base)) + off),
                               static_cast<uint32_t>(rest < 0x7fffffff ? rest : 0x7fffffff));
    }
    __device__ void load(u32x4 rs, uint32_t lds0, int i, int64_t kleft, int wave) const {
        const uint32_t v = (kleft < BK && kl[i] >= kleft) ? OOB : voff[i];
        direct_load16(rs, lds0 + (wave * PER_WAVE + i) * 1024, v);
    }
    __device__ void issue(LDS char *dst, int64_t stage, int64_t K, int wave) const {
        const u32x4 rs = rsrc(stage);
        const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst));
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) load(rs, lds0, i, K - stage * BK, wave);
    }

    // ---- through registers: n values of a chunk may be read, the rest are 0
    __device__ u32x4 fetch(int i, int64_t stage, int64_t K) const {
        const int64_t k = stage * BK + kl[i];
        const int64_t inner = KMAJOR ? K - k : left - rl[i], outer = KMAJOR ? left - rl[i] : K - k;
        u32x4 v = {0, 0, 0, 0};
        if (outer <= 0 || inner <= 0) return v;
        const uint16_t *src = base + (KMAJOR ? rl[i] * ld + k : k * ld + rl[i]);
        if (inner >= 8) return *reinterpret_cast<const u32x4_ea *>(src);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < inner) v[e / 2] |= uint32_t(src[e]) << (16 * (e % 2));
        return v;
    }
    __device__ void put(LDS char *dst, int i, u32x4 v, int wave, int lane) const {
        *reinterpret_cast<LDS u32x4 *>(dst + (wave * PER_WAVE + i) * 1024 + lane * 16) = v;
    }

    // Fragment of 32 rows (from row `row0` of the panel) for k16 step kk.
    static __device__ u32x4 frag(const LDS char *panel, int row0, int kk, int lane) {
        if (KMAJOR) {
            const int row = row0 + (lane & 31);
            const int c = kk * 2 + (lane >> 5);
            return *reinterpret_cast<const LDS u32x4 *>(panel + row * (2 * BK) + ((c ^ swz_k<CHK>(row)) << 4));
        }
        const int g = lane >> 5, h = (lane >> 4) & 1, ii = lane & 15;
        const int col = row0 + h * 16 + 4 * (ii & 3);
        u32x4 out;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
            const int krow = kk * 16 + g * 8 + e2 * 4 + (ii >> 2);
            const int c = (col >> 3) ^ swz_rows(krow);
            const LDS s16x4 *p = reinterpret_cast<const LDS s16x4 *>(
                panel + krow * (2 * ROWS) + (c << 4) + ((col & 7) << 1));
            const u32x2 v = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<LDS s16x4 *>(p)));
            out[2 * e2] = v[0];
            out[2 * e2 + 1] = v[1];
        }
        return out;
    }
};

template <class T, int BM_, int BN_, int WAVES_M, int WAVES_N, bool A_KMAJOR, bool B_KMAJOR, bool DIRECT, int BK_ = 64, int STAGES = 2>
struct Tile {
    static constexpr int TM = BM_, TN = BN_, BK = BK_;
    static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = WAVES * 64;
    static constexpr int WTM = TM / WAVES_M, WTN = TN / WAVES_N;
    static constexpr int FM = WTM / 32, FN = WTN / 32;
    using PA = Panel<A_KMAJOR, TM, WAVES, BK>;
    using PB = Panel<B_KMAJOR, TN, WAVES, BK>;
    static constexpr int STAGE = PA::BYTES + PB::BYTES;
    static constexpr int LDS_BYTES = STAGES * STAGE;
    static constexpr int NEED = (WAVES * 32 * WTN * 4 + STAGE - 1) / STAGE;  // stages the epilogue uses
    static_assert(LDS_BYTES <= 160 * 1024 && (NEED == 1 || 2 * NEED <= STAGES), "LDS budget");
    typedef f32x16 Acc[FM][FN];

    // Waves are dealt to the four SIMDs in turn: consecutive waves share a
    // column block, so the waves of a ragged last tile that have work spread
    // over all of them.
    static __device__ int wave_m(int wave) { return wave % WAVES_M; }
    static __device__ int wave_n(int wave) { return wave / WAVES_M; }
    // The LDS a wave stages its rows of C in: stages that the last one does not use.
    static __device__ LDS float *staging(LDS char *lds, int buf, int wave) {
        const int first = NEED == 1 ? (buf + 1 == STAGES ? 0 : buf + 1) : (buf >= NEED ? 0 : NEED);
        return reinterpret_cast<LDS float *>(lds + first * STAGE) + wave * 32 * WTN;
    }

    static __device__ void read(u32x4 (&fa)[FM], u32x4 (&fb)[FN], const LDS char *stage, int wm, int wn,
                                int kk, int lane) {
        // in the order the matrix instructions use them
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = PB::frag(stage + PA::BYTES, wn * WTN + j * 32, kk, lane);
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = PA::frag(stage, wm * WTM + i * 32, kk, lane);
    }

    // The tile at (m0, n0): acc <- sum over the stages [s0, s1) of 64 k, in
    // blocks of 32 x 32 whose operands are swapped (lane l has row l % 32
    // and columns 8q + 4*(l / 32) + 0..3 of a block).  Returns the LDS buffer
    // the last stage used; every wave has then passed the barrier after which
    // the other one is free.
    static __device__ __forceinline__ int run(const Operand16 &a, const Operand16 &b, int64_t K,
                                              int64_t m0, int64_t n0, int64_t s0, int64_t s1,
                                              LDS char *lds, Acc &acc) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave_m(wave), wn = wave_n(wave);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        if (s1 <= s0) return 0;
        PA pa;
        PB pb;
        pa.init(a, K, m0, wave, lane);
        pb.init(b, K, n0, wave, lane);
        if constexpr (DIRECT) return run_direct(pa, pb, K, s0, s1, lds, acc, wm, wn, wave, lane);
        else return run_staged(pa, pb, K, s0, s1, lds, acc, wm, wn, wave, lane);
    }

    static __device__ __forceinline__ void mfmas(const u32x4 (&fa)[FM], const u32x4 (&fb)[FN], Acc &acc) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma32<T>(fb[j], fa[i], acc[i][j]);
    }

    // One k step: the matrix instructions on the fragments of slot SLOT in order,
    // and between them, evenly, the reads of the next step's fragments (step kk
    // of `stage`) into the other slot and whatever `also(q)` issues after the
    // q-th.  The order is kept: left to itself the compiler bunches the loads
    // behind the instructions (192 x 192 tiles, 4096 x 4096 x 4096: 102 us, so 96).
    template <int SLOT, class Also>
    static __device__ __forceinline__ void step(u32x4 (&fa)[2][FM], u32x4 (&fb)[2][FN], const LDS char *stage,
                                                int wm, int wn, int kk, int lane, Acc &acc, Also also) {
        constexpr int N = FM * FN, READS = FM + FN;
        constexpr int EACH = (READS + N - 1) / N, EVERY = N > READS ? N / READS : 1;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int i = q / FN, j = q % FN;
            acc[i][j] = mfma32<T>(fb[SLOT][j], fa[SLOT][i], acc[i][j]);
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
                const int r = q / EVERY * EACH + u;  // in the order the next step uses them
                if (q % EVERY != 0 || r >= READS) continue;
                if (r < FN) fb[SLOT ^ 1][r] = PB::frag(stage + PA::BYTES, wn * WTN + r * 32, kk, lane);
                else fa[SLOT ^ 1][r - FN] = PA::frag(stage, wm * WTM + (r - FN) * 32, kk, lane);
            }
            also(q);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    static __device__ __forceinline__ int run_direct(const PA &pa, const PB &pb, int64_t K, int64_t s0,
                                                     int64_t s1, LDS char *lds, Acc &acc, int wm, int wn,
                                                     int wave, int lane) {
        constexpr int KK = BK / 16, N = FM * FN;
        static_assert(KK % 2 == 0, "a stage's first fragments are in slot 0");
        constexpr int PER_STAGE = PA::PER_WAVE + PB::PER_WAVE;
        const int64_t steps = s1 - s0;
#pragma unroll
        for (int st = 0; st < STAGES; ++st) {
            if (st < steps) {
                pa.issue(lds + st * STAGE, s0 + st, K, wave);
                pb.issue(lds + st * STAGE + PA::BYTES, s0 + st, K, wave);
            }
        }
        wait_stages<PER_STAGE, STAGES>(int(steps - 1 < STAGES - 1 ? steps - 1 : STAGES - 1));
        __syncthreads();
        u32x4 fa[2][FM], fb[2][FN];
        read(fa[0], fb[0], lds, wm, wn, 0, lane);
        // Every stage but the last: its last k step waits for the next stage
        // (this wave's loads, then every wave's through the barrier, which
        // also says that this buffer has been read), reads that stage's first
        // fragments and refills this buffer between its matrix instructions.
        int buf = 0;
        auto nothing = [](int) {};
        auto multiply = [&](int64_t s, auto refills) {
            LDS char *stage = lds + buf * STAGE;
            const int next = buf + 1 == STAGES ? 0 : buf + 1;
#pragma unroll
            for (int kk = 0; kk < KK - 1; ++kk) {
                if (kk & 1) step<1>(fa, fb, stage, wm, wn, kk + 1, lane, acc, nothing);
                else step<0>(fa, fb, stage, wm, wn, kk + 1, lane, acc, nothing);
            }
            if constexpr (decltype(refills)::value) {
                const int64_t refill = s0 + s + STAGES;
                const u32x4 ra = pa.rsrc(refill), rb = pb.rsrc(refill);
                const uint32_t la = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(stage));
                const int64_t kleft = K - refill * BK;
                wait_vmcnt<(STAGES - 2) * PER_STAGE>();
                wait_lgkmcnt0();
                __syncthreads();
                step<1>(fa, fb, lds + next * STAGE, wm, wn, 0, lane, acc, [&](int q) {
                    constexpr int EACH = (PER_STAGE + N - 1) / N;
#pragma unroll
                    for (int u = 0; u < EACH; ++u) {
                        const int l = q * EACH + u;
                        if (l < PA::PER_WAVE) pa.load(ra, la, l, kleft, wave);
                        else if (l < PER_STAGE) pb.load(rb, la + PA::BYTES, l - PA::PER_WAVE, kleft, wave);
                    }
                });
            } else {
                const int64_t later = steps - 2 - s;
                wait_stages<PER_STAGE, STAGES>(int(later < STAGES - 2 ? later : STAGES - 2));
                wait_lgkmcnt0();
                __syncthreads();
                step<1>(fa, fb, lds + next * STAGE, wm, wn, 0, lane, acc, nothing);
            }
            buf = next;
        };
        int64_t s = 0;
        for (; s < steps - STAGES; ++s) multiply(s, std::true_type{});
        for (; s < steps - 1; ++s) multiply(s, std::false_type{});
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if (kk < KK - 1) read(fa[(kk & 1) ^ 1], fb[(kk & 1) ^ 1], lds + buf * STAGE, wm, wn, kk + 1, lane);
            mfmas(fa[kk & 1], fb[kk & 1], acc);
        }
        return buf;
    }

    // Loads of the next stage are in registers while this one is computed.
    static __device__ __forceinline__ int run_staged(const PA &pa, const PB &pb, int64_t K, int64_t s0,
                                                     int64_t s1, LDS char *lds, Acc &acc, int wm, int wn,
                                                     int wave, int lane) {
        u32x4 ga[PA::PER_WAVE], gb[PB::PER_WAVE];
        auto fetch = [&](int64_t s) {
#pragma unroll
            for (int i = 0; i < PA::PER_WAVE; ++i) ga[i] = pa.fetch(i, s, K);
#pragma unroll
            for (int i = 0; i < PB::PER_WAVE; ++i) gb[i] = pb.fetch(i, s, K);
        };
        auto put = [&](LDS char *stage) {
#pragma unroll
            for (int i = 0; i < PA::PER_WAVE; ++i) pa.put(stage, i, ga[i], wave, lane);
#pragma unroll
            for (int i = 0; i < PB::PER_WAVE; ++i) pb.put(stage + PA::BYTES, i, gb[i], wave, lane);
        };
        fetch(s0);
        put(lds);
        __syncthreads();
        int buf = 0;
        for (int64_t s = s0; s < s1; ++s) {
            if (s + 1 < s1) fetch(s + 1);
            u32x4 fa[FM], fb[FN];
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
                read(fa, fb, lds + buf * STAGE, wm, wn, kk, lane);
                mfmas(fa, fb, acc);
            }
            if (s + 1 >= s1) break;
            // the other buffer was read in the step before the last barrier
            put(lds + (buf ^ 1) * STAGE);
            __syncthreads();
            buf ^= 1;
        }
        return buf;
    }
};

// Walks one wave's finished tile (top left at (mw, nw)) in pieces of 8
// columns: f(m, n, count, x, data) for every piece with m < M and n < N, count =
// min(8, N - n), x its fp32 accumulators.  Each strip of 32 rows passes
// through the wave's own LDS (chunk c of row r at c ^ (r mod 16)), so that a
// lane's piece is contiguous and eight lanes have a row: the epilogue's loads and
// stores move whole rows of 64 columns.  A lane sees the same columns,
// nw + 8*(lane % (FN*4)), in every call.
//
// What the epilogue reads, f.load(data, m, n, count), is asked for a strip
// ahead: read where it is needed, each of a tile's 16 pieces per lane would
// wait for memory by itself.
template <int FM, int FN, class F>
__device__ __forceinline__ void visit_tile(const f32x16 (&acc)[FM][FN], int64_t M, int64_t N, int64_t mw,
                                           int64_t nw, int lane, LDS float *scratch, F &&f) {
    constexpr int W = FN * 32, SWZ = W == 96 ? 7 : W / 4 - 1 < 15 ? W / 4 - 1 : 15;  // stays within the row
    // rows of 96 columns take 12 lanes each, four rows at a time
    constexpr int CPR = W / 8, RPI = CPR == 12 ? 4 : 64 / CPR, ITS = 32 / RPI, AHEAD = 4;
    static_assert(32 % RPI == 0 && CPR * RPI <= 64, "strip shape");
    typedef typename std::remove_reference_t<F>::Data Data;
    auto at = [&](int r, int col) { return scratch + r * W + (((col >> 2) ^ (r & SWZ)) << 2); };
    const int64_t n = nw + (lane % CPR) * 8;
    const int count = lane >= CPR * RPI ? 0 : N - n < 8 ? int(N - n) : 8;
    auto row_of = [&](int i, int it) { return mw + i * 32 + it * RPI + lane / CPR; };
    Data data[2][AHEAD];
    auto load = [&](int i, int it0, Data (&d)[AHEAD]) {
#pragma unroll
        for (int it = 0; it < AHEAD; ++it)
            if (it0 + it < ITS && row_of(i, it0 + it) < M && count > 0) f.load(d[it], row_of(i, it0 + it), n, count);
    };
    load(0, 0, data[0]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                *reinterpret_cast<LDS f32x4 *>(at(lane & 31, j * 32 + q * 8 + 4 * (lane >> 5))) = v;
            }
#pragma unroll
        for (int it0 = 0; it0 < ITS; it0 += AHEAD) {
            constexpr int GROUPS = (ITS + AHEAD - 1) / AHEAD;
            const int g = i * GROUPS + it0 / AHEAD;
            if (it0 + AHEAD < ITS) load(i, it0 + AHEAD, data[(g + 1) % 2]);
            else if (i + 1 < FM) load(i + 1, 0, data[(g + 1) % 2]);
#pragma unroll 1
            for (int it = 0; it < (ITS - it0 < AHEAD ? ITS - it0 : AHEAD); ++it) {
                const int r = (it0 + it) * RPI + lane / CPR;
                float x[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 v = *reinterpret_cast<const LDS f32x4 *>(at(r, (lane % CPR) * 8 + 4 * h));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * h + e] = v[e];
                }
                const Data d = pick(data[g % 2], it);
                if (mw + i * 32 + r < M && count > 0) f(mw + i * 32 + r, n, count, x, d);
            }
        }
    }
}

// The same tile turned: f(n, m, count, x, data) for pieces of 8 rows of a
// column n, count = min(8, M - m), through strips of 32 columns by up to 64 rows.
template <int FM, int FN, class F>
__device__ __forceinline__ void visit_tile_turned(const f32x16 (&acc)[FM][FN], int64_t M, int64_t N, int64_t mw,
                                                  int64_t nw, int lane, LDS float *scratch, F &&f) {
    constexpr int HIGH = FM < 2 ? 1 : 2, W = HIGH * 32, CPR = W / 8, RPI = 64 / CPR, ITS = 32 / RPI;
    constexpr int STRIPS = (FM + HIGH - 1) / HIGH;
    typedef typename std::remove_reference_t<F>::Data Data;
    const int c = (lane % CPR) * 8;
    Data data[2][4];
    auto load = [&](int strip, Data (&d)[4]) {
        const int j = strip / STRIPS, i0 = strip % STRIPS * HIGH;
        const int64_t m = mw + i0 * 32 + c;
        const bool live = m < M && i0 * 32 + c < FM * 32;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
            const int64_t n = nw + j * 32 + it * RPI + lane / CPR;
            if (live && n < N) f.load(d[it], n, m, M - m < 8 ? int(M - m) : 8);
        }
    };
    load(0, data[0]);
#pragma unroll
    for (int strip = 0; strip < FN * STRIPS; ++strip) {
        const int j = strip / STRIPS, i0 = strip % STRIPS * HIGH;
#pragma unroll
        for (int i = i0; i < i0 + HIGH && i < FM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                scratch[(8 * (e / 4) + 4 * (lane >> 5) + e % 4) * W + (i - i0) * 32 + (lane & 31)] = acc[i][j][e];
        if (strip + 1 < FN * STRIPS) load(strip + 1, data[(strip + 1) % 2]);
        const int64_t m = mw + i0 * 32 + c;
        const bool live = m < M && i0 * 32 + c < FM * 32;
#pragma unroll 1
        for (int it = 0; it < ITS; ++it) {
            const int r = it * RPI + lane / CPR;
            float x[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = *reinterpret_cast<const LDS f32x4 *>(scratch + r * W + c + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * h + e] = v[e];
            }
            const Data d = pick(data[strip % 2], it);
            if (live && nw + j * 32 + r < N) f(nw + j * 32 + r, m, M - m < 8 ? int(M - m) : 8, x, d);
        }
    }
}

}  // namespace tile16
}  // namespace libgemm
