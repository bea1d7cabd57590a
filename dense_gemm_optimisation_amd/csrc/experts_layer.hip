// A whole layer of experts for a few tokens (gemm_experts_layer), in two
// kernels that each read every live expert's weights once.
//
//   up_kernel    w h, h = act(Up[0 .. H) x) * (Up[H .. 2H) x): a wave has 16 of
//                H's rows, both halves, of one live expert, and the tokens that
//                chose it; where that leaves too few waves, up to eight share
//                the rows' D and meet in LDS.  w h leaves as two 16-bit
//                pieces, hi + lo, so it is not rounded to 16 bits in between;
//   down_kernel  y = sum over the token's experts of Down (w h): a workgroup
//                has 16 of y's columns for all tokens and goes through
//                every live expert, its waves dealing (expert, run of H) pairs,
//                so a token's weighted sum is formed in one place and one order:
//                no atomics.
//
// Bound by reading the weights.  The 16 x 16 x 32 matrix instruction takes
// them as its 16-row operand straight from global memory (a wave reads 16
// rows of 64 bytes), with the tokens as its other 16: padded tokens cost
// nothing that is not idle anyway.  8-bit codes are loaded 16 to a lane and
// taken as two steps of eight, with the activations' k in the same order, and
// widened exactly; a run of 128 has one scale.
//
// Each workgroup finds the live experts from the ids by itself (at most 2048
// of them, from L2), which saves a launch.
#include "activation.hpp"
#include "layers.hpp"
#include "tile16.hpp"

namespace libgemm {
namespace {

using namespace tile16;

constexpr int WAVES = 8, RUN = 128, STEPS = RUN / 32;
constexpr int MOST_SLOTS = LAYER_MAX_TOKENS * LAYER_MAX_TOP_K;

struct LayerArgs {
    ExpertsLayer p;
    // w h of each choice, two pieces of X's type: [token][choice][piece][ldh]; its first choice of an
    // expert has all of the token's
    uint16_t *h;
    int64_t ldh;  // H rounded up to 8, the filling zero
    int live_most;
    int slices;   // waves of up_kernel that share a block's columns
};

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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight codes as eight 16-bit values, exactly.
template <class T, int TYPE, bool HIGH>
__device__ inline uint32_t widen2(uint32_t w) {
    if constexpr (__is_same(T, BF16)) {
        const bf16x2 v = TYPE == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH)
                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, HIGH);
        return __builtin_bit_cast(uint32_t, v);
    } else {
        const f16x2 v = TYPE == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH)
                                  : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, HIGH);
        return __builtin_bit_cast(uint32_t, v);
    }
}
template <class T, int TYPE>
__device__ inline u32x4 widen(uint32_t lo, uint32_t hi) {
    return u32x4{widen2<T, TYPE, false>(lo), widen2<T, TYPE, true>(lo), widen2<T, TYPE, false>(hi), widen2<T, TYPE, true>(hi)};
}

__device__ inline u32x4 load16(const char *base, uint32_t offset) {
    return *reinterpret_cast<const u32x4 *>(base + offset);
}

// Where lane q of four (lane / 16) has its eight k of step s of a run: 16-bit
// weights are read as chunks of 8 at 32s + 8q, codes as chunks of 16 at
// 64(s/2) + 16q, the activations in the same order.
template <int TYPE>
__device__ constexpr int k_of(int s, int q) {
    return TYPE == 0 ? 32 * s + 8 * q : 64 * (s / 2) + 16 * q + 8 * (s % 2);
}
// Zeros for the values at K and beyond of a chunk that starts at k.
__device__ inline void cut(u32x4 &w, int k, int K) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e >= K) w[e / 2] &= e % 2 ? 0xffffu : 0xffff0000u;
}

// One row's weights of a run of 128 k, as a lane holds them.
template <int TYPE>
struct Run {
    static constexpr int LOADS = TYPE == 0 ? 4 : 2, PER = TYPE == 0 ? 8 : 16;
    u32x4 v[LOADS];

    // base: the rows at the run's first k (the same in the whole wave);
    // offset: of the lane's row and chunk.
    __device__ void fetch(const char *base, uint32_t offset) {
#pragma unroll
        for (int s = 0; s < LOADS; ++s) v[s] = load16(base, offset + s * 64);
    }
    // A last run of `left` < 128 values: chunks that start within them.
    __device__ void fetch_part(const char *base, uint32_t offset, int left, int q) {
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < LOADS; ++s) v[s] = s * 4 * PER + q * PER < left ? load16(base, offset + s * 64) : zero;
    }
    // The operand of step s.
    template <class T>
    __device__ u32x4 operand(int s) const {
        if constexpr (TYPE == 0) return v[s];
        else return widen<T, TYPE>(v[s / 2][2 * (s % 2)], v[s / 2][2 * (s % 2) + 1]);
    }
    template <class T>
    __device__ u32x4 operand_part(int s, int left, int q) const {
        u32x4 w = operand<T>(s);
        cut(w, k_of<TYPE>(s, q), left);
        return w;
    }
};

// The same of a run of activations, 16-bit, in the order of TYPE's weights.
template <int TYPE>
__device__ inline void fetch_values(u32x4 (&v)[STEPS], const char *base, uint32_t offset) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) v[s] = load16(base, offset + 2 * k_of<TYPE>(s, 0));
}
template <int TYPE>
__device__ inline void fetch_values_part(u32x4 (&v)[STEPS], const char *base, uint32_t offset, int left, int q) {
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        v[s] = k_of<TYPE>(s, q) < left ? load16(base, offset + 2 * k_of<TYPE>(s, 0)) : zero;
        cut(v[s], k_of<TYPE>(s, q), left);
    }
}
// Bytes from a row's start to lane q's first chunk of activations.
template <int TYPE>
__device__ inline uint32_t lane_bytes(int q) { return (TYPE == 0 ? 16 : 32) * q; }

template <class P>
__device__ inline P uniform_pointer(P p) {
    return reinterpret_cast<P>(uniform(reinterpret_cast<int64_t>(p)));
}

// What a workgroup finds out from the ids: the live experts in rising order.
struct Live {
    uint32_t bits[LAYER_MAX_EXPERTS / 32];
    uint16_t list[LAYER_MAX_EXPERTS];
    int16_t ids[MOST_SLOTS];  // -1: no expert
};

// Fills it; returns how many are live.  All threads of the workgroup call it.
__device__ int find_live(const LayerArgs &a, Live &live) {
    const int E = int(a.p.experts), slots = int(a.p.tokens * a.p.top_k), words = (E + 31) / 32;
    for (int i = threadIdx.x; i < words; i += blockDim.x) live.bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const uint32_t e = uint32_t(a.p.ids[i]);
        live.ids[i] = e < uint32_t(E) ? int16_t(e) : int16_t(-1);
        if (e < uint32_t(E)) atomicOr(&live.bits[e / 32], 1u << (e % 32));
    }
    __syncthreads();
    int before = 0, total = 0;
    const int mine = int(threadIdx.x);
    for (int i = 0; i < words; ++i) {
        const int n = __popc(live.bits[i]);
        if (i < mine) before += n;
        total += n;
    }
    if (mine < words)
        for (uint32_t b = live.bits[mine]; b != 0; b &= b - 1) live.list[before++] = uint16_t(32 * mine + __ffs(b) - 1);
    __syncthreads();
    return total;
}

// Token t's first choice of expert e, or -1.
__device__ inline int choice_of(const Live &live, int t, int k, int e) {
    int first = -1;
    for (int j = k - 1; j >= 0; --j)
        if (live.ids[t * k + j] == e) first = j;
    return first;
}

// A float at an address that is the same in the whole wave, by a scalar load:
// loads into vector registers return in order, so a scale fetched that way
// would wait for the weights on their way before it.
__device__ inline float scalar_load(const float *p) {
    typedef const float __attribute__((address_space(4))) *constant;
    return *reinterpret_cast<constant>(static_cast<uint64_t>(uniform(reinterpret_cast<int64_t>(p))));
}

// F: fragments of 16 tokens at a time; an expert with more reads its weights
// again, from L2.  A wave has 16 rows of both halves and 1 / slices of D;
// waves of one block of rows meet in LDS.
//
// Rows past H and tokens past the expert's are computed from rows that are
// there, and not stored: a row's and a token's results depend on no other.
template <class T, int TYPE, int F, int AHEAD>
__global__ __launch_bounds__(WAVES * 64, 1) void up_kernel(LayerArgs a) {
    const ExpertsLayer &p = a.p;
    __shared__ Live live;
    __shared__ int16_t token[LAYER_MAX_TOKENS], choice[LAYER_MAX_TOKENS];
    __shared__ int count_shared;
    __shared__ f32x4 part[WAVES][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slices = a.slices, per = WAVES / slices;  // blocks of 16 rows in a workgroup
    const int groups = int((p.H + 16 * per - 1) / (16 * per));
    const int n_live = find_live(a, live);
    const int which = blockIdx.x / groups;
    if (which >= n_live) return;
    const int e = __builtin_amdgcn_readfirstlane(live.list[which]), k = int(p.top_k);
    const int64_t h0 = (int64_t(blockIdx.x % groups) * per + wave / slices) * 16;
    const int slice = wave % slices;
    // the tokens that chose it, in rising order
    if (wave == 0) {
        const int c = lane < p.tokens ? choice_of(live, lane, k, e) : -1;
        const uint64_t mask = __ballot(c >= 0);
        if (c >= 0) {
            const int at = __popcll(mask & ((uint64_t(1) << lane) - 1));
            token[at] = int16_t(lane);
            choice[at] = int16_t(c);
        }
        if (lane == 0) count_shared = __popcll(mask);
    }
    __syncthreads();
    const int count = __builtin_amdgcn_readfirstlane(count_shared);
    const int r = lane & 15, q = lane >> 4;
    constexpr int ESZ = TYPE == 0 ? 2 : 1;
    const int64_t first = h0 < p.H ? h0 : p.H - 1;
    const int64_t row = first + r < p.H ? r : p.H - 1 - first;
    const char *gate = uniform_pointer(static_cast<const char *>(p.up.w) + (e * p.up.stride + first * p.up.ld) * ESZ);
    const char *mult = uniform_pointer(gate + p.H * p.up.ld * ESZ);
    const uint32_t offset = uint32_t(row * p.up.ld * ESZ) + 16 * q;
    // the 16 rows of the activated half lie in one block of 128, the others'
    // (lo .. hi) in two where H is no multiple of 16
    const int64_t last = h0 + 15 < p.H ? h0 + 15 : p.H - 1;
    const int64_t in_gate = uniform(first / 128), in_lo = uniform((p.H + first) / 128), in_hi = uniform((p.H + last) / 128);
    const int64_t in_first = in_hi * 128 - (p.H + h0);  // rows of the block of lo, where there are two
    const float *scale = p.up.scale + e * p.up.stride_scale;
    // Whole runs of weights and activations are on their way AHEAD runs before
    // they are multiplied; past the last one the last is fetched again, so
    // that nothing branches around a load.
    Run<TYPE> ng[AHEAD], nm[AHEAD];
    u32x4 nx[AHEAD][F][STEPS];
    float sg[AHEAD], sm_lo[AHEAD], sm_hi[AHEAD];
    uint32_t x[F];
    const int whole = int(p.D / RUN), mine = (whole - slice + slices - 1) / slices;  // of the slice
    const char *values = static_cast<const char *>(p.X);
    auto fetch_scales = [&](int i, int64_t run) {
        if (TYPE == 0) return;
        const float *sc = scale + run * p.up.lds;
        sg[i] = scalar_load(sc + in_gate);
        sm_lo[i] = scalar_load(sc + in_lo);
        sm_hi[i] = scalar_load(sc + in_hi);
    };
    auto fetch = [&](int i, int n) {
        const int64_t run = slice + int64_t(n < mine ? n : mine - 1) * slices;
        fetch_scales(i, run);
        ng[i].fetch(gate + run * RUN * ESZ, offset);
        nm[i].fetch(mult + run * RUN * ESZ, offset);
#pragma unroll
        for (int f = 0; f < F; ++f) fetch_values<TYPE>(nx[i][f], values + run * RUN * 2, x[f]);
    };
    for (int t0 = 0; t0 < count; t0 += 16 * F) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int at = t0 + 16 * f + r;
            x[f] = uint32_t(token[at < count ? at : 0] * p.ldx * 2) + lane_bytes<TYPE>(q);
        }
        f32x4 g[F], m[F];
#pragma unroll
        for (int f = 0; f < F; ++f) g[f] = f32x4{0, 0, 0, 0}, m[f] = f32x4{0, 0, 0, 0};
        // sums of one run (part: its `left` values) added to g and m
        auto multiply = [&](int i, bool part, int left) {
            f32x4 bg[F], bm[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                bg[f] = TYPE == 0 ? g[f] : f32x4{0, 0, 0, 0};
                bm[f] = TYPE == 0 ? m[f] : f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const u32x4 og = part ? ng[i].template operand_part<T>(s, left, q) : ng[i].template operand<T>(s);
                const u32x4 om = part ? nm[i].template operand_part<T>(s, left, q) : nm[i].template operand<T>(s);
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    bg[f] = mfma16<T>(og, nx[i][f][s], bg[f]);
                    bm[f] = mfma16<T>(om, nx[i][f][s], bm[f]);
                }
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                if (TYPE == 0) {
                    g[f] = bg[f];
                    m[f] = bm[f];
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float mult_scale = 4 * q + j < in_first ? sm_lo[i] : sm_hi[i];
                    g[f][j] = __builtin_fmaf(sg[i], bg[f][j], g[f][j]);
                    m[f][j] = __builtin_fmaf(mult_scale, bm[f][j], m[f][j]);
                }
            }
        };
        if (mine > 0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) fetch(i, i);
            int n = 0;
            for (; n + AHEAD <= mine; n += AHEAD)
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    multiply(i, false, RUN);
                    fetch(i, n + i + AHEAD);
                }
#pragma unroll
            for (int i = 0; i < AHEAD - 1; ++i)
                if (n + i < mine) multiply(i, false, RUN);
        }
        if (const int left = int(p.D % RUN); left != 0 && slice == whole % slices) {
            fetch_scales(0, whole);
            ng[0].fetch_part(gate + int64_t(whole) * RUN * ESZ, offset, left, q);
            nm[0].fetch_part(mult + int64_t(whole) * RUN * ESZ, offset, left, q);
#pragma unroll
            for (int f = 0; f < F; ++f) fetch_values_part<TYPE>(nx[0][f], values + int64_t(whole) * RUN * 2, x[f], left, q);
            multiply(0, true, left);
        }
        // a lane's registers: rows h0 + 4q + 0..3 of token r
#pragma unroll
        for (int f = 0; f < F; ++f) {
            if (t0 + 16 * f >= count) break;
            if (slices > 1) {
                if (t0 + f > 0) __syncthreads();
                part[wave][0][lane] = g[f];
                part[wave][1][lane] = m[f];
                __syncthreads();
                if (slice == 0)
                    for (int w = 1; w < slices; ++w) {
                        const f32x4 og = part[wave + w][0][lane], om = part[wave + w][1][lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j) g[f][j] += og[j], m[f][j] += om[j];
                    }
            }
            const int at = t0 + 16 * f + r;
            if (slice != 0 || at >= count || h0 + 4 * q >= a.ldh) continue;
            const int t = token[at];
            float w = 0.0f;
            for (int j = choice[at]; j < k; ++j)
                if (live.ids[t * k + j] == e) w += p.weights[t * k + j];
            float v[4] = {g[f][0], g[f][1], g[f][2], g[f][3]};
            act::apply(p.act, v);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = h0 + 4 * q + j < p.H ? v[j] * m[f][j] * w : 0.0f;
                hi[j] = encode<T>(v[j]);
                lo[j] = encode<T>(v[j] - decode<T>(hi[j]));
            }
            uint16_t *h = a.h + (t * k + choice[at]) * 2 * a.ldh + h0 + 4 * q;
            *reinterpret_cast<u32x2 *>(h) = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
            *reinterpret_cast<u32x2 *>(h + a.ldh) = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        }
    }
}

// A workgroup has 16 of y's columns; its waves deal (live expert, run of H)
// pairs.  A pair's tokens are those of the expert, 16 to a fragment; their
// sums are added to the tokens' in the wave's own part of LDS.
template <class T, int TYPE, int AHEAD>
__global__ __launch_bounds__(WAVES * 64, 1) void down_kernel(LayerArgs a) {
    const ExpertsLayer &p = a.p;
    __shared__ Live live;
    __shared__ uint8_t token[MOST_SLOTS];  // by live expert
    __shared__ uint16_t slot[MOST_SLOTS];  // token * top_k + choice
    __shared__ int16_t start[LAYER_MAX_EXPERTS + 1];
    extern __shared__ __attribute__((aligned(16))) char smem[];
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);  // [wave][token][four columns]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = int(p.top_k), tokens = int(p.tokens);
    const int n_live = find_live(a, live);
    const int r = lane & 15, q = lane >> 4;
    // the first choices of each live expert, by rising token
    for (int i = wave; i < n_live; i += WAVES) {
        const uint64_t mask = __ballot(lane < tokens && choice_of(live, lane, k, live.list[i]) >= 0);
        if (lane == 0) start[i + 1] = int16_t(__popcll(mask));
    }
    for (int i = threadIdx.x; i < WAVES * tokens * 4; i += WAVES * 64) sums[i] = f32x4{0, 0, 0, 0};
    __syncthreads();
    if (wave == 0) {
        int base = 0;
        for (int i0 = 0; i0 < n_live; i0 += 64) {
            int v = i0 + lane < n_live ? start[i0 + lane + 1] : 0;
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(v, d);
                if (lane >= d) v += o;
            }
            if (i0 + lane < n_live) start[i0 + lane + 1] = int16_t(base + v);
            base += __shfl(v, 63);
        }
        if (lane == 0) start[0] = 0;
    }
    __syncthreads();
    for (int i = wave; i < n_live; i += WAVES) {
        const int c = lane < tokens ? choice_of(live, lane, k, live.list[i]) : -1;
        const uint64_t mask = __ballot(c >= 0);
        if (c >= 0) {
            const int at = start[i] + __popcll(mask & ((uint64_t(1) << lane) - 1));
            token[at] = uint8_t(lane);
            slot[at] = uint16_t(lane * k + c);
        }
    }
    __syncthreads();
    const int64_t d0 = int64_t(blockIdx.x) * 16;
    constexpr int ESZ = TYPE == 0 ? 2 : 1;
    const int64_t row = d0 + r < p.D ? r : p.D - 1 - d0;  // rows past D: the last one's, not stored
    const char *down = static_cast<const char *>(p.down.w) + d0 * p.down.ld * ESZ;
    const uint32_t offset = uint32_t(row * p.down.ld * ESZ) + 16 * q;
    const int runs = int(p.H / RUN), units = n_live * runs;  // whole runs
    // Weights, and the pieces of w h of a unit's first tokens, are fetched
    // AHEAD units before they are multiplied; pieces fetched later than the
    // weights would wait for all weights asked for before.  Past the last unit
    // the last is fetched again, so that nothing branches around a load.
    struct Unit {
        int expert, run, first, end;  // first .. end: its slots
    };
    Run<TYPE> next[AHEAD];
    Unit unit[AHEAD];
    float next_scale[AHEAD];
    u32x4 hi[AHEAD][STEPS], lo[AHEAD][STEPS];
    // token r of the slots from `from` on; past the expert's, its first one
    // there, which is not added to a sum
    auto pieces_at = [&](const Unit &u, int from) {
        return uint32_t(slot[from + r < u.end ? from + r : from] * 4 * a.ldh) + lane_bytes<TYPE>(q);
    };
    auto pieces_base = [&](const Unit &u) { return reinterpret_cast<const char *>(a.h + int64_t(u.run) * RUN); };
    auto fetch_h = [&](int i, const Unit &u, int from) {
        const uint32_t at = pieces_at(u, from);
        fetch_values<TYPE>(hi[i], pieces_base(u), at);
        fetch_values<TYPE>(lo[i], pieces_base(u) + 2 * a.ldh, at);
    };
    auto weights_base = [&](const Unit &u) {
        const int e = __builtin_amdgcn_readfirstlane(live.list[u.expert]);
        return down + (e * p.down.stride + int64_t(u.run) * RUN) * ESZ;
    };
    auto fetch_scale = [&](int i, const Unit &u) {
        if (TYPE == 0) return;
        const int e = __builtin_amdgcn_readfirstlane(live.list[u.expert]);
        // 16 rows from a multiple of 16 lie in one block of 128
        next_scale[i] = scalar_load(p.down.scale + e * p.down.stride_scale + u.run * p.down.lds + d0 / 128);
    };
    auto unit_of = [&](int expert, int run) {
        return Unit{expert, run, __builtin_amdgcn_readfirstlane(start[expert]), __builtin_amdgcn_readfirstlane(start[expert + 1])};
    };
    // the sums of the 16 slots from s0 on, added to their tokens'
    auto multiply = [&](int i, const u32x4 (&od)[STEPS], const Unit &u, int s0) {
        f32x4 block = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            block = mfma16<T>(od[s], lo[i][s], block);
            block = mfma16<T>(od[s], hi[i][s], block);
        }
        if (s0 + r >= u.end) return;
        f32x4 *sum = sums + (wave * tokens + token[s0 + r]) * 4 + q;
        f32x4 v = *sum;
        const float scale = TYPE == 0 ? 1.0f : next_scale[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(scale, block[j], v[j]);
        *sum = v;
    };
    if (wave < units) {
        // the unit to fetch, and how far eight units are
        const int on_expert = WAVES / runs, on_run = WAVES % runs;
        int expert = wave / runs, run = wave % runs, at = wave;
        auto fetch = [&](int i) {
            unit[i] = unit_of(expert, run);
            next[i].fetch(weights_base(unit[i]), offset);
            fetch_scale(i, unit[i]);
            fetch_h(i, unit[i], unit[i].first);
            if (at + WAVES >= units) return;
            at += WAVES;
            expert += on_expert;
            run += on_run;
            if (run >= runs) run -= runs, ++expert;
        };
        auto step = [&](int i) {
            u32x4 od[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) od[s] = next[i].template operand<T>(s);
            const Unit u = unit[i];
            multiply(i, od, u, u.first);
            for (int s0 = u.first + 16; s0 < u.end; s0 += 16) {
                fetch_h(i, u, s0);
                multiply(i, od, u, s0);
            }
        };
        const int mine = (units - wave + WAVES - 1) / WAVES;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fetch(i);
        int n = 0;
        for (; n + AHEAD <= mine; n += AHEAD)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                step(i);
                fetch(i);
            }
#pragma unroll
        for (int i = 0; i < AHEAD - 1; ++i)
            if (n + i < mine) step(i);
    }
    if (const int left = int(p.H % RUN); left != 0)
        for (int i = wave; i < n_live; i += WAVES) {
            const Unit u = unit_of(i, runs);
            next[0].fetch_part(weights_base(u), offset, left, q);
            fetch_scale(0, u);
            u32x4 od[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) od[s] = next[0].template operand_part<T>(s, left, q);
            for (int s0 = u.first; s0 < u.end; s0 += 16) {
                const uint32_t at = pieces_at(u, s0);
                fetch_values_part<TYPE>(hi[0], pieces_base(u), at, left, q);
                fetch_values_part<TYPE>(lo[0], pieces_base(u) + 2 * a.ldh, at, left, q);
                multiply(0, od, u, s0);
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * 16; i += WAVES * 64) {
        const int t = i / 16;
        const int64_t d = d0 + i % 16, at = t * p.ldy + d;
        if (d >= p.D) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += reinterpret_cast<const float *>(sums)[w * tokens * 16 + i];
        if (p.out == 0) {
            float *y = static_cast<float *>(p.Y) + at;
            *y = p.beta != 0.0f ? __builtin_fmaf(p.beta, *y, s) : s;
        } else {
            uint16_t *y = static_cast<uint16_t *>(p.Y) + at;
            *y = uint16_t(encode<T>(p.beta != 0.0f ? __builtin_fmaf(p.beta, decode<T>(*y), s) : s));
        }
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Waves that share 16 rows: as many (1, 2, 4, 8) as it takes for 16 waves on
// each of 256 compute units when every slot has an expert of its own.
int up_slices(int64_t live, int64_t H) {
    const int64_t blocks = live * ceil_div(H, 16);
    int s = 1;
    while (s < WAVES && blocks * s < 4096) s *= 2;
    return s;
}

#ifndef UP_AHEAD
#define UP_AHEAD 2
#endif
#ifndef DOWN_AHEAD
#define DOWN_AHEAD 3
#endif
template <class T, int TYPE, int F>
hipError_t run(LayerArgs &a, hipStream_t stream) {
    a.slices = up_slices(a.live_most, a.p.H);
    const int64_t up = a.live_most * ceil_div(a.p.H, 16 * (WAVES / a.slices));
    if (up > 0x7fffff || ceil_div(a.p.D, 16) > 0x7fffff) return hipErrorInvalidConfiguration;
    up_kernel<T, TYPE, F, UP_AHEAD><<<dim3(unsigned(up)), dim3(WAVES * 64), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    down_kernel<T, TYPE, DOWN_AHEAD><<<dim3(unsigned(ceil_div(a.p.D, 16))), dim3(WAVES * 64), size_t(WAVES * a.p.tokens * 64), stream>>>(a);
    return hipGetLastError();
}
// Two fragments at a time where an expert has more than eight tokens in the mean.
template <class T, int TYPE>
hipError_t run_tokens(LayerArgs &a, hipStream_t stream) {
    return a.p.tokens > 16 && a.p.tokens * a.p.top_k > 8 * a.p.experts ? run<T, TYPE, 2>(a, stream) : run<T, TYPE, 1>(a, stream);
}
template <class T>
hipError_t run_type(LayerArgs &a, hipStream_t stream) {
    if (a.p.type == 0) return run_tokens<T, 0>(a, stream);
    return a.p.type == 1 ? run_tokens<T, 1>(a, stream) : run_tokens<T, 2>(a, stream);
}

}  // namespace

size_t experts_layer_workspace(int64_t tokens, int64_t, int64_t top_k, int64_t, int64_t H) {
    return size_t(tokens * top_k * 2 * ceil_div(H, 8) * 8 * 2 + 16);
}

hipError_t launch_experts_layer(const ExpertsLayer &p, hipStream_t stream) {
    LayerArgs a{p, static_cast<uint16_t *>(p.workspace), ceil_div(p.H, 8) * 8,
                int(p.experts < p.tokens * p.top_k ? p.experts : p.tokens * p.top_k), 1};
    return p.in == 1 ? run_type<BF16>(a, stream) : run_type<F16>(a, stream);
}

}  // namespace libgemm
