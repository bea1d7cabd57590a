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

// Eight codes as eight 16-bit values, exactly.
template <class T, int TYPE>
__device__ inline u32x4 widen(uint32_t lo, uint32_t hi) {
    float x[8];
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 a = TYPE == 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false) : __builtin_amdgcn_cvt_pk_f32_bf8(w[h], false);
        const f32x2 b = TYPE == 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true) : __builtin_amdgcn_cvt_pk_f32_bf8(w[h], true);
        x[4 * h] = a[0], x[4 * h + 1] = a[1], x[4 * h + 2] = b[0], x[4 * h + 3] = b[1];
    }
    return pack8<T>(x);
}

// One row's weights of a run of 128 from k0, as a lane holds them: 16-bit, the
// chunks of 8 at k0 + 32s + 8q; codes, the chunks of 16 at k0 + 64s + 16q
// (q = lane / 16).
template <int TYPE>
struct Run {
    static constexpr int LOADS = TYPE == 0 ? 4 : 2;
    u32x4 v[LOADS];

    // Chunks that begin at K or beyond are zeros; `row` is the row's start.
    __device__ void fetch(const char *row, bool live, int64_t k0, int64_t K, int q) {
        constexpr int PER = TYPE == 0 ? 8 : 16;
#pragma unroll
        for (int s = 0; s < LOADS; ++s) {
            const int64_t k = k0 + s * (4 * PER) + q * PER;
            const u32x4 zero = {0, 0, 0, 0};
            v[s] = live && k < K ? *reinterpret_cast<const u32x4 *>(row + k * (TYPE == 0 ? 2 : 1)) : zero;
        }
    }
    // The operand of step s; its values at K and beyond are zeros.
    template <class T>
    __device__ u32x4 operand(int s, int64_t k0, int64_t K, int q) const {
        u32x4 w = TYPE == 0 ? v[s % LOADS] : widen<T, TYPE>(v[s / 2 % LOADS][2 * (s & 1)], v[s / 2 % LOADS][2 * (s & 1) + 1]);
        cut(w, at(s, k0, q), K);
        return w;
    }
    // First k of step s's chunk.
    static __device__ int64_t at(int s, int64_t k0, int q) {
        return TYPE == 0 ? k0 + 32 * s + 8 * q : k0 + 64 * (s >> 1) + 16 * q + 8 * (s & 1);
    }
    static __device__ void cut(u32x4 &w, int64_t k, int64_t K) {
        if (k + 8 <= K) return;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e >= K) w[e / 2] &= e % 2 ? 0xffffu : 0xffff0000u;
    }
};

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
// again, from L2.  A wave has 16 rows of both halves and
// 1 / slices of D; waves of one block of rows meet in LDS.
template <class T, int TYPE, int F, int AHEAD>
__global__ __launch_bounds__(WAVES * 64, 1) void up_kernel(LayerArgs a) {
    const ExpertsLayer &p = a.p;
    __shared__ Live live;
    __shared__ int16_t token[LAYER_MAX_TOKENS], choice[LAYER_MAX_TOKENS];
    __shared__ int count_shared;
    __shared__ f32x4 part[WAVES][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slices = a.slices, per = WAVES / slices;  // blocks of 16 rows in a workgroup
    const int groups = int((p.H + 16 * per - 1) / (16 * per));
    const int n_live = find_live(a, live);
    const int which = blockIdx.x / groups;
    if (which >= n_live) return;
    const int e = live.list[which], k = int(p.top_k);
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
    const int count = count_shared;
    const int r = lane & 15, q = lane >> 4;
    const bool has_h = h0 + r < p.H;
    const int ESZ = TYPE == 0 ? 2 : 1;
    const char *gate = static_cast<const char *>(p.up.w) + (e * p.up.stride + (h0 + r) * p.up.ld) * ESZ;
    const char *mult = gate + p.H * p.up.ld * ESZ;
    // Runs of weights and activations are on their way AHEAD runs before they
    // are multiplied.
    Run<TYPE> ng[AHEAD], nm[AHEAD];
    u32x4 nx[AHEAD][F][STEPS];
    // the 16 rows of the activated half lie in one block of 128, the others'
    // (lo .. hi) in two where H is no multiple of 16
    float sg[AHEAD], sm_lo[AHEAD], sm_hi[AHEAD];
    const int64_t first = h0 < p.H ? h0 : p.H - 1, last = h0 + 15 < p.H ? h0 + 15 : p.H - 1;
    const int64_t in_gate = uniform(first / 128), in_lo = uniform((p.H + first) / 128), in_hi = uniform((p.H + last) / 128);
    const float *scale = p.up.scale + e * p.up.stride_scale;
    const char *x[F];
    bool has_x[F];
    auto fetch = [&](int i, int64_t k0) {
        if (TYPE != 0 && k0 < p.D) {
            const float *sc = scale + k0 / 128 * p.up.lds;
            sg[i] = scalar_load(sc + in_gate);
            sm_lo[i] = scalar_load(sc + in_lo);
            sm_hi[i] = scalar_load(sc + in_hi);
        }
        ng[i].fetch(gate, has_h, k0, p.D, q);
        nm[i].fetch(mult, has_h, k0, p.D, q);
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int64_t at = Run<TYPE>::at(s, k0, q);
                const u32x4 zero = {0, 0, 0, 0};
                nx[i][f][s] = has_x[f] && at < p.D ? *reinterpret_cast<const u32x4 *>(x[f] + at * 2) : zero;
            }
    };
    for (int t0 = 0; t0 < count; t0 += 16 * F) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int at = t0 + 16 * f + r;
            has_x[f] = at < count;
            x[f] = static_cast<const char *>(p.X) + (has_x[f] ? token[at] * p.ldx * 2 : 0);
        }
        f32x4 g[F], m[F];
#pragma unroll
        for (int f = 0; f < F; ++f) g[f] = f32x4{0, 0, 0, 0}, m[f] = f32x4{0, 0, 0, 0};
        const int64_t stride = int64_t(slices) * RUN;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fetch(i, slice * RUN + i * stride);
        for (int64_t k1 = slice * RUN; k1 < p.D; k1 += AHEAD * stride)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int64_t k0 = k1 + i * stride;
                if (k0 >= p.D) break;
                const float gate_scale = sg[i], lo_scale = sm_lo[i], hi_scale = sm_hi[i];
                f32x4 bg[F], bm[F];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    bg[f] = TYPE == 0 ? g[f] : f32x4{0, 0, 0, 0};
                    bm[f] = TYPE == 0 ? m[f] : f32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const u32x4 og = ng[i].template operand<T>(s, k0, p.D, q), om = nm[i].template operand<T>(s, k0, p.D, q);
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        u32x4 xv = nx[i][f][s];
                        Run<TYPE>::cut(xv, Run<TYPE>::at(s, k0, q), p.D);
                        bg[f] = mfma16<T>(og, xv, bg[f]);
                        bm[f] = mfma16<T>(om, xv, bm[f]);
                    }
                }
                fetch(i, k0 + AHEAD * stride);
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float mult_scale = (p.H + h0 + 4 * q + j) / 128 == in_lo ? lo_scale : hi_scale;
                        g[f][j] = TYPE == 0 ? bg[f][j] : __builtin_fmaf(gate_scale, bg[f][j], g[f][j]);
                        m[f][j] = TYPE == 0 ? bm[f][j] : __builtin_fmaf(mult_scale, bm[f][j], m[f][j]);
                    }
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
    __shared__ uint8_t token[MOST_SLOTS], choice[MOST_SLOTS];  // by live expert
    __shared__ int16_t start[LAYER_MAX_EXPERTS + 1];
    extern __shared__ __attribute__((aligned(16))) char smem[];
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);  // [wave][token][four columns]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
            choice[at] = uint8_t(c);
        }
    }
    __syncthreads();
    const int64_t d0 = int64_t(blockIdx.x) * 16;
    const bool has_d = d0 + r < p.D;
    const int ESZ = TYPE == 0 ? 2 : 1;
    const char *down = static_cast<const char *>(p.down.w) + (d0 + r) * p.down.ld * ESZ;
    const int runs = int((p.H + RUN - 1) / RUN), units = n_live * runs;
    Run<TYPE> next[AHEAD];
    float next_scale[AHEAD];
    auto fetch = [&](int i, int u) {
        if (u >= units) return;
        const int e = live.list[u / runs];
        const int64_t k0 = int64_t(u % runs) * RUN;
        next[i].fetch(down + e * p.down.stride * ESZ, has_d, k0, p.H, q);
        // 16 rows from a multiple of 16 lie in one block of 128
        if (TYPE != 0) next_scale[i] = scalar_load(p.down.scale + e * p.down.stride_scale + (k0 / 128) * p.down.lds + d0 / 128);
    };
    // the pieces of w h of a unit's first tokens, fetched with its weights:
    // fetched later, they would wait for all weights asked for before
    u32x4 hi[AHEAD][STEPS], lo[AHEAD][STEPS];
    auto fetch_h = [&](u32x4 (&vh)[STEPS], u32x4 (&vl)[STEPS], int u, int at) {
        // token `at` of the unit's expert
        if (u >= units) return;
        at += start[u / runs] + r;
        const bool has = at < start[u / runs + 1];
        const uint16_t *h = a.h + (has ? (token[at] * k + choice[at]) * 2 * a.ldh : 0);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int64_t from = Run<TYPE>::at(s, int64_t(u % runs) * RUN, q);
            const u32x4 zero = {0, 0, 0, 0};
            vh[s] = has && from < p.H ? *reinterpret_cast<const u32x4 *>(h + from) : zero;
            vl[s] = has && from < p.H ? *reinterpret_cast<const u32x4 *>(h + a.ldh + from) : zero;
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        fetch(i, wave + i * WAVES);
        fetch_h(hi[i], lo[i], wave + i * WAVES, 0);
    }
    for (int u0 = wave; u0 < units; u0 += AHEAD * WAVES)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int u = u0 + i * WAVES;
            if (u >= units) break;
            const int64_t k0 = int64_t(u % runs) * RUN;
            const int first = start[u / runs], end = start[u / runs + 1];
            const float scale = TYPE == 0 ? 1.0f : next_scale[i];
            u32x4 od[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) od[s] = next[i].template operand<T>(s, k0, p.H, q);
            for (int s0 = first; s0 < end; s0 += 16) {
                if (s0 > first) fetch_h(hi[i], lo[i], u, s0 - first);
                f32x4 block = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    block = mfma16<T>(od[s], lo[i][s], block);
                    block = mfma16<T>(od[s], hi[i][s], block);
                }
                if (s0 + r < end) {
                    f32x4 *sum = sums + (wave * tokens + token[s0 + r]) * 4 + q;
                    f32x4 v = *sum;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(scale, block[j], v[j]);
                    *sum = v;
                }
            }
            fetch(i, u + AHEAD * WAVES);
            fetch_h(hi[i], lo[i], u + AHEAD * WAVES, 0);
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
