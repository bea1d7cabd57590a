// A whole layer of experts for a few tokens (gemm_experts_layer), in two
// kernels that each read every live expert's weights once.
//
//   up_kernel    h = act(Up[0 .. H) x) * (Up[H .. 2H) x): a workgroup has 16 of
//                H's rows, both halves, of one live expert, and up to 16, 32 or 64
//                tokens that chose it; its eight waves deal the contracted D
//                in runs of 128 and their sums meet in LDS;
//   down_kernel  y = sum over the token's experts of w Down h: a workgroup
//                has 16 of y's columns for all tokens and goes through
//                every live expert, its waves dealing (expert, run of H) pairs,
//                so a token's weighted sum is formed in one place and one order:
//                no atomics.  h is scaled by the token's weight, in fp32, and
//                split into two 16-bit pieces, so it is not rounded to 16
//                bits in between.
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

struct LayerArgs {
    ExpertsLayer p;
    float *h;  // [token][choice][H], fp32
    int live_most;
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

// The live experts, in rising order, in `list`; returns how many.  All
// threads of the workgroup call it.
__device__ int find_live(const LayerArgs &a, uint32_t *bits, uint16_t *list) {
    const int E = int(a.p.experts), slots = int(a.p.tokens * a.p.top_k), words = (E + 31) / 32;
    for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const uint32_t e = uint32_t(a.p.ids[i]);
        if (e < uint32_t(E)) atomicOr(&bits[e / 32], 1u << (e % 32));
    }
    __syncthreads();
    int before = 0, total = 0;
    const int mine = int(threadIdx.x);
    for (int i = 0; i < words; ++i) {
        const int n = __popc(bits[i]);
        if (i < mine) before += n;
        total += n;
    }
    if (mine < words)
        for (uint32_t b = bits[mine]; b != 0; b &= b - 1) list[before++] = uint16_t(32 * mine + __ffs(b) - 1);
    __syncthreads();
    return total;
}

// Whether token t chose expert e: its first choice of it, or -1, and the sum
// of its weights.
__device__ inline int choice_of(const LayerArgs &a, const int32_t *ids, int t, int e, float &w) {
    int first = -1;
    w = 0.0f;
    const int k = int(a.p.top_k);
    for (int j = 0; j < k; ++j)
        if (ids[t * k + j] == e) {
            w += a.p.weights[t * k + j];
            first = first < 0 ? j : first;
        }
    return first;
}

// F: fragments of 16 tokens.
template <class T, int TYPE, int F>
__global__ __launch_bounds__(WAVES * 64) void up_kernel(LayerArgs a) {
    const ExpertsLayer &p = a.p;
    __shared__ uint32_t bits[LAYER_MAX_EXPERTS / 32];
    __shared__ uint16_t list[LAYER_MAX_EXPERTS];
    __shared__ int16_t token[LAYER_MAX_TOKENS], choice[LAYER_MAX_TOKENS];
    __shared__ int count_shared;
    __shared__ f32x4 part[WAVES][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int live = find_live(a, bits, list);
    const int64_t which = blockIdx.x / ((p.H + 15) / 16), h0 = blockIdx.x % ((p.H + 15) / 16) * 16;
    if (which >= live) return;
    const int e = list[which];
    // the tokens that chose it, in rising order
    if (wave == 0) {
        float w;
        const int c = lane < p.tokens ? choice_of(a, p.ids, lane, e, w) : -1;
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
    for (int t0 = 0; t0 < count; t0 += 16 * F) {
        const char *x[F];
        bool has_x[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int i = t0 + 16 * f + r;
            has_x[f] = i < count;
            x[f] = static_cast<const char *>(p.X) + (has_x[f] ? token[i] * p.ldx * 2 : 0);
        }
        f32x4 g[F], m[F];
#pragma unroll
        for (int f = 0; f < F; ++f) g[f] = f32x4{0, 0, 0, 0}, m[f] = f32x4{0, 0, 0, 0};
        Run<TYPE> ng, nm;
        ng.fetch(gate, has_h, wave * RUN, p.D, q);
        nm.fetch(mult, has_h, wave * RUN, p.D, q);
        for (int64_t k0 = wave * RUN; k0 < p.D; k0 += WAVES * RUN) {
            const Run<TYPE> cg = ng, cm = nm;
            ng.fetch(gate, has_h, k0 + WAVES * RUN, p.D, q);
            nm.fetch(mult, has_h, k0 + WAVES * RUN, p.D, q);
            f32x4 bg[F], bm[F];
            if (TYPE != 0)
#pragma unroll
                for (int f = 0; f < F; ++f) bg[f] = f32x4{0, 0, 0, 0}, bm[f] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int64_t k = Run<TYPE>::at(s, k0, q);
                const u32x4 og = cg.template operand<T>(s, k0, p.D, q), om = cm.template operand<T>(s, k0, p.D, q);
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    u32x4 xv = {0, 0, 0, 0};
                    if (has_x[f] && k < p.D) xv = *reinterpret_cast<const u32x4 *>(x[f] + k * 2);
                    Run<TYPE>::cut(xv, k, p.D);
                    if (TYPE == 0) {
                        g[f] = mfma16<T>(og, xv, g[f]);
                        m[f] = mfma16<T>(om, xv, m[f]);
                    } else {
                        bg[f] = mfma16<T>(og, xv, bg[f]);
                        bm[f] = mfma16<T>(om, xv, bm[f]);
                    }
                }
            }
            if (TYPE != 0) {
                // the 16 rows lie in one or, where H is not a multiple of 16,
                // the multiplied half's in two blocks of 128 rows: by row
                const float *sc = p.up.scale + e * p.up.stride_scale + (k0 / 128) * p.up.lds;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t hr = h0 + 4 * q + i < p.H ? h0 + 4 * q + i : h0;
                    const float sg = sc[hr / 128], sm = sc[(p.H + hr) / 128];
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        g[f][i] = __builtin_fmaf(sg, bg[f][i], g[f][i]);
                        m[f][i] = __builtin_fmaf(sm, bm[f][i], m[f][i]);
                    }
                }
            }
        }
        // a lane's registers: rows h0 + 4q + 0..3 of token r
#pragma unroll
        for (int f = 0; f < F; ++f) {
            __syncthreads();
            part[wave][0][lane] = g[f];
            part[wave][1][lane] = m[f];
            __syncthreads();
            if (wave == 0) {
                f32x4 sg = {0, 0, 0, 0}, sm = {0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    const f32x4 og = part[w][0][lane], om = part[w][1][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sg[i] += og[i], sm[i] += om[i];
                }
                const int i = t0 + 16 * f + r;
                if (i < count) {
                    float *h = a.h + (token[i] * p.top_k + choice[i]) * p.H + h0 + 4 * q;
                    float v[4] = {sg[0], sg[1], sg[2], sg[3]};
                    act::apply(p.act, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (h0 + 4 * q + j < p.H) h[j] = v[j] * sm[j];
                }
            }
        }
    }
}

// F: fragments of 16 tokens, F * 16 >= tokens.
template <class T, int TYPE, int F>
__global__ __launch_bounds__(WAVES * 64) void down_kernel(LayerArgs a) {
    const ExpertsLayer &p = a.p;
    __shared__ uint32_t bits[LAYER_MAX_EXPERTS / 32];
    __shared__ uint16_t list[LAYER_MAX_EXPERTS];
    __shared__ f32x4 part[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int live = find_live(a, bits, list);
    const int r = lane & 15, q = lane >> 4;
    const int64_t d0 = int64_t(blockIdx.x) * 16;
    const bool has_d = d0 + r < p.D;
    const int ESZ = TYPE == 0 ? 2 : 1;
    const char *down = static_cast<const char *>(p.down.w) + (d0 + r) * p.down.ld * ESZ;
    const int runs = int((p.H + RUN - 1) / RUN), units = live * runs;
    f32x4 acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = f32x4{0, 0, 0, 0};
    Run<TYPE> next;
    auto fetch = [&](int u) {
        if (u < units) next.fetch(down + list[u / runs] * p.down.stride * ESZ, has_d, int64_t(u % runs) * RUN, p.H, q);
    };
    fetch(wave);
    for (int u = wave; u < units; u += WAVES) {
        const Run<TYPE> cur = next;
        fetch(u + WAVES);
        const int e = list[u / runs];
        const int64_t k0 = int64_t(u % runs) * RUN;
        float w;
        const int c = lane < p.tokens ? choice_of(a, p.ids, lane, e, w) : -1;
        const uint64_t mask = __ballot(c >= 0);
        f32x4 block[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            block[f] = f32x4{0, 0, 0, 0};
            if ((mask >> (16 * f) & 0xffffu) == 0) continue;  // the same for the whole wave
            const int ct = __shfl(c, 16 * f + r);
            const float wt = __shfl(w, 16 * f + r);
            const float *h = a.h + ((16 * f + r) * p.top_k + ct) * p.H;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int64_t k = Run<TYPE>::at(s, k0, q);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.0f;
                if (ct >= 0 && k < p.H) load8f(h + k, p.H - k < 8 ? int(p.H - k) : 8, x);
                float lo[8];
                u32x4 hi;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= wt;
                    lo[i] = x[i] - decode<T>(encode<T>(x[i]));
                }
                hi = pack8<T>(x);
                const u32x4 od = cur.template operand<T>(s, k0, p.H, q);
                block[f] = mfma16<T>(od, pack8<T>(lo), block[f]);
                block[f] = mfma16<T>(od, hi, block[f]);
            }
        }
        float sc[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (TYPE != 0) {
            // d0 is a multiple of 16: the workgroup's rows lie in one block
            const float v = p.down.scale[e * p.down.stride_scale + (k0 / 128) * p.down.lds + d0 / 128];
            sc[0] = sc[1] = sc[2] = sc[3] = v;
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[f][i] = TYPE == 0 ? acc[f][i] + block[f][i] : __builtin_fmaf(sc[i], block[f][i], acc[f][i]);
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
        __syncthreads();
        part[wave][lane] = acc[f];
        __syncthreads();
        const int64_t t = 16 * f + r;
        if (wave != 0 || t >= p.tokens) continue;
        f32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const f32x4 o = part[w][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += o[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t d = d0 + 4 * q + i, at = t * p.ldy + d;
            if (d >= p.D) continue;
            if (p.out == 0) {
                float *y = static_cast<float *>(p.Y) + at;
                *y = p.beta != 0.0f ? __builtin_fmaf(p.beta, *y, s[i]) : s[i];
            } else {
                uint16_t *y = static_cast<uint16_t *>(p.Y) + at;
                *y = uint16_t(encode<T>(p.beta != 0.0f ? __builtin_fmaf(p.beta, decode<T>(*y), s[i]) : s[i]));
            }
        }
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class T, int TYPE, int F>
hipError_t run(const LayerArgs &a, hipStream_t stream) {
    const int64_t up = a.live_most * ceil_div(a.p.H, 16);
    if (up > 0x7fffff || ceil_div(a.p.D, 16) > 0x7fffff) return hipErrorInvalidConfiguration;
    up_kernel<T, TYPE, F><<<dim3(unsigned(up)), dim3(WAVES * 64), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    down_kernel<T, TYPE, F><<<dim3(unsigned(ceil_div(a.p.D, 16))), dim3(WAVES * 64), 0, stream>>>(a);
    return hipGetLastError();
}
template <class T, int TYPE>
hipError_t run_tokens(const LayerArgs &a, hipStream_t stream) {
    if (a.p.tokens <= 16) return run<T, TYPE, 1>(a, stream);
    if (a.p.tokens <= 32) return run<T, TYPE, 2>(a, stream);
    return run<T, TYPE, 4>(a, stream);
}
template <class T>
hipError_t run_type(const LayerArgs &a, hipStream_t stream) {
    if (a.p.type == 0) return run_tokens<T, 0>(a, stream);
    return a.p.type == 1 ? run_tokens<T, 1>(a, stream) : run_tokens<T, 2>(a, stream);
}

}  // namespace

size_t experts_layer_workspace(int64_t tokens, int64_t, int64_t top_k, int64_t, int64_t H) {
    return size_t(tokens * top_k * H * 4 + 16);
}

hipError_t launch_experts_layer(const ExpertsLayer &p, hipStream_t stream) {
    LayerArgs a{p, static_cast<float *>(p.workspace), int(p.experts < p.tokens * p.top_k ? p.experts : p.tokens * p.top_k)};
    return p.in == 1 ? run_type<BF16>(a, stream) : run_type<F16>(a, stream);
}

}  // namespace libgemm
