// Routing tokens to experts: scores, the choice, the weights, and the rows of
// each expert; and the weights' gradient.
//
// One wave chooses for one token, lane l holding experts l, l + 64, ...: the
// largest key is found top_k times over the wave.  A workgroup's 64 tokens
// leave one 64-bit mask per expert (bit t: token t of the block chose it), in
// which a token's rank among the block's is a count of bits; a second kernel
// adds what earlier blocks hold.  No order of atomics enters a result.
#include "f8_block.hpp"

#include <cmath>

namespace libgemm {
namespace {

constexpr int WAVES = 4;

__device__ inline float load_logit(const void *x, int64_t at, int type) {
    if (type == 0) return static_cast<const float *>(x)[at];
    const uint16_t b = static_cast<const uint16_t *>(x)[at];
    return type == 1 ? __builtin_bit_cast(float, uint32_t(b) << 16)
                     : static_cast<float>(__builtin_bit_cast(_Float16, b));
}

struct Best {
    double key;
    int at;
};
// The larger key; of equal ones the lower index.
__device__ inline Best better(Best a, Best b) {
    return b.key > a.key || (b.key == a.key && b.at < a.at) ? b : a;
}
__device__ inline Best wave_best(Best x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = better(x, Best{__shfl_xor(x.key, d), __shfl_xor(x.at, d)});
    return x;
}
template <typename T>
__device__ inline T wave_sum(T x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

constexpr int NOBODY = 1 << 30;

// PER: experts per lane.
template <int PER>
__device__ inline void choose(const RouteArgs &a, int64_t t, int lane, unsigned long long *masks, int bit) {
    const double none = -INFINITY;
    const int E = a.experts;
    int32_t *ids = a.ids + t * a.top_k;
    float *weights = a.weights + t * a.top_k;
    bool live = a.keep == nullptr || a.keep[t] != 0;
    double l[PER], key[PER];
    bool odd = false;
    double top = none;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E && live ? double(load_logit(a.logits, t * a.ldl + e, a.type)) : none;
        odd = odd || l[i] != l[i] || l[i] == INFINITY;
        top = l[i] > top ? l[i] : top;
    }
    const bool undefined = !a.sigmoid && __ballot(odd) != 0;
    double sum = 0.0;
    if (!a.sigmoid) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_xor(top, d);
            top = o > top ? o : top;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += l[i] > none ? exp(l[i] - top) : 0.0;
        sum = wave_sum(sum);
    }
    auto score = [&](double x) { return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum; };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        key[i] = none;
        if (e >= E || undefined || !(l[i] > none)) continue;
        // without a bias or groups the logits rank as their scores do
        key[i] = a.bias == nullptr && a.groups == 1 ? l[i] : score(l[i]);
        if (a.bias != nullptr) key[i] += double(a.bias[e]);
        if (!(key[i] > none)) key[i] = none;
    }
    if (a.groups > 1) {
        const int per = E / a.groups;
        double rank = none;  // lane g's is group g's
        for (int g = 0; g < a.groups; ++g) {
            Best first{none, NOBODY}, second{none, NOBODY};
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 64 * i;
                if (e < E && e / per == g && key[i] > none) first = better(first, Best{key[i], e});
            }
            first = wave_best(first);
            double r = first.key;
            if (a.group_top == 2) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = lane + 64 * i;
                    if (e < E && e / per == g && e != first.at && key[i] > none)
                        second = better(second, Best{key[i], e});
                }
                second = wave_best(second);
                if (second.key > none) r += second.key;
            }
            if (lane == g) rank = r;
        }
        unsigned long long kept = 0;
        for (int n = 0; n < a.top_groups; ++n) {
            const Best b = wave_best(Best{rank, lane < a.groups && !(kept >> lane & 1) ? lane : NOBODY + lane});
            // groups with nobody rank -infinity and come last, by index
            if (b.at < NOBODY) kept |= 1ull << b.at;
            if (lane == b.at) rank = none;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            if (e < E && !(kept >> (e / per) & 1)) key[i] = none;
        }
    }
    double chosen = none;  // lane j's: the logit of choice j
    int id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        Best b{none, NOBODY};
        double logit = none;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > none) b = better(b, Best{key[i], lane + 64 * i});
        b = wave_best(b);
        if (b.at == NOBODY) break;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i == b.at) {
                logit = l[i];
                key[i] = none;
            }
        logit = __shfl(logit, b.at & 63);
        if (lane == j) {
            id = b.at;
            chosen = logit;
        }
    }
    double w = id >= 0 ? score(chosen) : 0.0;
    if (a.renormalise) {
        double first = 0.0;
        if (!a.sigmoid) {  // relative to the largest chosen: the sum cannot vanish
            first = id >= 0 ? chosen : none;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_xor(first, d);
                first = o > first ? o : first;
            }
            w = id >= 0 ? exp(chosen - first) : 0.0;
        }
        const double total = wave_sum(w);
        w = total > 0.0 ? w / total : 0.0;
    }
    w *= double(a.scale);
    if (id < 0) w = 0.0;
    if (undefined && live) w = __builtin_nan("");
    if (lane < a.top_k) {
        ids[lane] = id;
        weights[lane] = float(w);
        if (masks != nullptr && id >= 0) atomicOr(&masks[id], 1ull << bit);
    }
}

template <int PER>
__global__ __launch_bounds__(WAVES * 64) void choose_kernel(RouteArgs a) {
    __shared__ unsigned long long masks[ROUTE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool layout = a.masks != nullptr;
    if (layout) {
        for (int e = threadIdx.x; e < a.experts; e += WAVES * 64) masks[e] = 0;
        __syncthreads();
    }
    for (int i = wave; i < ROUTE_BLOCK; i += WAVES) {
        const int64_t t = int64_t(blockIdx.x) * ROUTE_BLOCK + i;
        if (t < a.tokens) choose<PER>(a, t, lane, layout ? masks : nullptr, i);
    }
    if (layout) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.experts; e += WAVES * 64)
            a.masks[int64_t(blockIdx.x) * a.experts + e] = masks[e];
    }
}

// Block b of tokens: where each of its rows goes.
__global__ __launch_bounds__(256) void place_kernel(RouteArgs a, int64_t blocks) {
    __shared__ int start[ROUTE_MAX_EXPERTS + 1];   // offsets
    __shared__ int before[ROUTE_MAX_EXPERTS];      // rows of earlier blocks
    __shared__ int count[ROUTE_MAX_EXPERTS];
    const int E = a.experts;
    const int64_t b = blockIdx.x;
    for (int e = threadIdx.x; e < E; e += 256) {
        int all = 0, earlier = 0;
        for (int64_t o = 0; o < blocks; ++o) {
            if (o == b) earlier = all;
            all += __popcll(a.masks[o * E + e]);
        }
        count[e] = all;
        before[e] = earlier;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        for (int e = 0; e < E; ++e) {
            start[e] = at;
            at += (count[e] + a.align - 1) / a.align * a.align;
        }
        start[E] = at;
    }
    __syncthreads();
    if (b == 0)
        for (int e = threadIdx.x; e <= E; e += 256) a.offsets[e] = start[e];
    // fillings: those of the experts b, b + blocks, ..., and a share of what is behind the last segment
    for (int64_t e = b; e < E; e += gridDim.x)
        for (int r = start[e] + count[e] + int(threadIdx.x); r < start[e + 1]; r += 256) a.row_tokens[r] = -1;
    for (int64_t r = start[E] + b * 256 + threadIdx.x; r < a.rows; r += int64_t(gridDim.x) * 256)
        a.row_tokens[r] = -1;
    for (int s = threadIdx.x; s < ROUTE_BLOCK * a.top_k; s += 256) {
        const int i = s / a.top_k;
        const int64_t t = b * ROUTE_BLOCK + i;
        if (t >= a.tokens) break;
        const int64_t slot = t * a.top_k + s % a.top_k;
        const int e = a.ids[slot];
        int place = -1;
        if (e >= 0) {
            place = start[e] + before[e] + __popcll(a.masks[b * E + e] & ((1ull << i) - 1));
            a.row_tokens[place] = int(t);
        }
        a.places[slot] = place;
    }
}

// One wave per token.  With p the scores, c the scale and g = c d_weights:
//   renormalised, S the sum of the chosen p: dp_i = (g_i - sum_j g_j p_j / S) / S for the chosen
//   sigmoid: dl_i = dp_i p_i (1 - p_i);  softmax: dl_i = p_i (dp_i - sum_j dp_j p_j)
template <int PER>
__global__ __launch_bounds__(WAVES * 64) void route_backward_kernel(RouteBackwardArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = int64_t(blockIdx.x) * WAVES + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const int E = a.experts;
    int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    if (id < 0 || id >= E) id = -1;
    const float g = id >= 0 ? a.scale * a.d_weights[t * a.top_k + lane] : 0.0f;
    const bool any = __ballot(id >= 0) != 0;
    float l[PER], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E && any ? load_logit(a.logits, t * a.ldl + e, a.type) : -INFINITY;
        top = fmaxf(top, l[i]);
    }
    const float mine = id >= 0 ? load_logit(a.logits, t * a.ldl + id, a.type) : -INFINITY;
    float sum = 1.0f, p;
    if (a.sigmoid) {
        p = id >= 0 ? 1.0f / (1.0f + expf(-mine)) : 0.0f;
    } else {
        // renormalised, the other experts' scores cancel: only the chosen matter
        if (a.renormalise) top = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        p = id >= 0 ? expf(mine - top) : 0.0f;
        if (!a.renormalise) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
            sum = wave_sum(sum);
            p /= sum;
        }
    }
    float dp = g;
    if (a.renormalise) {
        const float total = wave_sum(p);
        const float mean = total > 0.0f ? wave_sum(g * p) / total : 0.0f;
        dp = total > 0.0f ? (g - mean) / total : 0.0f;
    }
    float d;
    if (a.sigmoid) d = id >= 0 ? dp * p * (1.0f / (1.0f + expf(mine))) : 0.0f;
    else d = dp * p;
    const float inner = a.sigmoid || a.renormalise ? 0.0f : wave_sum(dp * p);
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        out[i] = inner != 0.0f && l[i] > -INFINITY ? -(expf(l[i] - top) / sum) * inner : 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        const int e = __shfl(id, j);
        const float v = __shfl(d, j);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e >= 0 && lane + 64 * i == e) out[i] += v;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        const int64_t at = t * a.ldd + e;
        if (a.type == 0) static_cast<float *>(a.d_logits)[at] = out[i];
        else if (a.type == 1) static_cast<uint16_t *>(a.d_logits)[at] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(out[i]));
        else static_cast<uint16_t *>(a.d_logits)[at] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(out[i]));
    }
}

template <int PER>
hipError_t go(const RouteArgs &r, hipStream_t stream) {
    RouteArgs a = r;
    const int64_t blocks = (a.tokens + ROUTE_BLOCK - 1) / ROUTE_BLOCK;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    if (blocks > 0) {
        void *args[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&choose_kernel<PER>),
                                             dim3(unsigned(blocks)), dim3(WAVES * 64), args, 0, stream);
        if (e != hipSuccess) return e;
    }
    if (a.offsets == nullptr) return hipSuccess;
    int64_t n = blocks;
    void *args[] = {&a, &n};
    return hipLaunchKernel(reinterpret_cast<const void *>(&place_kernel),
                           dim3(unsigned(blocks > 0 ? blocks : 1)), dim3(256), args, 0, stream);
}

template <int PER>
hipError_t go(const RouteBackwardArgs &r, hipStream_t stream) {
    RouteBackwardArgs a = r;
    const int64_t blocks = (a.tokens + WAVES - 1) / WAVES;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&route_backward_kernel<PER>),
                           dim3(unsigned(blocks)), dim3(WAVES * 64), args, 0, stream);
}

template <typename Args>
hipError_t by_experts(const Args &a, hipStream_t stream) {
    if (a.experts <= 64) return go<1>(a, stream);
    if (a.experts <= 128) return go<2>(a, stream);
    if (a.experts <= 256) return go<4>(a, stream);
    if (a.experts <= 512) return go<8>(a, stream);
    return go<16>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) { return by_experts(a, stream); }

hipError_t launch_route_backward(const RouteBackwardArgs &a, hipStream_t stream) {
    if (a.tokens == 0) return hipSuccess;
    return by_experts(a, stream);
}

}  // namespace libgemm
