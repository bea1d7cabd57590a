// Routing tokens to experts: scores, the choice, the weights, and the rows of
// each expert; and the weights' gradient.
//
// The choice.  One wave per token, or a quarter of one; lane l holds PER consecutive experts from
// PER*l on, so of equal keys the lowest lane's is the lowest index.  The
// largest key is found top_k times over the wave with data-parallel moves.
// Without a bias the logits rank as their scores do and are compared as they
// are.  With one, keys are computed in fp32, and where two that are compared
// lie closer than twice their error the token is chosen again in 64 bits:
// about one token in 500 of 256 experts, and ties.
//
// The rows.  A block of 64 tokens leaves one 64-bit mask per expert (bit t:
// token t of the block chose it), in which a token's rank among the block's
// is a count of bits; what earlier blocks hold comes from byte counts that the
// first kernel leaves.  No order of atomics enters a result.
//
// Both kernels are bound by latency at the sizes of a decode step and by
// instruction issue beyond; they read the logits once.  64 tokens of 256
// experts in 8 groups: 8.3 us and 3.2; 16384 tokens of 64: 8.5 and 6.4.  A
// token chosen again adds 4 us to such a decode step.
#include "f8_block.hpp"

#include <cmath>

namespace libgemm {
namespace {

constexpr int BLOCK = ROUTE_BLOCK;
constexpr int LANES = 64;
constexpr float NONE = -INFINITY;

__device__ inline float decode(uint16_t b, int type) {
    return type == 1 ? __builtin_bit_cast(float, uint32_t(b) << 16)
                     : static_cast<float>(__builtin_bit_cast(_Float16, b));
}
__device__ inline float load_logit(const void *x, int64_t at, int type) {
    if (type == 0) return static_cast<const float *>(x)[at];
    return decode(static_cast<const uint16_t *>(x)[at], type);
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
template <int N> struct Vec;
template <> struct Vec<1> { typedef uint16_t h; typedef float f; };
template <> struct Vec<2> { typedef u16x2_t h; typedef f32x2_t f; };
template <> struct Vec<4> { typedef u16x4_t h; typedef f32x4_t f; };
template <> struct Vec<8> { typedef u16x8_t h; };

// A lane's PER logits from element `at` on, `n` of them there (the others are
// -infinity).  whole: they may be read in vectors.
template <int PER>
__device__ inline void load_logits(const void *x, int64_t at, int type, int n, bool whole, float (&l)[PER]) {
    if (whole && n >= PER) {
        if (type == 0) {
            constexpr int W = PER < 4 ? PER : 4;
            typedef typename Vec<W>::f V;
#pragma unroll
            for (int i = 0; i < PER; i += W) {
                const V v = *reinterpret_cast<const V *>(static_cast<const float *>(x) + at + i);
                if constexpr (W == 1) l[i] = v;
                else
#pragma unroll
                    for (int j = 0; j < W; ++j) l[i + j] = v[j];
            }
        } else {
            constexpr int W = PER < 8 ? PER : 8;
            typedef typename Vec<W>::h V;
#pragma unroll
            for (int i = 0; i < PER; i += W) {
                const V v = *reinterpret_cast<const V *>(static_cast<const uint16_t *>(x) + at + i);
                if constexpr (W == 1) l[i] = decode(v, type);
                else
#pragma unroll
                    for (int j = 0; j < W; ++j) l[i + j] = decode(v[j], type);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = i < n ? load_logit(x, at + i, type) : NONE;
}

template <int PER>
__device__ inline void store_logits(void *x, int64_t at, int type, int n, bool whole, const float (&l)[PER]) {
    auto bits = [&](float v) {
        return type == 1 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v))
                         : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    };
    if (whole && n >= PER) {
        if (type == 0) {
            constexpr int W = PER < 4 ? PER : 4;
            typedef typename Vec<W>::f V;
#pragma unroll
            for (int i = 0; i < PER; i += W) {
                V v;
                if constexpr (W == 1) v = l[i];
                else
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = l[i + j];
                *reinterpret_cast<V *>(static_cast<float *>(x) + at + i) = v;
            }
        } else {
            constexpr int W = PER < 8 ? PER : 8;
            typedef typename Vec<W>::h V;
#pragma unroll
            for (int i = 0; i < PER; i += W) {
                V v;
                if constexpr (W == 1) v = bits(l[i]);
                else
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = bits(l[i + j]);
                *reinterpret_cast<V *>(static_cast<uint16_t *>(x) + at + i) = v;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i >= n) continue;
        if (type == 0) static_cast<float *>(x)[at + i] = l[i];
        else static_cast<uint16_t *>(x)[at + i] = bits(l[i]);
    }
}

// x of the lane that a data-parallel move of control CTRL names, `other`
// where there is none.
template <int CTRL, int ROWS>
__device__ inline float moved(float other, float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, other), __builtin_bit_cast(int, x),
                                           CTRL, ROWS, 0xf, false));
}
__device__ inline float lane_of(float x, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
// Over the wave, in every lane (row_shr 1, 2, 4, 8, then the rows' last lanes).
__device__ inline float wave_max(float x) {
    x = fmaxf(x, moved<0x111, 0xf>(x, x));
    x = fmaxf(x, moved<0x112, 0xf>(x, x));
    x = fmaxf(x, moved<0x114, 0xf>(x, x));
    x = fmaxf(x, moved<0x118, 0xf>(x, x));
    x = fmaxf(x, moved<0x142, 0xa>(x, x));
    x = fmaxf(x, moved<0x143, 0xc>(x, x));
    return lane_of(x, 63);
}
__device__ inline float wave_sum(float x) {
    x += moved<0x111, 0xf>(0.0f, x);
    x += moved<0x112, 0xf>(0.0f, x);
    x += moved<0x114, 0xf>(0.0f, x);
    x += moved<0x118, 0xf>(0.0f, x);
    x += moved<0x142, 0xa>(0.0f, x);
    x += moved<0x143, 0xc>(0.0f, x);
    return lane_of(x, 63);
}
__device__ inline int moved_int(int x, int by) {  // row_ror
    return by == 1   ? __builtin_amdgcn_update_dpp(0, x, 0x121, 0xf, 0xf, true)
           : by == 2 ? __builtin_amdgcn_update_dpp(0, x, 0x122, 0xf, 0xf, true)
           : by == 4 ? __builtin_amdgcn_update_dpp(0, x, 0x124, 0xf, 0xf, true)
                     : __builtin_amdgcn_update_dpp(0, x, 0x128, 0xf, 0xf, true);
}
__device__ inline float turned(float x, int by) {
    return __builtin_bit_cast(float, moved_int(__builtin_bit_cast(int, x), by));
}

// The lanes that share a token: a whole wave, or a row of 16 lanes of the
// data-parallel moves, four tokens to a wave.
template <int WIDTH>
struct Team;
template <>
struct Team<64> {
    static __device__ float max(float x) { return wave_max(x); }
    static __device__ float sum(float x) { return wave_sum(x); }
    static __device__ unsigned long long ballot(bool b, int) { return __ballot(b); }
    // x of place i.
    static __device__ float of(float x, int i, int) { return lane_of(x, i); }
    static __device__ int of(int x, int i, int) { return __builtin_amdgcn_readlane(x, i); }
    // x of the first lane where b is set (in one it is).
    static __device__ int first(bool b, int x) { return __builtin_amdgcn_readlane(x, __builtin_ctzll(__ballot(b))); }
};
template <>
struct Team<16> {
    static __device__ float max(float x) {
        x = fmaxf(x, turned(x, 1));
        x = fmaxf(x, turned(x, 2));
        x = fmaxf(x, turned(x, 4));
        return fmaxf(x, turned(x, 8));
    }
    static __device__ float sum(float x) {
        x += turned(x, 1);
        x += turned(x, 2);
        x += turned(x, 4);
        return x + turned(x, 8);
    }
    static __device__ unsigned long long ballot(bool b, int lane) { return __ballot(b) >> (lane & 48) & 0xffff; }
    static __device__ float of(float x, int i, int lane) { return __shfl(x, (lane & 48) + i); }
    static __device__ int of(int x, int i, int lane) { return __shfl(x, (lane & 48) + i); }
    static __device__ int first(bool b, int x) {  // x rises with the lane
        auto min = [](int p, int q) { return p < q ? p : q; };
        x = b ? x : 0x7fffffff;
        x = min(x, moved_int(x, 1));
        x = min(x, moved_int(x, 2));
        x = min(x, moved_int(x, 4));
        return min(x, moved_int(x, 8));
    }
};

// e^(a - b) with the rounding of the difference put back.
__device__ inline float exp_difference(float a, float b) {
    const float d = a - b, t = d - a;
    const float rest = (a - (d - t)) - (b + t);
    const float e = expf(d);
    return d > -126.0f ? __builtin_fmaf(e, rest, e) : e;  // (a rest of infinities is no number)
}

// The sigmoid of x over e^min(top, 0), for x <= top: e^min(x, 0) / (1 + e^-|x|)
// is the sigmoid, and e^min(top, 0) the largest's but for a factor of 1 to 2.
// Where e^-top passes 64 bits' range, and the sigmoid of top with it, 0.
constexpr float SIGMOID_ZERO = -709.7827f;  // the float below -ln of the largest 64-bit number
__device__ inline float relative_sigmoid(float x, float top) {
    const float w = exp_difference(fminf(x, 0.0f), fminf(top, 0.0f)) / (1.0f + expf(-fabsf(x)));
    return top > SIGMOID_ZERO ? w : 0.0f;
}

// ---- in 64 bits

// Over the wave, in every lane.
__device__ inline uint32_t wave_max(uint32_t x) {
    auto step = [&](int o) { x = uint32_t(o) > x ? uint32_t(o) : x; };
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x111, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x112, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x114, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x118, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x142, 0xa, 0xf, false));
    step(__builtin_amdgcn_update_dpp(int(x), int(x), 0x143, 0xc, 0xf, false));
    return __builtin_amdgcn_readlane(x, 63);
}
// The largest x of the wave, and the first lane that has it.  The bits of a
// number order as it does once a negative one's are all turned and a positive
// one's sign is, so the largest is found by reductions of their halves, which
// are far quicker than one of doubles.
__device__ inline double wave_max(double x, int &owner) {
    constexpr uint64_t SIGN = uint64_t(1) << 63;
    const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);  // (-0 as 0)
    const uint64_t order = b & SIGN ? ~b : b | SIGN;
    const uint32_t high = uint32_t(order >> 32), low = uint32_t(order);
    const uint32_t top_high = wave_max(high), top_low = wave_max(high == top_high ? low : 0u);
    owner = __builtin_ctzll(__ballot(high == top_high && low == top_low));
    const uint64_t top = uint64_t(top_high) << 32 | top_low;
    return __builtin_bit_cast(double, top & SIGN ? top ^ SIGN : ~top);
}
__device__ inline double lane_of(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(b), lane), hi = __builtin_amdgcn_readlane(uint32_t(b >> 32), lane);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// Lane j's choice (or -1) of a token whose scores are defined, over a whole wave.
template <int PER>
__device__ int choose_exactly(const RouteArgs &a, const float (&l)[PER], int lane) {
    const double none = -INFINITY;
    const int E = a.experts, first_e = lane * PER;
    double key[PER], sum = 0.0;
    float top = NONE;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
    if (!a.sigmoid) {
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += l[i] > NONE ? exp(double(l[i]) - double(top)) : 0.0;
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) sum += __shfl_xor(sum, d);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = none;
        if (!(l[i] > NONE)) continue;
        const double x = l[i];
        key[i] = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - double(top)) / sum;
        if (a.bias != nullptr) key[i] += double(a.bias[first_e + i]);
        if (!(key[i] > none)) key[i] = none;
    }
    int owner;
    if (a.groups > 1) {
        const int per = E / a.groups, width = per / PER;
        double rank = none;  // lane g's is group g's
        auto largest = [](double x, double y) { return x > y ? x : y; };
        auto smallest = [](double x, double y) { return x > y ? y : x; };
        if (per % PER == 0 && (width & (width - 1)) == 0) {
            double first = none, second = none;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                second = largest(second, smallest(first, key[i]));
                first = largest(first, key[i]);
            }
            for (int d = 1; d < width; d <<= 1) {
                const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
                second = largest(largest(second, s), smallest(first, f));
                first = largest(first, f);
            }
            if (a.group_top == 2 && second > none) first += second;
            rank = __shfl(first, lane * width & 63);
            if (lane >= a.groups) rank = none;
        } else {
            for (int g = 0; g < a.groups; ++g) {
                double first = none, second = none;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const double k = (first_e + i) / per == g ? key[i] : none;
                    second = largest(second, smallest(first, k));
                    first = largest(first, k);
                }
                double r = wave_max(first, owner);
                if (a.group_top == 2) {
                    int unused;
                    const double s = wave_max(lane == owner ? second : first, unused);
                    if (s > none) r += s;
                }
                if (lane == g) rank = r;
            }
        }
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double r = lane_of(rank, g);
            ahead += r > rank || (r == rank && g < lane);
        }
        const unsigned long long kept = __ballot(lane < a.groups && ahead < a.top_groups);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (first_e + i < E && !(kept >> ((first_e + i) / per) & 1)) key[i] = none;
    }
    if (a.bias == nullptr) {  // the logits rank as their scores do, and do not run together
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = key[i] > none ? double(l[i]) : none;
    }
    int id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        double mine = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) mine = key[i] > mine ? key[i] : mine;
        const double m = wave_max(mine, owner);
        if (!(m > none)) break;
        int at = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) at = key[i] == mine ? i : at;
        const int e = __builtin_amdgcn_readlane(first_e + at, owner);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (first_e + i == e) key[i] = none;
        if (lane == j) id = e;
    }
    return id;
}

// ---- in 32 bits

// The rank of group `place` of the team (its group_top largest keys' sum),
// -infinity in places without one, and what its error goes by.
template <int PER, int WIDTH>
__device__ inline void group_ranks(const RouteArgs &a, const float (&key)[PER], int lane, float &rank, float &size) {
    using T = Team<WIDTH>;
    const int place = lane & (WIDTH - 1);
    const int per = a.experts / a.groups, width = per / PER;
    auto join = [&](float first, float second, float &r, float &z) {
        const bool two = a.group_top == 2 && second > NONE;
        r = two ? first + second : first;
        z = first > NONE ? fabsf(first) + (two ? fabsf(second) : 0.0f) : 0.0f;
        // a sum past fp32 (two biases of its lowest value, say) is no rank: its error has no end
        if (two && fabsf(r) == INFINITY && fabsf(first) < INFINITY) {
            r = first;
            z = INFINITY;
        }
    };
    if (per % PER == 0 && width <= 16 && (width & (width - 1)) == 0) {
        // a group is `width` lanes, a power of two: its two largest come together in log2 steps
        float first = NONE, second = NONE;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            second = fmaxf(second, fminf(first, key[i]));
            first = fmaxf(first, key[i]);
        }
        for (int d = 1; d < width; d <<= 1) {
            const float f = __shfl_xor(first, d), s = __shfl_xor(second, d);
            second = fmaxf(fmaxf(second, s), fminf(first, f));
            first = fmaxf(first, f);
        }
        float r, z;
        join(first, second, r, z);
        const int from = (lane & ~(WIDTH - 1)) + (place * width & (WIDTH - 1));
        r = __shfl(r, from);
        z = __shfl(z, from);
        rank = place < a.groups ? r : NONE;
        size = z;
        return;
    }
    rank = NONE;
    size = 0.0f;
    for (int g = 0; g < a.groups; ++g) {
        float first = NONE, second = NONE;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float k = (place * PER + i) / per == g ? key[i] : NONE;
            second = fmaxf(second, fminf(first, k));
            first = fmaxf(first, k);
        }
        const float m = T::max(first);
        const int at = T::first(first == m, place);
        const float s = T::max(place == at ? second : first);
        float r, z;
        join(m, s, r, z);
        if (place == g) {
            rank = r;
            size = z;
        }
    }
}

// Chooses for token t (in a team without one, live is not set): place j of
// the team gets choice j and its weight.
template <int PER, int WIDTH>
__device__ inline void choose(const RouteArgs &a, int64_t t, bool live, int lane, bool whole, int &id, float &w) {
    using T = Team<WIDTH>;
    const int E = a.experts, place = lane & (WIDTH - 1), first_e = place * PER;
    id = -1;
    w = 0.0f;
    if (live && a.keep != nullptr) live = a.keep[t] != 0;
    if (WIDTH == 64 && !live) return;
    float l[PER], key[PER];
    load_logits<PER>(a.logits, t * a.ldl + first_e, a.type, live ? E - first_e : 0, whole, l);
    float top = NONE;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        odd = odd || l[i] != l[i] || l[i] == INFINITY;
        l[i] = l[i] > NONE ? l[i] : NONE;
        top = fmaxf(top, l[i]);
    }
    float sum = 0.0f;
    bool undefined = false;
    if (!a.sigmoid) {
        undefined = T::ballot(odd, lane) != 0;
        if (undefined) {
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = NONE;
            top = NONE;
        }
        top = T::max(top);
        if (a.bias != nullptr || !a.renormalise || (a.groups > 1 && a.group_top == 2)) {
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += l[i] > NONE ? expf(l[i] - top) : 0.0f;
            sum = T::sum(sum);
        }
    }
    // The error of a key is below off * (the largest score + its own size).
    // Sigmoid: e^-l within 1 ulp, 1 + e and the quotient rounded: 2 steps of
    // 2^-24 at most in a score of 1, and one of the sum with the bias.
    // Softmax: per score the rounding of l - top (weighted by e^(l - top), at
    // most 0.4 steps), e within 2, the quotient, and the sum: 2 per term, 7 for
    // the terms' arguments (their mean is the entropy, at most ln 1024) and
    // PER + 6 additions.
    const float off = (a.sigmoid ? 2.25f : PER + 20.0f) * 0x1p-24f;
    const float largest = a.sigmoid ? 1.0f : 1.0f / sum;
    const bool exact_keys = a.bias == nullptr;
    bool near = false;
    if (exact_keys && !(a.groups > 1 && a.group_top == 2)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = l[i];
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = a.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - top) / sum;
            if (a.bias != nullptr && first_e + i < E) key[i] += a.bias[first_e + i];
            key[i] = l[i] > NONE && key[i] > NONE ? key[i] : NONE;
        }
    }
    if (a.groups > 1) {
        const int per = E / a.groups;
        const bool exact_ranks = exact_keys && a.group_top == 1;
        float rank, size;
        group_ranks<PER, WIDTH>(a, key, lane, rank, size);
        const float error = off * (2.0f * largest + 2.0f * size);  // two keys, and their sum's rounding
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float r = T::of(rank, g, lane);
            ahead += r > rank || (r == rank && g < place);
            if (!exact_ranks && g != place && place < a.groups && fabsf(r - rank) <= error + T::of(error, g, lane))
                near = true;
        }
        const unsigned long long kept = T::ballot(place < a.groups && ahead < a.top_groups, lane);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int g = (first_e + i) / per;
            const bool in = first_e + i < E && (kept >> (g & 63) & 1);
            key[i] = !in || !(key[i] > NONE) ? NONE : exact_keys ? l[i] : key[i];
        }
    }
    float last = INFINITY;
    const int rounds = exact_keys || a.top_k == E ? a.top_k : a.top_k + 1;  // one more shows how close the next is
    for (int j = 0; j < rounds; ++j) {
        float mine = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) mine = fmaxf(mine, key[i]);
        const float m = T::max(mine);
        if (WIDTH == 64 ? !(m > NONE) : __ballot(m > NONE) == 0) break;
        if (!exact_keys && m > NONE && last - m <= 2.0f * off * (largest + fabsf(m))) near = true;
        last = m;
        int at = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) at = key[i] == m ? i : at;
        const int e = T::first(mine == m, first_e + at);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (first_e + i == e) key[i] = NONE;
        if (place == j && m > NONE) id = e;
    }
    if (place >= a.top_k) id = -1;
    unsigned long long again = __ballot(near);
    if (again != 0) {
        constexpr int PER64 = PER * WIDTH / 64 > 0 ? PER * WIDTH / 64 : 1;
        for (int team = 0; team < 64 / WIDTH; ++team) {
            if ((again >> (team * (WIDTH & 63)) & (WIDTH == 64 ? ~0ull : 0xffffull)) == 0) continue;
            const int64_t token = __shfl(t, team * (WIDTH & 63));
            float x[PER64];
            load_logits<PER64>(a.logits, token * a.ldl + lane * PER64, a.type, E - lane * PER64, false, x);
#pragma unroll
            for (int i = 0; i < PER64; ++i) x[i] = x[i] > NONE ? x[i] : NONE;
            const int chosen = choose_exactly<PER64>(a, x, lane);
            const int mine = __shfl(chosen, place);
            if (lane / WIDTH == team) id = mine;
        }
    }

    const float x = id >= 0 ? load_logit(a.logits, t * a.ldl + id, a.type) : NONE;
    // renormalised: relative to the largest chosen, so the sum cannot vanish
    if (a.renormalise) top = T::max(x);
    if (a.sigmoid) {
        w = id < 0 ? 0.0f : a.renormalise ? relative_sigmoid(x, top) : 1.0f / (1.0f + expf(-x));
    } else {
        w = id >= 0 ? exp_difference(x, top) : 0.0f;
        if (!a.renormalise && id >= 0) w /= sum;
    }
    if (a.renormalise) {
        const float total = T::sum(w);
        w = total > 0.0f ? w / total : 0.0f;
    }
    w *= a.scale;
    if (id < 0) w = 0.0f;
    if (undefined) w = __builtin_nanf("");
}

__host__ __device__ inline int64_t count_pitch(int64_t experts) { return (experts + 3) / 4 * 4; }

// Waves per workgroup at most.  16 experts per lane spill where 16 waves share
// the registers (65536 tokens of 256 experts, four per wave: 155 us, with 8
// waves 139); 8 per lane spill a little and still gain by 16 (of 512 experts,
// one per wave: 240 us, with 8 waves 318).
constexpr int choose_waves(int per) { return per >= 16 ? 8 : 16; }

// `span` consecutive tokens per workgroup, its teams taking them in turn.
// With counts: counts[workgroup][expert], the tokens of the span that chose it.
template <int PER, int WIDTH>
__global__ __launch_bounds__(choose_waves(PER) * 64) void choose_kernel(RouteArgs a, int span, uint8_t *counts) {
    __shared__ uint32_t count[ROUTE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int TEAMS = 64 / WIDTH;  // per wave
    const int step = (blockDim.x >> 6) * TEAMS, place = lane & (WIDTH - 1);
    if (counts != nullptr) {
        for (int e = threadIdx.x; e < a.experts; e += blockDim.x) count[e] = 0;
        __syncthreads();
    }
    // rows of logits that start where their vectors are aligned
    const int64_t bytes = int64_t(PER < 4 ? PER : 4) * 4;
    const bool whole = (reinterpret_cast<uintptr_t>(a.logits) | uint64_t(a.ldl * (a.type == 0 ? 4 : 2))) % bytes == 0;
    for (int i = wave * TEAMS; i < span; i += step) {
        const int64_t t0 = int64_t(blockIdx.x) * span + i;
        if (t0 >= a.tokens) break;
        const int64_t t = TEAMS == 1 ? t0 : t0 + lane / WIDTH;
        const bool live = TEAMS == 1 || (t < a.tokens && i + lane / WIDTH < span);
        int id;
        float w;
        choose<PER, WIDTH>(a, live ? t : t0, live, lane, whole, id, w);
        if (live && place < a.top_k) {
            a.ids[t * a.top_k + place] = id;
            a.weights[t * a.top_k + place] = w;
            if (counts != nullptr && id >= 0) atomicAdd(&count[id], 1u);
        }
    }
    if (counts != nullptr) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
            counts[blockIdx.x * count_pitch(a.experts) + e] = uint8_t(count[e]);
    }
}

// Workgroup g lays out the 64-token blocks from g*own on, `own` of them.
// counts: one row of E bytes, made up to whole words, per `span` tokens (a
// divisor of 64), or null when there is one block, which then counts for
// itself.
__global__ __launch_bounds__(1024) void place_kernel(RouteArgs a, int64_t own, int span, const uint8_t *counts) {
    constexpr int THREADS = 1024;
    __shared__ unsigned long long mask[ROUTE_MAX_EXPERTS];
    __shared__ int start[ROUTE_MAX_EXPERTS + 1];  // offsets
    __shared__ int total[ROUTE_MAX_EXPERTS];
    __shared__ int next[ROUTE_MAX_EXPERTS];  // rows of earlier blocks
    __shared__ int wave_total[THREADS / 64];
    const int E = a.experts, tid = threadIdx.x, lane = tid & 63;
    const int64_t first_block = int64_t(blockIdx.x) * own;
    // A block's slots, by thread: their experts, on their way while the counts are read.
    constexpr int SLOTS = BLOCK * ROUTE_MAX_TOP_K / THREADS;
    int chosen[SLOTS];
    auto load_ids = [&](int64_t block) {
        const int64_t t0 = block * BLOCK;
        const int slots = t0 < a.tokens ? int((a.tokens - t0 < BLOCK ? a.tokens - t0 : BLOCK) * a.top_k) : 0;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) chosen[i] = tid + i * THREADS < slots ? a.ids[t0 * a.top_k + tid + i * THREADS] : -1;
        return slots;
    };
    auto fill_masks = [&]() {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (chosen[i] >= 0) atomicOr(&mask[chosen[i]], 1ull << ((tid + i * THREADS) / a.top_k));
    };
    int slots = load_ids(first_block);
    for (int e = tid; e < E; e += THREADS) {
        mask[e] = 0;
        total[e] = next[e] = 0;
    }
    __syncthreads();
    if (counts == nullptr) {
        fill_masks();
        __syncthreads();
        for (int e = tid; e < E; e += THREADS) total[e] = __popcll(mask[e]);
    } else {
        // four experts' bytes at a time
        const int64_t rows = (a.tokens + span - 1) / span, before = first_block * BLOCK / span;
        const int quads = (E + 3) / 4, parts = THREADS / quads;
        const int q = tid % quads, part = tid / quads;
        if (part < parts) {
            int sum[4] = {0, 0, 0, 0}, early[4] = {0, 0, 0, 0};
            for (int64_t r = part; r < rows; r += parts) {
                const uint32_t v = reinterpret_cast<const uint32_t *>(counts)[r * quads + q];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = v >> (8 * i) & 255;
                    sum[i] += c;
                    early[i] += r < before ? c : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * q + i >= E) break;
                atomicAdd(&total[4 * q + i], sum[i]);
                atomicAdd(&next[4 * q + i], early[i]);
            }
        }
    }
    __syncthreads();
    // the segments' starts: a scan of the aligned totals, one expert per thread (E <= THREADS)
    {
        const int64_t len = tid < E ? (int64_t(total[tid]) + a.align - 1) / a.align * a.align : 0;
        int sum = int(len);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 63) wave_total[tid >> 6] = sum;
        __syncthreads();
        int add = 0;
        for (int w = 0; w < tid >> 6; ++w) add += wave_total[w];
        if (tid < E) start[tid + 1] = add + sum;
        if (tid == 0) start[0] = 0;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += THREADS) a.offsets[e] = start[e];
    // fillings, a wave each: experts g, g + grid, ..., and a share of what is behind the last segment
    if (a.align > 1)
        for (int64_t e = int64_t(blockIdx.x) * (THREADS / 64) + (tid >> 6); e < E; e += int64_t(gridDim.x) * (THREADS / 64)) {
            // (counted from the filling's start: rows end at 2^31)
            const int from = start[e] + total[e], n = start[e + 1] - from;
            for (int i = lane; i < n; i += 64) a.row_tokens[int64_t(from) + i] = -1;
        }
    for (int64_t r = start[E] + int64_t(blockIdx.x) * THREADS + tid; r < a.rows; r += int64_t(gridDim.x) * THREADS)
        a.row_tokens[r] = -1;
    for (int64_t block = first_block; block < first_block + own && block * BLOCK < a.tokens; ++block) {
        const int64_t t0 = block * BLOCK;
        if (block > first_block) {
            slots = load_ids(block);
            __syncthreads();
            for (int e = tid; e < E; e += THREADS) {
                next[e] += __popcll(mask[e]);
                mask[e] = 0;
            }
            __syncthreads();
        }
        if (counts != nullptr) {
            fill_masks();
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int s = tid + i * THREADS, bit = s / a.top_k, e = chosen[i];
            if (s >= slots) continue;
            int place = -1;
            if (e >= 0) {
                place = start[e] + next[e] + __popcll(mask[e] & ((1ull << bit) - 1));
                a.row_tokens[place] = int(t0 + bit);
            }
            a.places[t0 * a.top_k + s] = place;
        }
    }
}

// A wave or a quarter of one per token.  With p the scores, c the scale and g = c d_weights:
//   d_i = p_i g_i for the chosen; renormalised, S the sum of their p: (p_i / S) (g_i - sum_j g_j p_j / S)
//   sigmoid: dl_i = d_i (1 - p_i);  softmax: dl_i = d_i - p_i sum_j d_j
// (renormalised softmax: the d_i sum to 0).  In a share p_i / S any common factor of the p cancels.
// Bound by the loads' latency: 16384 tokens of 128 experts 5.9 to 7 us, 1.3 to 1.6 TB/s.
constexpr int BACK_WAVES = 4;
template <int PER, int WIDTH>
__global__ __launch_bounds__(BACK_WAVES * 64) void route_backward_kernel(RouteBackwardArgs a) {
    using T = Team<WIDTH>;
    constexpr int TEAMS = 64 / WIDTH;  // tokens per wave
    const int lane = threadIdx.x & 63, place = lane & (WIDTH - 1);
    const int64_t t0 = (int64_t(blockIdx.x) * BACK_WAVES + (threadIdx.x >> 6)) * TEAMS;
    if (t0 >= a.tokens) return;
    const bool live = t0 + lane / WIDTH < a.tokens;
    const int64_t t = live ? t0 + lane / WIDTH : t0;
    const int E = a.experts, first_e = place * PER;
    const int esize = a.type == 0 ? 4 : 2;
    const int64_t bytes = int64_t(PER < 4 ? PER : 4) * 4;
    auto aligned = [&](const void *x, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(x) | uint64_t(ld * esize)) % bytes == 0;
    };
    // every logit has a gradient: they are on their way while the ids arrive
    const bool dense = !a.sigmoid && !a.renormalise;
    float l[PER], top = NONE;
    if (dense) {
        load_logits<PER>(a.logits, t * a.ldl + first_e, a.type, E - first_e, aligned(a.logits, a.ldl), l);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = NONE;
    }
    int id = live && place < a.top_k ? a.ids[t * a.top_k + place] : -1;
    float g = live && place < a.top_k ? a.d_weights[t * a.top_k + place] : 0.0f;
    if (id < 0 || id >= E) id = -1;
    g = id >= 0 ? a.scale * g : 0.0f;
    const bool any = T::ballot(id >= 0, lane) != 0;
    const float mine = id >= 0 ? load_logit(a.logits, t * a.ldl + id, a.type) : NONE;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (!any) l[i] = NONE;  // nothing flows, whatever the logits are
        top = fmaxf(top, l[i]);
    }
    float p;
    // renormalised, the other experts' scores cancel: only the chosen matter
    top = T::max(a.renormalise ? mine : top);
    if (a.sigmoid) {
        p = id < 0 ? 0.0f : a.renormalise ? relative_sigmoid(mine, top) : 1.0f / (1.0f + expf(-mine));
    } else {
        p = id >= 0 ? expf(mine - top) : 0.0f;
        if (dense) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                l[i] = l[i] > NONE ? expf(l[i] - top) : l[i] != l[i] ? l[i] : 0.0f;
                sum += l[i];
            }
            sum = T::sum(sum);
            const float inverse = any ? 1.0f / sum : 0.0f;
            p *= inverse;
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] *= inverse;
        }
    }
    float d = g * p;
    if (a.renormalise) {  // the share first: g over a vanishing S would leave fp32
        const float total = T::sum(p), share = total > 0.0f ? p / total : 0.0f;
        d = share * (g - T::sum(g * share));
    }
    if (a.sigmoid) d = id >= 0 ? d * (1.0f / (1.0f + expf(mine))) : 0.0f;
    const float inner = dense ? T::sum(d) : 0.0f;
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] = dense ? -l[i] * inner : 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        const int e = T::of(id, j, lane);
        const float v = T::of(d, j, lane);
#pragma unroll
        for (int i = 0; i < PER; ++i) out[i] += first_e + i == e ? v : 0.0f;
    }
    store_logits<PER>(a.d_logits, t * a.ldd + first_e, a.type, live ? E - first_e : 0, aligned(a.d_logits, a.ldd), out);
}

// Threads of a launch, which has fewer than 2^32: more tokens take several.
constexpr int64_t LAUNCH_THREADS = int64_t(1) << 31;

template <int PER, int WIDTH>
hipError_t back_go(const RouteBackwardArgs &r, hipStream_t stream) {
    constexpr int TOKENS = BACK_WAVES * 64 / WIDTH;
    constexpr int64_t step = LAUNCH_THREADS / (BACK_WAVES * 64) * TOKENS;
    const int esize = r.type == 0 ? 4 : 2;
    for (int64_t t = 0; t < r.tokens; t += step) {
        RouteBackwardArgs a = r;
        a.tokens = r.tokens - t < step ? r.tokens - t : step;
        a.logits = static_cast<const char *>(r.logits) + t * r.ldl * esize;
        a.ids = r.ids + t * r.top_k;
        a.d_weights = r.d_weights + t * r.top_k;
        a.d_logits = static_cast<char *>(r.d_logits) + t * r.ldd * esize;
        void *args[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&route_backward_kernel<PER, WIDTH>),
                                             dim3(unsigned((a.tokens + TOKENS - 1) / TOKENS)), dim3(BACK_WAVES * 64),
                                             args, 0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int PER, int WIDTH>
hipError_t choose_go(const RouteArgs &r, int span, uint8_t *counts, hipStream_t stream) {
    const int tokens_per_wave = 64 / WIDTH, all = (span + tokens_per_wave - 1) / tokens_per_wave;
    const int waves = all < choose_waves(PER) ? all : choose_waves(PER);
    const int64_t step = LAUNCH_THREADS / (choose_waves(PER) * 64) * span;
    for (int64_t t = 0; t < r.tokens; t += step) {
        RouteArgs a = r;
        a.tokens = r.tokens - t < step ? r.tokens - t : step;
        a.logits = static_cast<const char *>(r.logits) + t * r.ldl * (r.type == 0 ? 4 : 2);
        if (r.keep != nullptr) a.keep = r.keep + t;
        a.ids = r.ids + t * r.top_k;
        a.weights = r.weights + t * r.top_k;
        uint8_t *counted = counts == nullptr ? nullptr : counts + t / span * count_pitch(r.experts);
        void *args[] = {&a, &span, &counted};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&choose_kernel<PER, WIDTH>),
                                             dim3(unsigned((a.tokens + span - 1) / span)), dim3(unsigned(waves) * 64),
                                             args, 0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Tokens from which four share a wave, where 16 lanes hold a token's experts:
// 16384 tokens of 64 experts 21 -> 14 us, their gradient of 128 9.0 -> 6.6;
// with fewer tokens compute units are idle and a whole wave is done sooner
// (64 tokens of 256 experts 11.5 us, by fours 16.5).
constexpr int64_t TEAMS_FROM = 512;

hipError_t choose_by_size(const RouteArgs &a, int span, uint8_t *counts, hipStream_t stream) {
    if (a.tokens >= TEAMS_FROM && a.experts <= 256 && a.top_k <= 16 && a.groups <= 16) {
        if (a.experts <= 16) return choose_go<1, 16>(a, span, counts, stream);
        if (a.experts <= 32) return choose_go<2, 16>(a, span, counts, stream);
        if (a.experts <= 64) return choose_go<4, 16>(a, span, counts, stream);
        if (a.experts <= 128) return choose_go<8, 16>(a, span, counts, stream);
        return choose_go<16, 16>(a, span, counts, stream);
    }
    if (a.experts <= 64) return choose_go<1, 64>(a, span, counts, stream);
    if (a.experts <= 128) return choose_go<2, 64>(a, span, counts, stream);
    if (a.experts <= 256) return choose_go<4, 64>(a, span, counts, stream);
    if (a.experts <= 512) return choose_go<8, 64>(a, span, counts, stream);
    return choose_go<16, 64>(a, span, counts, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs &r, hipStream_t stream) {
    RouteArgs a = r;
    const bool layout = a.offsets != nullptr;
    const int64_t blocks = (a.tokens + BLOCK - 1) / BLOCK;
    // A workgroup's tokens: few while that leaves most of the chip empty.
    int span = a.tokens <= BLOCK ? 4 : a.tokens <= 4096 ? 16 : BLOCK;
    uint8_t *counts = layout && a.tokens > BLOCK ? static_cast<uint8_t *>(a.workspace) : nullptr;
    if (a.tokens > 0) {
        const hipError_t e = choose_by_size(a, span, counts, stream);
        if (e != hipSuccess) return e;
    }
    if (!layout) return hipSuccess;
    // every workgroup reads all counts: at most 256 of them, so that this does not grow with the square
    int64_t own = (blocks + 255) / 256;
    if (own < 1) own = 1;
    const int64_t grid = blocks > 0 ? (blocks + own - 1) / own : 1;
    const uint8_t *read = counts;
    void *args[] = {&a, &own, &span, &read};
    return hipLaunchKernel(reinterpret_cast<const void *>(&place_kernel), dim3(unsigned(grid)), dim3(1024), args, 0, stream);
}

hipError_t launch_route_backward(const RouteBackwardArgs &a, hipStream_t stream) {
    if (a.tokens == 0) return hipSuccess;
    if (a.tokens >= TEAMS_FROM && a.experts <= 256 && a.top_k <= 16) {
        if (a.experts <= 16) return back_go<1, 16>(a, stream);
        if (a.experts <= 32) return back_go<2, 16>(a, stream);
        if (a.experts <= 64) return back_go<4, 16>(a, stream);
        if (a.experts <= 128) return back_go<8, 16>(a, stream);
        return back_go<16, 16>(a, stream);
    }
    if (a.experts <= 64) return back_go<1, 64>(a, stream);
    if (a.experts <= 128) return back_go<2, 64>(a, stream);
    if (a.experts <= 256) return back_go<4, 64>(a, stream);
    if (a.experts <= 512) return back_go<8, 64>(a, stream);
    return back_go<16, 64>(a, stream);
}

size_t route_workspace(int64_t tokens, int64_t experts) {
    // a row of byte counts for each span of tokens, at most one per 16
    const size_t rows = tokens <= 4096 ? size_t((tokens + 15) / 16) : size_t((tokens + BLOCK - 1) / BLOCK);
    return ((rows > 0 ? rows : 1) * size_t(count_pitch(experts)) + 15) / 16 * 16;
}

}  // namespace libgemm
