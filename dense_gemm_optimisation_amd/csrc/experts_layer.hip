// A whole layer of experts for a few tokens (gemm_experts_layer), in two
// kernels that read the live experts' weights once.
//
//   up_kernel    w h, h = act(Up[0 .. H) x) * (Up[H .. 2H) x): a workgroup takes
//                blocks of 16 of H's rows, both halves, of an expert, for up
//                to XR of the tokens that chose it.  w h leaves as two
//                16-bit pieces, hi + lo, so it is not rounded to 16 bits in
//                between;
//   down_kernel  y = sum over the token's experts of Down (w h): a workgroup
//                has 16 of y's columns for all tokens and goes through
//                every live expert, its waves dealing (expert, run of H) pairs,
//                so a token's weighted sum is formed in one place and one order:
//                no atomics.
//
// Bound by reading the weights, so each wave keeps the next runs of its 16
// rows on their way into its own part of LDS, 128 bytes of each row at a time, by direct
// loads that take eight whole lines; the eight waves of a workgroup take
// neighbouring runs, 1 KiB of each row together.  (Loads in the
// matrix instruction's own order, 16 bytes of 16 rows, kept the address unit
// busy for 51 cycles each: 32 tokens of 64 experts of 1024 x 4096 in 8 bits took 131 and 95 us
// that way.)  The activations come the same way, behind the weights: then
// only these loads are counted, and waiting for one run leaves the later ones in flight.
// The 16 x 16 x 32 matrix instruction takes the weights as its 16-row
// operand and the tokens as the other; 8-bit codes are widened exactly on the way
// from LDS, and a run of 128 has one scale.
//
// 64 experts of 1024 x 4096: one token of eight in bf16 30 + 17 us (4.3 TB/s), 32
// tokens in 8 bits 115 + 82 us (100 to 143 and 77 to 87; 4.1 TB/s: there widening
// and the short runs' latency count too, without memory 78 and 75).
//
// Each workgroup finds the live experts and their tokens from the ids by
// itself (at most 2048 of them, from L2), which saves a launch.
#include "activation.hpp"
#include "layers.hpp"
#include "tile16.hpp"

namespace libgemm {
namespace {

using namespace tile16;

constexpr int WAVES = 8, THREADS = WAVES * 64;

template <int TYPE>
struct Form {
    static constexpr int ESZ = TYPE == 0 ? 2 : 1;  // bytes of a weight
    static constexpr int PER = 16 / ESZ;           // weights per 16-byte chunk
    static constexpr int RUN = 128 / ESZ;          // k of a run: 128 bytes of a row
    static constexpr int STEPS = RUN / 32;         // matrix instructions
    // A run's scales come with it, a float for each lane.
    static constexpr int SCALES = TYPE == 0 ? 0 : 1, SCALE_BYTES = SCALES * 256;
};

struct LayerArgs {
    ExpertsLayer p;
    // w h of each choice: [token * top_k + choice][run][piece][RUN] of X's type; a token's first choice
    // of an expert has all of its weights for it
    uint16_t *h;
    int64_t ldh;  // elements of a choice
    int ring_up, ring_down;
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

// The two pieces of w h: hi of w h * TIMES, and lo of what hi leaves out * REST.
// fp16 has a few powers of two more below w h's usual values than above them;
// lo is as large as hi, so it is a subnormal only where hi is.
template <class T>
struct Pieces {
    static constexpr float TIMES = __is_same(T, F16) ? 0x1p-4f : 1.0f, REST = __is_same(T, F16) ? 0x1p11f : 1.0f;
};

// Lane q of four (lane / 16) has eight k of each step: 16-bit weights those
// of chunk 4s + q, 32s + 8q; codes half s % 2 of chunk 4(s / 2) + q, 64(s / 2) + 16q +
// 8(s % 2); the activations in the same order, by their own chunks of 8.
template <int TYPE>
__device__ inline int k_of(int s, int q) {
    return TYPE == 0 ? 32 * s + 8 * q : 64 * (s / 2) + 16 * q + 8 * (s % 2);
}
// Zeros for the values at K and beyond of eight that start at k.
__device__ inline void cut(u32x4 &w, int k, int K) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e >= K) w[e / 2] &= e % 2 ? 0xffffu : 0xffff0000u;
}

// p is the same in the whole wave.
__device__ inline u32x4 buffer_at(const void *p) {
    return dma::raw_buffer(static_cast<uint64_t>(uniform(reinterpret_cast<int64_t>(p))), 0x7fffffff);
}
// direct_load16 from `soffset` bytes further on: a run's place in its rows,
// without a descriptor of its own.
__device__ inline void direct_load16_at(u32x4 rs, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(voffset), "s"(rs), "s"(soffset)
        : "memory", "m0");
}

// 16 rows of a run of weights in LDS: 128 bytes per row, chunk c of row r at
// c ^ swz(r).  Two direct loads of eight rows.
template <int TYPE>
struct Rows {
    uint32_t voff[2];
    int chunk[2];  // first k of this lane's chunk

    // `rows` rows are there; the others are copies of the last.
    __device__ void init(int64_t ld, int64_t rows, int lane) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * j + lane / 8, c = (lane % 8) ^ swz_k<8>(r);
            voff[j] = uint32_t((r < rows ? r : rows - 1) * ld * Form<TYPE>::ESZ) + c * 16;
            chunk[j] = c * Form<TYPE>::PER;
        }
    }
    // left: values from the run's first one
    __device__ void issue(u32x4 rs, uint32_t soffset, uint32_t to, int left) const {
        if (left >= Form<TYPE>::RUN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) direct_load16_at(rs, to + j * 1024, voff[j], soffset);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) direct_load16_at(rs, to + j * 1024, chunk[j] < left ? voff[j] : OOB, soffset);
        }
    }
    template <class T>
    static __device__ u32x4 operand(const LDS char *at, int s, int r, int q) {
        const int c = TYPE == 0 ? 4 * s + q : 4 * (s / 2) + q;
        const u32x4 v = *reinterpret_cast<const LDS u32x4 *>(at + r * 128 + ((c ^ swz_k<8>(r)) << 4));
        if constexpr (TYPE == 0) return v;
        else return s % 2 ? widen<T, TYPE>(v[2], v[3]) : widen<T, TYPE>(v[0], v[1]);
    }
};

// N rows of activations in LDS, BYTES (128, 256 or 512) per row, 16-byte
// chunk c of row r at c ^ f(r), f(r) = swz(r) in rows of 128 bytes, r else.
template <int N, int BYTES>
struct Values {
    static constexpr int LOADS = N * BYTES / 1024, CHUNKS = BYTES / 16, PER_LOAD = 64 / CHUNKS;
    static constexpr int SIZE = N * BYTES;
    static_assert(LOADS >= 1 && N * BYTES % 1024 == 0, "whole loads");
    uint32_t voff[LOADS];
    int chunk[LOADS];
    static __device__ int swizzle(int r) { return BYTES == 128 ? swz_k<8>(r) : r & 15; }
    static __device__ int row_of(int j, int lane) { return j * PER_LOAD + lane / CHUNKS; }
    // start(r): byte offset of row r
    template <class F>
    __device__ void init(int lane, F &&start) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int r = row_of(j, lane), c = (lane % CHUNKS) ^ swizzle(r);
            chunk[j] = c;
            voff[j] = start(r) + c * 16;
        }
    }
    // whole: every chunk is read; else those of which live(c), others are zeros
    template <class F>
    __device__ void issue(u32x4 rs, uint32_t soffset, uint32_t to, bool whole, F &&live) const {
        if (whole) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) direct_load16_at(rs, to + j * 1024, voff[j], soffset);
        } else {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) direct_load16_at(rs, to + j * 1024, live(chunk[j]) ? voff[j] : OOB, soffset);
        }
    }
    static __device__ u32x4 at(const LDS char *base, int r, int c) {
        return *reinterpret_cast<const LDS u32x4 *>(base + r * BYTES + ((c ^ swizzle(r)) << 4));
    }
};

// Waits until at most `later` stages of PER loads are in flight (later < 4).
template <int PER>
__device__ inline void wait_for(int later) {
    if (later >= 3) wait_vmcnt<3 * PER>();
    else if (later == 2) wait_vmcnt<2 * PER>();
    else if (later == 1) wait_vmcnt<PER>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
}

// What a workgroup finds out from the ids, in LDS: where each expert's
// choices (a token's first one of it) start, and its groups of up to `size` of them.
struct Found {
    LDS int32_t *choices;  // [experts + 1]: where they end, behind a 0
    LDS int16_t *groups;   // [experts + 1], the same of groups
    LDS int16_t *ids;      // [slots], -1: no expert
    __device__ Found(LDS char *at, int64_t experts)
        : choices(reinterpret_cast<LDS int32_t *>(at)), groups(reinterpret_cast<LDS int16_t *>(choices + experts + 1)),
          ids(groups + experts + 1) {}
};
int64_t found_bytes(const ExpertsLayer &p) { return 6 * (p.experts + 1) + 2 * p.tokens * p.top_k; }

// Token t's first choice of expert e, or -1.
__device__ inline int choice_of(const LDS int16_t *ids, int t, int k, int e) {
    int first = -1;
    for (int j = k - 1; j >= 0; --j)
        if (ids[t * k + j] == e) first = j;
    return first;
}

// All threads of the workgroup call it.
__device__ void find(const ExpertsLayer &p, const Found &f, int size) {
    const int E = int(p.experts), k = int(p.top_k), slots = int(p.tokens) * k;
    for (int i = threadIdx.x; i <= E; i += THREADS) f.choices[i] = 0;
    for (int i = threadIdx.x; i < slots; i += THREADS) {
        const uint32_t e = uint32_t(p.ids[i]);
        f.ids[i] = e < uint32_t(E) ? int16_t(e) : int16_t(-1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += THREADS) {
        const int e = f.ids[i];
        if (e < 0) continue;
        bool first = true;
        for (int j = i - i % k; j < i; ++j) first = first && f.ids[j] != e;
        if (first) __hip_atomic_fetch_add(f.choices + e + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        // running sums, 64 experts at a time
        const int lane = threadIdx.x;
        int choices = 0, groups = 0;
        if (lane == 0) f.groups[0] = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            int c = e < E ? f.choices[e + 1] : 0, g = (c + size - 1) / size;
            for (int d = 1; d < 64; d *= 2) {
                const int oc = __shfl_up(c, d), og = __shfl_up(g, d);
                if (lane >= d) c += oc, g += og;
            }
            if (e < E) {
                f.choices[e + 1] = choices + c;
                f.groups[e + 1] = int16_t(groups + g);
            }
            choices += __shfl(c, 63);
            groups += __shfl(g, 63);
        }
    }
    __syncthreads();
}

// XR: tokens of a group at most.  The blocks of 16 rows of all groups are dealt
// to the workgroups in equal shares, one workgroup per compute unit: finding
// the experts takes 4 us, which a workgroup for every few blocks would pay over
// and over.
template <class T, int TYPE, int XR>
__global__ __launch_bounds__(THREADS, 1) void up_kernel(LayerArgs a) {
    using F = Form<TYPE>;
    using X = Values<XR, F::RUN * 2>;
    constexpr int STAGE = 4096 + X::SIZE + F::SCALE_BYTES, PER = 4 + X::LOADS + F::SCALES;
    const ExpertsLayer &p = a.p;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    __shared__ int16_t token[XR], choice[XR];
    __shared__ float share[XR];
    __shared__ int expert_shared;
    LDS char *lds = (LDS char *)smem;
    LDS float *part = reinterpret_cast<LDS float *>(lds + WAVES * a.ring_up * STAGE);  // [wave][half][q][token][4]
    const Found found(reinterpret_cast<LDS char *>(part + WAVES * 2 * 16 * XR), p.experts);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = int(p.top_k), E = int(p.experts);
    find(p, found, XR);
    const int r = lane & 15, q = lane >> 4;
    const int64_t all_blocks = (p.H + 15) / 16, total = found.groups[E] * all_blocks;
    int64_t from = total * blockIdx.x / gridDim.x;
    const int64_t until = total * (blockIdx.x + 1) / gridDim.x;
    while (from < until) {
        const int group = int(from / all_blocks);
        const int64_t first_block = from % all_blocks;
        const int blocks = int(all_blocks - first_block < until - from ? all_blocks - first_block : until - from);
        from += blocks;
        for (int i = threadIdx.x; i < E; i += THREADS)
            if (found.groups[i] <= group && group < found.groups[i + 1]) expert_shared = i;
        __syncthreads();
        const int e = __builtin_amdgcn_readfirstlane(expert_shared);
        const int skip = (group - found.groups[e]) * XR;  // choices of the expert's earlier groups
        const int all = found.choices[e + 1] - found.choices[e];
        const int count = __builtin_amdgcn_readfirstlane(all - skip < XR ? all - skip : XR);
        // its tokens, by rising token
        if (wave == 0) {
            const int c = lane < p.tokens ? choice_of(found.ids, lane, k, e) : -1;
            const uint64_t mask = __ballot(c >= 0);
            const int at = __popcll(mask & ((uint64_t(1) << lane) - 1)) - skip;
            if (c >= 0 && at >= 0 && at < XR) {
                float w = 0.0f;
                for (int j = c; j < k; ++j)
                    if (found.ids[lane * k + j] == e) w += p.weights[lane * k + j];
                token[at] = int16_t(lane);
                choice[at] = int16_t(c);
                share[at] = w;
            }
        }
        __syncthreads();
        X x;
        x.init(lane, [&](int row) { return uint32_t(token[row < count ? row : 0] * p.ldx * 2); });
        const int runs = int((p.D + F::RUN - 1) / F::RUN), D = int(p.D);
        const int mine = (runs - wave + WAVES - 1) / WAVES;  // runs of each block
        const char *up = static_cast<const char *>(p.up.w) + e * p.up.stride * F::ESZ;
        const u32x4 values = buffer_at(p.X);
        const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + wave * a.ring_up * STAGE;
        const uint32_t ring1 = ring0 + a.ring_up * STAGE;
        Rows<TYPE> rows;
        u32x4 gate, mult;
        const float *scale = nullptr;
        uint32_t scale_at = 0;
        // items are (block, run) in turn; what is to be issued next
        int issued = 0, issue_block = 0, issue_run = 0;
        uint32_t to = ring0;
        const int items = blocks * mine;
        auto issue = [&]() {
            const int run = wave + issue_run * WAVES;
            if (issue_run == 0) {
                const int64_t h0 = (first_block + issue_block) * 16;
                rows.init(p.up.ld, p.H - h0, lane);
                gate = buffer_at(up + h0 * p.up.ld * F::ESZ);
                mult = buffer_at(up + (p.H + h0) * p.up.ld * F::ESZ);
                if (TYPE != 0) {
                    // lanes 0, 1, 2: of the activated half's rows, which lie in one
                    // block of 128, and of the first and last of the others', which
                    // lie in two where H is no multiple of 16
                    const int64_t last = h0 + 15 < p.H ? h0 + 15 : p.H - 1;
                    scale_at = uint32_t((lane == 0 ? h0 / 128 : (p.H + (lane == 1 ? h0 : last)) / 128) * 4);
                    scale = p.up.scale + e * p.up.stride_scale + wave * p.up.lds;
                }
            }
            const int left = D - run * F::RUN;
            rows.issue(gate, run * 128, to, left);
            rows.issue(mult, run * 128, to + 2048, left);
            x.issue(values, run * (F::RUN * 2), to + 4096, left >= F::RUN, [&](int c) { return c * 8 < left; });
            if (TYPE != 0) {
                dma::direct_load4(buffer_at(scale), to + 4096 + X::SIZE, scale_at);
                scale += WAVES * p.up.lds;
            }
            ++issued;
            to = to + STAGE == ring1 ? ring0 : to + STAGE;
            if (++issue_run == mine) issue_run = 0, ++issue_block;
        };
        for (int i = 0; i < a.ring_up && i < items; ++i) issue();
        int done = 0;
        const LDS char *const first_stage = lds + wave * a.ring_up * STAGE, *stage = first_stage;
        for (int b = 0; b < blocks; ++b) {
            const int64_t h0 = (first_block + b) * 16, last = h0 + 15 < p.H ? h0 + 15 : p.H - 1;
            const int in_first = int((p.H + last) / 128 * 128 - (p.H + h0));  // the others' rows of the first of two blocks
            f32x4 g = {0, 0, 0, 0}, m = {0, 0, 0, 0};
            for (int i = 0; i < mine; ++i, ++done) {
                const int left = D - (wave + i * WAVES) * F::RUN;
                wait_for<PER>(issued - 1 - done);
                u32x4 og[F::STEPS], om[F::STEPS], xv[F::STEPS];
#pragma unroll
                for (int s = 0; s < F::STEPS; ++s) {
                    og[s] = Rows<TYPE>::template operand<T>(stage, s, r, q);
                    om[s] = Rows<TYPE>::template operand<T>(stage + 2048, s, r, q);
                    // columns past the group's tokens are not stored
                    xv[s] = X::at(stage + 4096, r % XR, k_of<TYPE>(s, q) / 8);
                }
                float sg = 1.0f, s_lo = 1.0f, s_hi = 1.0f;
                if (TYPE != 0) {
                    const LDS float *sc = reinterpret_cast<const LDS float *>(stage + 4096 + X::SIZE);
                    sg = sc[0];
                    s_lo = sc[1];
                    s_hi = sc[2];
                }
                wait_lgkmcnt0();
                asm volatile("" ::: "memory");
                if (issued < items) issue();
                stage = stage + STAGE == first_stage + a.ring_up * STAGE ? first_stage : stage + STAGE;
                if (left < F::RUN)
#pragma unroll
                    for (int s = 0; s < F::STEPS; ++s) {
                        cut(og[s], k_of<TYPE>(s, q), left);
                        cut(om[s], k_of<TYPE>(s, q), left);
                        cut(xv[s], k_of<TYPE>(s, q), left);
                    }
                f32x4 bg = TYPE == 0 ? g : f32x4{0, 0, 0, 0}, bm = TYPE == 0 ? m : f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < F::STEPS; ++s) {
                    bg = mfma16<T>(og[s], xv[s], bg);
                    bm = mfma16<T>(om[s], xv[s], bm);
                }
                if (TYPE == 0) {
                    g = bg;
                    m = bm;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] = __builtin_fmaf(sg, bg[j], g[j]);
                        m[j] = __builtin_fmaf(4 * q + j < in_first ? s_lo : s_hi, bm[j], m[j]);
                    }
                }
            }
            // the waves' sums: lane l has rows h0 + 4(l / 16) + 0..3 of token l % 16
            if (r < XR) {
                *reinterpret_cast<LDS f32x4 *>(part + (wave * 2 + 0) * (16 * XR) + (q * XR + r) * 4) = g;
                *reinterpret_cast<LDS f32x4 *>(part + (wave * 2 + 1) * (16 * XR) + (q * XR + r) * 4) = m;
            }
            __syncthreads();
            const int at = (threadIdx.x / 4) % XR, j = threadIdx.x / (4 * XR) * 4 + threadIdx.x % 4;
            if (threadIdx.x < 16 * XR && at < count) {
                float v[1] = {0.0f}, o = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    v[0] += part[(w * 2 + 0) * (16 * XR) + threadIdx.x];
                    o += part[(w * 2 + 1) * (16 * XR) + threadIdx.x];
                }
                act::apply(p.act, v);
                const float wh = h0 + j < p.H ? v[0] * o * share[at] * Pieces<T>::TIMES : 0.0f;
                const uint32_t hi = encode<T>(wh);
                uint16_t *h = a.h + (token[at] * k + choice[at]) * a.ldh + (h0 + j) / F::RUN * (2 * F::RUN) + (h0 + j) % F::RUN;
                h[0] = uint16_t(hi);
                h[F::RUN] = uint16_t(encode<T>((wh - decode<T>(hi)) * Pieces<T>::REST));
            }
            __syncthreads();
        }
    }
}

// A workgroup has 16 of y's columns; its waves deal (group of up to DT of an
// expert's choices, run of H) pairs.  A pair's sums are added to the tokens'
// in the wave's own part of LDS.
template <class T, int TYPE, int DT>
__global__ __launch_bounds__(THREADS, 1) void down_kernel(LayerArgs a) {
    using F = Form<TYPE>;
    using V = Values<DT, F::RUN * 4>;  // both pieces
    constexpr int STAGE = 2048 + V::SIZE + F::SCALE_BYTES, PER = 2 + V::LOADS + F::SCALES;
    const ExpertsLayer &p = a.p;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    LDS char *lds = (LDS char *)smem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = int(p.top_k), tokens = int(p.tokens), E = int(p.experts), slots = tokens * k;
    // behind the runs: the tokens' sums [wave][token][16]; by choice, in the
    // order of experts, where its w h starts and (by group its choices'
    // start, number and expert) whose it is
    LDS f32x4 *sums = reinterpret_cast<LDS f32x4 *>(lds + WAVES * a.ring_down * STAGE);
    LDS uint32_t *from = reinterpret_cast<LDS uint32_t *>(sums + WAVES * tokens * 4), *group = from + slots;
    LDS uint8_t *token = reinterpret_cast<LDS uint8_t *>(group + slots);
    const Found found(lds, p.experts);  // where the runs will be
    find(p, found, DT);
    const int groups = __builtin_amdgcn_readfirstlane(found.groups[E]);
    for (int i = threadIdx.x; i < WAVES * tokens * 4; i += THREADS) sums[i] = f32x4{0, 0, 0, 0};
    for (int e = wave; e < E; e += WAVES) {
        const int g0 = found.groups[e], g1 = found.groups[e + 1], c0 = found.choices[e];
        if (g0 == g1) continue;
        const int c = lane < tokens ? choice_of(found.ids, lane, k, e) : -1;
        const uint64_t mask = __ballot(c >= 0);
        if (c >= 0) {
            const int at = c0 + __popcll(mask & ((uint64_t(1) << lane) - 1));
            from[at] = uint32_t((lane * k + c) * a.ldh * 2);
            token[at] = uint8_t(lane);
        }
        if (lane < g1 - g0) {
            const int rest = found.choices[e + 1] - c0 - lane * DT;
            group[g0 + lane] = uint32_t(e << 16 | (rest < DT ? rest : DT) << 12 | (c0 + lane * DT));
        }
    }
    __syncthreads();  // the last read of what was found
    const int r = lane & 15, q = lane >> 4;
    const int64_t d0 = int64_t(blockIdx.x) * 16;
    const char *down = static_cast<const char *>(p.down.w) + d0 * p.down.ld * F::ESZ;
    Rows<TYPE> rows;
    rows.init(p.down.ld, p.D - d0, lane);
    const int runs = int((p.H + F::RUN - 1) / F::RUN), units = groups * runs, H = int(p.H);
    const int on_group = WAVES / runs, on_run = WAVES % runs;
    const int items = units > wave ? (units - wave + WAVES - 1) / WAVES : 0;
    const u32x4 pieces = buffer_at(a.h);
    const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)) + wave * a.ring_down * STAGE;
    const uint32_t ring1 = ring0 + a.ring_down * STAGE;
    // A unit is a group and a run.  What it says (`info`: expert, number and
    // start of its choices) and where their w h starts is read from LDS
    // before the unit before it is waited for.
    struct Unit {
        int group, run;
    };
    auto advance = [&](Unit &u) {
        u.group += on_group;
        u.run += on_run;
        if (u.run >= runs) u.run -= runs, ++u.group;
    };
    Unit next{wave / runs, wave % runs}, now = next;
    uint32_t next_info = 0, to = ring0;
    V v;
    int issued = 0;
    auto look_up = [&]() {
        next_info = group[next.group];
        const int first = next_info & 0xfff, count = next_info >> 12 & 15;
        // past the group's choices, its first one's, not added to a sum
        v.init(lane, [&](int row) { return from[row < count ? first + row : first]; });
    };
    auto issue = [&]() {
        const int e = __builtin_amdgcn_readfirstlane(next_info >> 16);
        const int left = H - next.run * F::RUN;
        rows.issue(buffer_at(down + e * p.down.stride * F::ESZ), next.run * 128, to, left);
        // chunks of eight in each piece, as far as the rows go
        v.issue(pieces, next.run * (F::RUN * 4), to + 2048, left >= F::RUN, [&](int c) { return c % (F::RUN / 8) * 8 < left; });
        // 16 rows from a multiple of 16 lie in one block of 128
        if (TYPE != 0)
            dma::direct_load4(buffer_at(p.down.scale + e * p.down.stride_scale + next.run * p.down.lds + d0 / 128),
                              to + 2048 + V::SIZE, 0);
        to = to + STAGE == ring1 ? ring0 : to + STAGE;
        advance(next);
        if (++issued < items) look_up();
    };
    if (items > 0) look_up();
    for (int i = 0; i < a.ring_down && i < items; ++i) issue();
    const LDS char *const first_stage = lds + wave * a.ring_down * STAGE, *stage = first_stage;
    uint32_t now_info = items > 0 ? group[now.group] : 0;
    for (int done = 0; done < items; ++done) {
        const int first = now_info & 0xfff, count = now_info >> 12 & 15;
        const int t = token[r < count ? first + r : first];
        const int left = H - now.run * F::RUN;
        advance(now);
        if (done + 1 < items) now_info = group[now.group];
        wait_for<PER>(issued - 1 - done);
        u32x4 od[F::STEPS], hi[F::STEPS], lo[F::STEPS];
#pragma unroll
        for (int s = 0; s < F::STEPS; ++s) {
            od[s] = Rows<TYPE>::template operand<T>(stage, s, r, q);
            hi[s] = V::at(stage + 2048, r % DT, k_of<TYPE>(s, q) / 8);
            lo[s] = V::at(stage + 2048, r % DT, F::RUN / 8 + k_of<TYPE>(s, q) / 8);
        }
        const float scale = TYPE == 0 ? 1.0f : *reinterpret_cast<const LDS float *>(stage + 2048 + V::SIZE);
        wait_lgkmcnt0();
        asm volatile("" ::: "memory");
        if (issued < items) issue();
        stage = stage + STAGE == first_stage + a.ring_down * STAGE ? first_stage : stage + STAGE;
        // up_kernel has filled the pieces' last chunks with zeros
        if (left < F::RUN)
#pragma unroll
            for (int s = 0; s < F::STEPS; ++s) cut(od[s], k_of<TYPE>(s, q), left);
        f32x4 block = {0, 0, 0, 0}, rest = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < F::STEPS; ++s) {
            rest = mfma16<T>(od[s], lo[s], rest);
            block = mfma16<T>(od[s], hi[s], block);
        }
        if (r < count) {
            LDS f32x4 *sum = sums + (wave * tokens + t) * 4 + q;
            f32x4 y = *sum;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = __builtin_fmaf(scale / Pieces<T>::TIMES, __builtin_fmaf(1.0f / Pieces<T>::REST, rest[j], block[j]), y[j]);
            *sum = y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * 16; i += THREADS) {
        const int t = i / 16;
        const int64_t d = d0 + i % 16, at = t * p.ldy + d;
        if (d >= p.D) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += reinterpret_cast<const LDS float *>(sums)[w * tokens * 16 + i];
        if (p.out == 0) {
            float *y = static_cast<float *>(p.Y) + at;
            *y = p.beta != 0.0f ? __builtin_fmaf(p.beta, *y, s) : s;
        } else {
            uint16_t *y = static_cast<uint16_t *>(p.Y) + at;
            *y = uint16_t(encode<T>(p.beta != 0.0f ? __builtin_fmaf(p.beta, decode<T>(*y), s) : s));
        }
    }
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

constexpr int MOST_LDS = 160 * 1024;
constexpr int UNITS = 256;  // compute units of an MI355X
static_assert(4 * (LAYER_MAX_EXPERTS + 1) + 2 * (LAYER_MAX_EXPERTS + 1) + 2 * LAYER_MAX_TOKENS * LAYER_MAX_TOP_K <= WAVES * 2 * 4096,
              "what is found fits where the runs will be");

// Stages of the ring: up to four, as many as fit.
int ring_of(int64_t stage, int64_t beside) { return int(least(4, (MOST_LDS - 1024 - beside) / (WAVES * stage))); }

template <class K>
hipError_t allow(K kernel, size_t bytes, hipStream_t stream) {
    return bytes <= 64 * 1024 ? hipSuccess : allow_lds(reinterpret_cast<const void *>(kernel), MOST_LDS - 1024, stream);
}

template <class T, int TYPE, int XR>
hipError_t run_up(LayerArgs &a, hipStream_t stream) {
    const ExpertsLayer &p = a.p;
    constexpr int64_t stage = 4096 + XR * Form<TYPE>::RUN * 2 + Form<TYPE>::SCALE_BYTES, part = WAVES * 2 * 64 * XR;
    const int64_t beside = part + found_bytes(p);
    a.ring_up = ring_of(stage, beside);
    const size_t lds = size_t(WAVES * a.ring_up * stage + beside);
    hipError_t e = allow(up_kernel<T, TYPE, XR>, lds, stream);
    if (e != hipSuccess) return e;
    const int64_t blocks = p.tokens * p.top_k * ceil_div(p.H, 16);  // at most
    up_kernel<T, TYPE, XR><<<dim3(unsigned(least(blocks, UNITS))), dim3(THREADS), lds, stream>>>(a);
    return hipGetLastError();
}
template <class T, int TYPE, int DT>
hipError_t run_down(LayerArgs &a, hipStream_t stream) {
    const ExpertsLayer &p = a.p;
    constexpr int64_t stage = 2048 + DT * Form<TYPE>::RUN * 4 + Form<TYPE>::SCALE_BYTES;
    const int64_t beside = WAVES * p.tokens * 64 + 9 * p.tokens * p.top_k;
    a.ring_down = ring_of(stage, beside);
    const size_t lds = size_t(WAVES * a.ring_down * stage + beside);
    hipError_t e = allow(down_kernel<T, TYPE, DT>, lds, stream);
    if (e != hipSuccess) return e;
    down_kernel<T, TYPE, DT><<<dim3(unsigned(ceil_div(p.D, 16))), dim3(THREADS), lds, stream>>>(a);
    return hipGetLastError();
}
// A group of tokens more reads the weights again, from L2; room for more
// leaves less of LDS for the weights on their way.
template <class T, int TYPE>
hipError_t run_tokens(LayerArgs &a, hipStream_t stream) {
    const ExpertsLayer &p = a.p;
    a.ldh = ceil_div(p.H, Form<TYPE>::RUN) * 2 * Form<TYPE>::RUN;
    const int64_t slots = p.tokens * p.top_k;
    const hipError_t e = p.tokens > 8 && slots > 5 * p.experts ? run_up<T, TYPE, 16>(a, stream) : run_up<T, TYPE, 8>(a, stream);
    if (e != hipSuccess) return e;
    return p.tokens <= 4 || slots <= 2 * p.experts ? run_down<T, TYPE, 4>(a, stream) : run_down<T, TYPE, 8>(a, stream);
}
template <class T>
hipError_t run_type(LayerArgs &a, hipStream_t stream) {
    if (a.p.type == 0) return run_tokens<T, 0>(a, stream);
    return a.p.type == 1 ? run_tokens<T, 1>(a, stream) : run_tokens<T, 2>(a, stream);
}

}  // namespace

size_t experts_layer_workspace(int64_t tokens, int64_t, int64_t top_k, int64_t, int64_t H) {
    return size_t(tokens * top_k * 2 * ceil_div(H, 128) * 128 * 2 + 16);
}

hipError_t launch_experts_layer(const ExpertsLayer &p, hipStream_t stream) {
    LayerArgs a{};
    a.p = p;
    a.h = static_cast<uint16_t *>(p.workspace);
    return p.in == 1 ? run_type<BF16>(a, stream) : run_type<F16>(a, stream);
}

}  // namespace libgemm
