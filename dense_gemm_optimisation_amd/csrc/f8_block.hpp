// The canonical block-scaled 8-bit problem that the host layer hands to the
// kernels, and the launchers of the kernels for operands of that kind and of
// the experts' routing.  The host layer has validated every argument and
// rewritten a column-major C as the row-major C^T = B^T A^T.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "tile_schedule.hpp"

namespace libgemm {

// What a problem's segments (device offsets) cut: nothing, the rows of A and
// C (each segment with its own B), or the contracted dimension (each segment
// with its own C).
enum class Segments : int { None = 0, Rows = 1, Contracted = 2 };

// A launch has fewer than 2^32 threads.
inline bool launch_over(double workgroups, int threads) { return workgroups * threads >= 4294967296.0; }

// Operand X of R rows: code (r, k) at x[r*ld + k], scale (r, kb) at
// s[kb*lds + (r >> shift)], shift 0 (a scale per row) or 7 (per 128 rows).
struct BlockOperand {
    const uint8_t *x;
    int64_t ld, stride;
    const float *s;
    int64_t lds, sstride;
    int shift;
    int e5m2;
};

// Which of the 256 x 256 tiles a launch takes: all; those of whole rounds of
// ROUND tiles; or, in quarters, the others.
enum class TilePart { All, Rounds, Rest };
constexpr uint32_t ROUND = 256;

struct BlockProblem {
    Segments segments;
    int64_t M, N, K;  // K = 0, and alpha too, where nothing is multiplied
    float alpha, beta;
    BlockOperand a, b;
    void *C;
    int64_t ldc, sC;
    int out;  // 0 fp32, 1 bf16, 2 fp16
    bool c_turned;           // C(i, j) at C[j*ldc + i] (few rows only)
    TilePart part;           // (All with segments)
    int64_t batch;           // slices; with segments, the experts
    const int32_t *offsets;  // batch + 1, with segments
};

enum class BlockKernel { None, Tile256, Tile256Edge, Tile256Rest, Tile128, Tile128Two, Few16, Few32, Few64 };
// general: the general kernel, Tile256; split: K and the edges may be split off.
BlockKernel block_choose(const BlockProblem &p, bool general, bool split);
const char *block_kernel_name(BlockKernel k);
hipError_t launch_block(BlockKernel k, const BlockProblem &p, hipStream_t stream);

// x (rows x cols, type 0 fp32, 1 bf16, 2 fp16) to codes and scales; q or qt
// may be null.
struct QuantizeArgs {
    int64_t rows, cols;
    const void *x;
    int64_t ldx;
    int type;
    const int32_t *index;
    int64_t x_rows;
    int e5m2, block;
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t lds;
    uint8_t *qt;
    int64_t ldqt;
    float *st;
    int64_t ldst;
    int64_t batch, sx, sq, ss, sqt, sst;
};
hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t stream);

struct RouteArgs {
    int64_t tokens;
    int experts;
    const void *logits;
    int64_t ldl;
    int type;
    const float *bias;
    const uint8_t *keep;
    int sigmoid, groups, top_groups, group_top, top_k, renormalise;
    float scale;
    int32_t *ids;
    float *weights;
    int align;
    int64_t rows;
    int32_t *offsets, *row_tokens, *places;  // all null: no layout
    void *workspace;
};
// Tokens whose choices of one expert a 64-bit mask holds.
constexpr int ROUTE_BLOCK = 64;
constexpr int ROUTE_MAX_EXPERTS = 1024, ROUTE_MAX_TOP_K = 32;
size_t route_workspace(int64_t tokens, int64_t experts);  // bytes
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);

struct RouteBackwardArgs {
    int64_t tokens;
    int experts;
    const void *logits;
    int64_t ldl;
    int type;
    int sigmoid, top_k, renormalise;
    float scale;
    const int32_t *ids;
    const float *d_weights;
    void *d_logits;
    int64_t ldd;
};
hipError_t launch_route_backward(const RouteBackwardArgs &a, hipStream_t stream);

}  // namespace libgemm
