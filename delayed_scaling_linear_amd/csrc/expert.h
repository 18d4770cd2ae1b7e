// The plan of tokens sorted by expert, shared by the kernels that use it, their
// launchers and the C-ABI layer (which sizes the caller's buffers).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8dsl.h"

namespace fp8dsl {

constexpr int kExpertsMax = FP8DSL_EXPERTS_MAX;
// Rows of one tile of the cast: a tile holds rows of one segment.
constexpr int kExpertTile = 128;
// Pairs that one workgroup of the plan sorts alone, in one launch; more are split into
// pieces of kPlanPiece or more over at most kPlanPieces workgroups, in two.  us a call with
// one / two: 8192 pairs of 8 experts 10.2 / 9.5, of 64 12.5 / 9.5, of 256 16.4 / 9.8; alone
// 4096 pairs take 6.9, 7.9 and 9.7.
constexpr int64_t kPlanAlone = 4096;
constexpr int64_t kPlanPiece = 2048;
constexpr int64_t kPlanPieces = 128;

// Device layout of a plan (int32 words).
//   header   {magic, tokens, top_k, experts, capacity, tiles, rows of all segments}
//   offsets  [experts + 1], counts [experts], slots [pairs], sources [rows]
//   tiles    [tiles_max] {first row of the tile in its segment, rows of the
//            segment, first row of the segment, 0}
//   hist     [pieces, experts]: pairs of each expert in each piece of the ids
constexpr int32_t kExpertMagic = 0x45585031;
constexpr int kExpertHeader = 16;
struct ExpertShape {
    int64_t tokens, pairs, capacity, rows, tiles_max, pieces;
    int32_t top_k, experts;
    int64_t offsets, counts, slots, sources, tiles, hist, words;
    explicit ExpertShape(const fp8_expert_sizes_t &s)
        : tokens(s.tokens), pairs(s.tokens * s.top_k), capacity(s.capacity), top_k(s.top_k),
          experts(s.experts) {
        const int64_t segments = std::min<int64_t>(experts, pairs);
        if (capacity) {
            rows = experts * capacity;
            tiles_max = experts * ((capacity + kExpertTile - 1) / kExpertTile);
        } else {
            rows = (pairs + 15 * segments) / 16 * 16;
            tiles_max = rows / kExpertTile + segments;
        }
        pieces = pairs <= kPlanAlone ? 1 : std::min(pairs / kPlanPiece, kPlanPieces);
        const auto up = [](int64_t v) { return (v + 15) / 16 * 16; };
        offsets = kExpertHeader;
        counts = offsets + up(experts + 1);
        slots = counts + up(experts);
        sources = slots + up(pairs);
        tiles = sources + up(rows);
        hist = tiles + up(4 * tiles_max);
        words = hist + (pieces > 1 ? up(pieces * experts) : 0);
    }
};

// A plan as the kernels see it.
struct ExpertView {
    const int32_t *header, *offsets, *slots, *sources;
    const int4 *tiles;
    int32_t tokens, top_k, experts, capacity, rows;
    uint32_t reciprocal;     // 2^32 / top_k rounded up; 0 stands for 2^32
    ExpertView(const ExpertShape &s, const int32_t *plan)
        : header(plan), offsets(plan + s.offsets), slots(plan + s.slots),
          sources(plan + s.sources), tiles(reinterpret_cast<const int4 *>(plan + s.tiles)),
          tokens((int32_t)s.tokens), top_k(s.top_k), experts(s.experts),
          capacity((int32_t)s.capacity), rows((int32_t)s.rows),
          reciprocal((uint32_t)((((uint64_t)1 << 32) + s.top_k - 1) / s.top_k)) {}
    // pair / top_k.  The rounding of the reciprocal, less than top_k <= 64 in 2^32, times
    // a pair below 2^23 does not reach a unit of the quotient.
    __device__ __forceinline__ uint32_t token_of(uint32_t pair) const {
        return reciprocal ? __umulhi(pair, reciprocal) : pair;
    }
    // A buffer that no plan of these sizes was written to has no work in it.
    __device__ __forceinline__ bool built() const {
        return (header[0] == kExpertMagic) & (header[1] == tokens) & (header[2] == top_k) &
               (header[3] == experts) & (header[4] == capacity);
    }
};

hipError_t launch_expert_plan(const ExpertShape &shape, const int32_t *ids, int32_t *plan,
                              hipStream_t stream);

// y[slot] = x[t] and zeros in the segments' other rows.
hipError_t launch_expert_gather(const ExpertShape &shape, const int32_t *plan, const uint16_t *x,
                                int64_t ldx, uint16_t *y, int64_t ldy, int64_t cols,
                                hipStream_t stream);

// The same with weights (or null) and the cast; q and qt as a cast's outputs.
hipError_t launch_expert_gather_cast(const ExpertShape &shape, const int32_t *plan,
                                     const uint16_t *x, int64_t ldx, int64_t cols,
                                     const float *weights, const float *scale, int fmt, uint8_t *q,
                                     uint8_t *qt, float *amax_cur, float *scale_inv_out,
                                     const int32_t *noop, hipStream_t stream);

hipError_t launch_expert_combine(const ExpertShape &shape, const int32_t *plan, const uint16_t *x,
                                 int64_t ldx, const float *weights, const uint16_t *base,
                                 int64_t ldbase, uint16_t *y, int64_t ldy, int64_t cols,
                                 hipStream_t stream);

// dx may be null.
hipError_t launch_expert_combine_backward(const ExpertShape &shape, const int32_t *plan,
                                          const uint16_t *dy, int64_t lddy, const uint16_t *x,
                                          int64_t ldx, const float *weights, float *dweights,
                                          uint16_t *dx, int64_t lddx, int64_t cols,
                                          hipStream_t stream);

}  // namespace fp8dsl
