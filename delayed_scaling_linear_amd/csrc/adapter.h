// Shapes and work splits of the low-rank adapter kernels, shared by the
// launchers and the C-ABI layer (which sizes the caller's buffers).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dropout.h"

namespace fp8dsl {

// Rows of one tile: two 16-row MFMA blocks.  A tile holds rows of one adapter.
constexpr int kAdapterTile = 32;
constexpr int kAdapterMaxRank = 128;
constexpr int kAdapterMaxCount = 4096;
// Columns of one workgroup of the expand and of the weight-gradient kernel.
constexpr int kAdapterCols = 512;
// bf16 parts of a short operand of the weight gradients: together all 24 bits of
// an fp32 value.
constexpr int kAdapterGradParts = 3;

// Device layout of a plan (int32 words): the batch's rows sorted by adapter,
// every adapter's rows starting a new tile.
//   header       {magic, rows, adapters, tiles, tiles that have an adapter}
//   group_tile0  [adapters + 2]: first tile of each adapter, then of the rows
//                without one, then the tile count
//   group_rank   [adapters]: adapters before this one that have rows
//   tile_adapter [tiles_max]: an adapter, -1 (rows without one), -2 (unused)
//   tile_row     [32 * tiles_max]: row of each position, -1 past a group's end
constexpr int32_t kPlanMagic = 0x414c5031;
constexpr int kPlanHeader = 16;
struct AdapterPlanShape {
    int64_t rows, adapters, tiles_max;
    int64_t group_tile0, group_rank, tile_adapter, tile_row, words;
    AdapterPlanShape(int64_t rows_, int64_t adapters_) : rows(rows_), adapters(adapters_) {
        const int64_t groups = std::min(adapters + 1, rows);
        tiles_max = (rows + (kAdapterTile - 1) * groups) / kAdapterTile;
        const auto up = [](int64_t v) { return (v + 15) / 16 * 16; };
        group_tile0 = kPlanHeader;
        group_rank = group_tile0 + up(adapters + 2);
        tile_adapter = group_rank + up(adapters);
        tile_row = tile_adapter + up(tiles_max);
        words = tile_row + kAdapterTile * tiles_max;
    }
};

// Ranks as the kernels see them: the next of 16, 32, 64, 128.
inline int64_t adapter_padded_rank(int64_t rank) {
    return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
}

// K parts of the contraction over C columns: workgroups per tile (per two tiles
// of rank 128) of the shrink kernel.
//   Fewer tiles than CUs: a workgroup per CU, each at least 256 columns, at most
//   16.
//   Else up to `resident` workgroups, if each keeps 2048 columns.  A CU holds two
//   (512 in all), from rank 33 to 64 three (768); `resident` is a little more, so
//   that the few tiles that the adapters' ends add to a full batch take no part
//   away.  A forward of 8192 rows from 8192 columns to 2048, us by parts (* the
//   rule's):
//                              1     2     3     4
//     rank 16, 257 tiles      41*   45    49    49
//              265 tiles      56*   52    52    51
//     rank 32, 257 tiles      44    48*   51    54
//              265 tiles      62*   57    56    55
//     rank 64, 257 tiles      63    58    61*   65
//              265 tiles      81    72    72*   72
//     rank 128, 257 tiles    105   108    93    85*
//               265 tiles    114   123   111*  117
//               388 tiles    120   136*  129   132
//   (257: one adapter, exactly 256 tiles with rows; 265: nine, a few more than one a
//   CU.)  So it pays from rank 33 on while tiles are few more than CUs.  It costs a
//   tenth at rank 32 with 257 to 260 tiles; at rank 128 with more than 270 an
//   eighth, and over 40 adapters (295 tiles) 157 us against 122.  Over 2048 columns
//   parts measured no faster (rank 64, 260 tiles: 65 us, 69 with two).
inline int adapter_parts(int64_t tiles, int64_t C, int64_t rank) {
    const int64_t groups = std::max<int64_t>(1, rank > 64 ? (tiles + 1) / 2 : tiles);
    const int64_t resident = rank <= 16 ? 256 : rank <= 32 || rank > 64 ? 520 : 800;
    const int64_t fill = std::min<int64_t>({256 / groups, C / 256, 16});
    return (int)std::max<int64_t>({1, fill, std::min(resident / groups, C / 2048)});
}
// Rows of the sums of all parts where there is more than one: workgroups (256, or
// `resident`) times rows of one, at most 520 * 64.
constexpr int64_t kAdapterSumRows = 520 * 64;

// Tiles of one weight-gradient workgroup: a partial sum of R fp32 per column
// is written and read per workgroup, so as few of them as fill the chip (two
// workgroups per CU; one of rank 128, which has twice the threads).
inline int64_t adapter_chunks(int64_t rank, int64_t in, int64_t out) {
    const int64_t blocks = (in + kAdapterCols - 1) / kAdapterCols +
                           (out + kAdapterCols - 1) / kAdapterCols;
    return std::max<int64_t>(1, (rank > 64 ? 256 : 512) / blocks);
}
inline int64_t adapter_chunk(int64_t tiles, int64_t rank, int64_t in, int64_t out) {
    const int64_t chunks = adapter_chunks(rank, in, out);
    return std::max<int64_t>(1, (tiles + chunks - 1) / chunks);
}

// Tiles of one expand workgroup: more where its weights (2 rank bytes a column)
// weigh more against a tile's base and output (128 bytes a column), while
// enough workgroups are left.
inline int64_t adapter_expand_chunk(int64_t tiles, int64_t C, int64_t rank) {
    if (rank <= 32) return 1;
    const int64_t blocks = (C + kAdapterCols - 1) / kAdapterCols;
    return std::max<int64_t>(1, std::min(rank / 12, (tiles * blocks + 1023) / 1024));
}

// Partial sums of the weight gradients: one per (chunk of tiles, adapter
// with rows in it); chunk + rank of the adapter is distinct for each.
inline int64_t adapter_slots(const AdapterPlanShape &p, int64_t chunk) {
    return (p.tiles_max + chunk - 1) / chunk + std::min(p.adapters, p.rows);
}

// Workspace: K-part sums of h or g, both short operands of the weight
// gradients as bf16 parts, and the gradients' partial sums.
// Each is sized by a bound that does not fall when rows, adapters or rank
// rise, so that the workspace of a program's largest batch serves all of its
// batches.  (The splits themselves do not rise: fewer tiles run in more K
// parts, and 300 rows of one adapter need more sums than 2000.)
struct AdapterWorkspace {
    int64_t sums, packed, grads, bytes;
    // What a call without weight gradients is asked for: the sums alone, where the
    // rest counts (1 MiB and more: small workspaces are one size for all calls).
    int64_t no_grads;
    AdapterWorkspace(const AdapterPlanShape &p, int64_t rank, int64_t in, int64_t out) {
        sums = (sum_rows(p.rows, in, out) * rank * 4 + 255) / 256 * 256;
        packed = 2 * p.tiles_max * kAdapterTile * adapter_padded_rank(rank) *
                 kAdapterGradParts * 2;
        grads = grad_bytes(p, rank, in, out);
        if (rank > 64) grads = std::max(grads, grad_bytes(p, 64, in, out));
        bytes = sums + packed + grads;
        no_grads = std::min(bytes, std::max<int64_t>(sums, 1 << 20));
    }

private:
    // Rows of sums, over all K parts: at most 16 parts or 2048 columns a part, and
    // either one part or no more workgroups than adapter_parts aims at, of 32 rows
    // (64 at rank 128).
    static int64_t sum_rows(int64_t rows, int64_t in, int64_t out) {
        const int64_t C = std::max(in, out);
        const int64_t parts = std::max<int64_t>({1, std::min<int64_t>(C / 256, 16), C / 2048});
        return std::max(rows, std::min(rows * parts, kAdapterSumRows));
    }
    // As adapter_slots: ceil(tiles / chunk) is at most the chunks aimed at, and
    // at most the tiles.
    static int64_t grad_bytes(const AdapterPlanShape &p, int64_t rank, int64_t in, int64_t out) {
        const int64_t slots = std::min(p.tiles_max, adapter_chunks(rank, in, out)) +
                              std::min(p.adapters, p.rows);
        return slots * rank * (in + out) * 4;
    }
};

struct AdapterArgs {
    const uint16_t *a, *b;      // bf16 [count, rank, in], [count, out, rank]
    const float *alpha;         // [count]
    int32_t count, rank;
    int64_t in, out;
};

hipError_t launch_adapter_plan(const int32_t *row_adapter, const AdapterPlanShape &shape,
                               int32_t *plan, hipStream_t stream);

hipError_t launch_adapter_fwd(const AdapterArgs &w, const AdapterPlanShape &shape,
                              const int32_t *plan, const DropoutArgs &drop, const uint16_t *x,
                              int64_t ldx, const uint16_t *base, int64_t ldbase, uint16_t *y,
                              int64_t ldy, float *h, void *ws, hipStream_t stream);

// dx may be null (no data gradient), da and db both null (no weight gradient).
hipError_t launch_adapter_backward(const AdapterArgs &w, const AdapterPlanShape &shape,
                                   const int32_t *plan, const DropoutArgs &drop,
                                   const uint16_t *x, int64_t ldx, const uint16_t *dy,
                                   int64_t lddy, const float *h, const uint16_t *base,
                                   int64_t ldbase, uint16_t *dx, int64_t lddx, void *da, void *db,
                                   int out_dtype, void *ws, hipStream_t stream);

// da = db = 0 (a batch without rows).
hipError_t launch_adapter_clear_grads(const AdapterArgs &w, void *da, void *db, int out_dtype,
                                      hipStream_t stream);

}  // namespace fp8dsl
