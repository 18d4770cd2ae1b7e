// Low-rank adapters of many requests beside a shared projection.
//
// Row r of a batch belongs to adapter a (or to none), and with x' = dropout(x)
//
//   forward    h = alpha_a x' A_a^T            y  = base + h B_a^T
//   backward   g = alpha_a dy B_a              dx = base + f keep (g A_a)
//              dA_a = sum of g^T x'            dB_a = sum of dy^T h
//
// Ranks are at most 128, so every product is bound by the memory traffic of
// its long operand (x, dy or y), not by the matrix cores; each kernel streams
// that operand once and takes the adapter's weights from the L2.
//
//   plan     sorts the rows by adapter once per batch; 32-row tiles of one
//            adapter are the unit of work of all other kernels, so rows may
//            come in any order and a tile's weights are read once for it.
//   shrink   [32 rows, C] x [C, R]: h and g.  Waves split C, sums meet in LDS.
//   expand   [32 rows, R] x [R, C] added to base: y and dx.
//   wgrad    [R, rows] x [rows, C] over a chunk of tiles: partial dA and dB,
//            added in chunk order by a second pass (no atomics: the same
//            bits on every run).
//
// h and g are held in fp32.  Where they feed a matrix core they are split
// into bf16 parts that add up to them: two (the error is 2^-16 of h) for y and
// dx, bf16 results beside a base, three (all of an fp32 value's 24 bits) for dA
// and dB, which bf16 takes as the fp32 result rounded once: with two parts one
// in 200 of its values went to the other neighbour.
// Dropout multiplies by the mask on the operand (exact) and by f in fp32 on
// the sums.
//
// Measured on MI355X, where a large copy moves 5.1 TB/s (us of a whole call on
// inputs that are not in the caches, and in brackets its bytes at that rate): 8192
// rows of 2048 -> 6144, rank 64, nine requests 66 to 70 (47); 2048 -> 8192, rank
// 16 with dropout, forward 66 (59), backward 92 to 94 (46, reading dy once; it is
// read twice); 16384 rows of 8192 -> 2048, rank 128, backward 324 to 343 over
// several cards (178).
#include "adapter.h"

#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;
constexpr int TILE = kAdapterTile;

// v_mfma_f32_16x16x32_bf16: lane l gives row (or column) l % 16 of an
// operand, contraction indices 8 (l / 16) .. + 7, and holds column l % 16,
// rows 4 (l / 16) .. + 3 of the result.
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t bf16_rne(float f) {
    const uint32_t u = __float_as_uint(f);
    return (f != f) ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// v as a sum of PARTS bf16 values per element: truncations, the last one
// rounded.  An infinity or NaN goes to the first part alone (rare: a wave that
// sees none skips those steps).
template <int PARTS, bool SPECIAL>
__device__ __forceinline__ void split8_steps(const float v[8], u32x4 (&out)[PARTS]) {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (p == PARTS - 1) {
                out[p][d] = pack_bf16(rest[2 * d], rest[2 * d + 1]);
                continue;
            }
            uint32_t bits[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float &r = rest[2 * d + k];
                const uint32_t u = __float_as_uint(r);
                bits[k] = u & 0xFFFF0000u;
                if constexpr (SPECIAL) {
                    const bool special = (u & 0x7F800000u) == 0x7F800000u;
                    if (special && r != r) bits[k] |= 0x00400000u;
                    r = special ? 0.0f : r - __uint_as_float(bits[k]);
                } else {
                    r -= __uint_as_float(bits[k]);
                }
            }
            out[p][d] = high_halves(bits[0], bits[1]);
        }
    }
}

template <int PARTS>
__device__ __forceinline__ void split8(const float v[8], u32x4 (&out)[PARTS]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    if (__any(most >= 0x7F800000u))
        split8_steps<PARTS, true>(v, out);
    else
        split8_steps<PARTS, false>(v, out);
}

// ---- the plan ---------------------------------------------------------------

struct PlanView {
    const int32_t *header, *group_tile0, *group_rank, *tile_adapter, *tile_row;
    int32_t rows, adapters;
    // A buffer that no plan of these sizes was written to has no work in it.
    __device__ __forceinline__ bool built() const {
        return (header[0] == kPlanMagic) & (header[1] == rows) & (header[2] == adapters);
    }
};

PlanView view_of(const AdapterPlanShape &s, const int32_t *plan) {
    return {plan, plan + s.group_tile0, plan + s.group_rank, plan + s.tile_adapter,
            plan + s.tile_row, (int32_t)s.rows, (int32_t)s.adapters};
}

__device__ __forceinline__ int group_of(int32_t a, int adapters) {
    return (uint32_t)a < (uint32_t)adapters ? a : adapters;
}

// One workgroup: rows per group (LDS counters; a count does not depend on
// their order), then each group's first tile and rank by a scan.
constexpr int PLAN_THREADS = 1024;
__global__ __launch_bounds__(PLAN_THREADS) void adapter_plan_groups_kernel(
    const int32_t *__restrict__ row_adapter, int32_t rows, int32_t adapters,
    int32_t *__restrict__ header, int32_t *__restrict__ group_tile0,
    int32_t *__restrict__ group_rank) {
    __shared__ int count[kAdapterMaxCount + 1];
    __shared__ int2 scan[PLAN_THREADS];
    const int tid = threadIdx.x, groups = adapters + 1;
    for (int g = tid; g < groups; g += PLAN_THREADS) count[g] = 0;
    __syncthreads();
    for (int r = tid; r < rows; r += PLAN_THREADS)
        atomicAdd(&count[group_of(row_adapter[r], adapters)], 1);
    __syncthreads();
    // Each thread's run of groups, then an inclusive scan over the threads.
    const int per = (groups + PLAN_THREADS - 1) / PLAN_THREADS;
    const int g0 = min(groups, tid * per), g1 = min(groups, g0 + per);
    int2 mine = {0, 0};
    for (int g = g0; g < g1; ++g) {
        mine.x += (count[g] + TILE - 1) / TILE;
        mine.y += count[g] > 0;
    }
    scan[tid] = mine;
    for (int step = 1; step < PLAN_THREADS; step *= 2) {
        __syncthreads();
        const int2 add = tid >= step ? scan[tid - step] : int2{0, 0};
        __syncthreads();
        scan[tid].x += add.x;
        scan[tid].y += add.y;
    }
    int tile = scan[tid].x - mine.x, rank = scan[tid].y - mine.y;
    for (int g = g0; g < g1; ++g) {
        group_tile0[g] = tile;
        if (g < adapters) group_rank[g] = rank;
        if (g == adapters) {
            const int all = tile + (count[g] + TILE - 1) / TILE;
            group_tile0[g + 1] = all;
            header[0] = kPlanMagic;
            header[1] = rows;
            header[2] = adapters;
            header[3] = all;
            header[4] = tile;
        }
        tile += (count[g] + TILE - 1) / TILE;
        rank += count[g] > 0;
    }
}

// One workgroup per group (the last: rows without an adapter, and the unused
// tiles): its rows in batch order, found by ballots.
__global__ __launch_bounds__(THREADS) void adapter_plan_rows_kernel(
    const int32_t *__restrict__ row_adapter, int32_t rows, int32_t adapters, int32_t tiles_max,
    const int32_t *__restrict__ group_tile0, int32_t *__restrict__ tile_adapter,
    int32_t *__restrict__ tile_row) {
    __shared__ int wave_count[2][WAVES];
    const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = group_tile0[group], t1 = group_tile0[group + 1];
    if (group == adapters)
        for (int t = t1 + tid; t < tiles_max; t += THREADS) tile_adapter[t] = -2;
    if (t0 == t1) return;
    for (int t = t0 + tid; t < t1; t += THREADS) tile_adapter[t] = group < adapters ? group : -1;
    int at = t0 * TILE;
    int buf = 0;
    for (int r0 = 0; r0 < rows; r0 += THREADS, buf ^= 1) {
        const int r = r0 + tid;
        const bool hit = r < rows && group_of(row_adapter[r], adapters) == group;
        const uint64_t votes = __ballot(hit);
        if (lane == 0) wave_count[buf][wave] = __popcll(votes);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) before += wave_count[buf][w];
            all += wave_count[buf][w];
        }
        if (hit) tile_row[at + before + __popcll(votes & ((1ull << lane) - 1))] = r;
        at += all;
    }
    for (int p = at + tid; p < t1 * TILE; p += THREADS) tile_row[p] = -1;
}

// ---- shrink: h = alpha f (keep x) W ------------------------------------------

// Element 0 of row `row` (not negative) of a bf16 matrix: one 32 x 32 + 64 bit
// multiply-add with the stride in bytes.
__device__ __forceinline__ const uint16_t *row_at(const uint16_t *p, int row, uint32_t ld_bytes) {
    return reinterpret_cast<const uint16_t *>(reinterpret_cast<const char *>(p) +
                                              (uint64_t)(uint32_t)row * ld_bytes);
}
__device__ __forceinline__ uint16_t *row_at(uint16_t *p, int row, uint32_t ld_bytes) {
    return const_cast<uint16_t *>(row_at(const_cast<const uint16_t *>(p), row, ld_bytes));
}

// L bf16 columns, as loaded and stored.
template <int L>
struct Cols {
    uint32_t d[L / 2];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (L == 8) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = v[i];
        } else if constexpr (L == 4) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
            d[0] = v.x;
            d[1] = v.y;
        } else {
            static_assert(L == 2, "2, 4 or 8 columns");
            d[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    // What is read once: past the last-level cache.
    __device__ __forceinline__ void load_once(const uint16_t *p) {
        static_assert(L >= 4, "4 or 8 columns");
        if constexpr (L == 8) {
            const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = v[i];
        } else {
            const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
            d[0] = v.x;
            d[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        static_assert(L >= 4, "4 or 8 columns");
        if constexpr (L == 8)
            *reinterpret_cast<u32x4 *>(p) = u32x4{d[0], d[1], d[2], d[3]};
        else
            *reinterpret_cast<u32x2 *>(p) = u32x2{d[0], d[1]};
    }
    __device__ __forceinline__ void clear_unless(bool ok) {
#pragma unroll
        for (int i = 0; i < L / 2; ++i) d[i] = ok ? d[i] : 0u;
    }
};

__device__ __forceinline__ u32x4 keep_chunk(u32x4 v, const DropoutKey &key, uint64_t e,
                                            uint32_t threshold) {
    uint32_t w[4];
    dropout_words(key, e, w);
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] &= dropout_keep2(w[d], threshold);
    return v;
}

// The shrink's shape for a padded rank: its waves split the columns, each in
// steps through LDS of its own.  From rank 64 on four waves, so that two
// workgroups and more fit a CU: with one, a few more tiles than CUs take a
// second round.
constexpr int shrink_waves(int rp) { return rp >= 64 ? 4 : 8; }
constexpr int shrink_threads(int rp) { return 64 * shrink_waves(rp); }
constexpr int shrink_step(int rp) { return rp >= 128 ? 32 : 64; }
// Tiles of a workgroup: rank 128's weights are four times a tile's x, so two
// tiles of an adapter share them.  A pair of two adapters' tiles is split: its
// second tile goes to one of the workgroups, one for each adapter, behind those of the
// pairs (a second pass over the weights instead made such a workgroup the kernel's
// tail).
constexpr int shrink_tiles(int rp) { return rp >= 128 ? 2 : 1; }
// 16-byte pieces of LDS a wave stages: x (two row blocks a tile) and W (rp / 16).
constexpr int shrink_wave_pieces(int rp) {
    return shrink_step(rp) / 32 * (2 * shrink_tiles(rp) + rp / 16) * 64;
}
constexpr int shrink_lds_bytes(int rp) { return shrink_waves(rp) * shrink_wave_pieces(rp) * 16; }
static_assert(shrink_wave_pieces(128) * 16 >= 16 * 128 * 4 &&
                  shrink_wave_pieces(64) * 16 >= 16 * 64 * 4 &&
                  shrink_wave_pieces(16) * 16 >= 16 * 16 * 4,
              "the sums of 16 rows meet in the same LDS");

// Grid: (groups of T tiles, and for T = 2 the adapters; K parts); part y sums columns [y * kpart,
// (y + 1) * kpart) and writes sums[y][row][0 .. R).
//
// A lane of an MFMA operand holds one row's 8 columns, so sixteen neighbouring
// lanes want sixteen rows: read from memory that way, a 16-byte load costs the
// L1 an access per lane.  Here lanes read runs of 64 or 128 bytes of a row, and
// a wave turns them into operands in LDS that only it uses (no barrier in the
// loop); the next step's loads are in flight meanwhile.  Octet k of row r sits
// at lane 16 (k % 4) + (r ^ 2 k ^ r / 16) % 16 of its block of 16 rows: writes of
// a row's octets, or of every fourth row, and reads of a block's rows all spread
// over the banks.
//   TRANS false, W [R, C] (A in the forward): staged as x is.
//   TRANS true, W [C, R] (B in the backward): a lane reads V ranks of 8 columns
//   and turns them in registers.
// Bound by reading x at low rank: dy [8192, 8192] at rank 16 30 us (134 MB, 4.5
// TB/s; a library maximum over as much reads 3.0).  Workgroups that begin at
// different steps, against the memory channels that rows a multiple of 4 KiB apart
// share, take 28, but a row's sums then follow from the tile that it is in; two
// starting points over two sums gain nothing.  From rank 32 on the weights, read
// again by each tile, and the latency of a wave's steps count: 39 us at rank 32, 47
// at 64, 51 at 128; x [8192, 2048] at rank 64 17 us; [16384, 2048] at rank 128 52
// (as long with one tile a workgroup or steps of 64 columns).
template <int RP, bool TRANS, bool DROP>
__global__ __launch_bounds__(shrink_threads(RP), 2) void adapter_shrink_kernel(
    PlanView plan, int tiles_max, const uint16_t *__restrict__ src, uint32_t ld, int64_t C,
    const uint16_t *__restrict__ weights, const float *__restrict__ alpha, int R,
    float *__restrict__ sums, int64_t part_stride, int64_t kpart, DropoutArgs drop) {
    constexpr int STEP = shrink_step(RP), OCTS = STEP / 8, U = STEP / 32, J = RP / 16;
    constexpr int NW = shrink_waves(RP), T = shrink_tiles(RP), MB = 2 * T;
    constexpr int XI = T * TILE * OCTS / 64;             // 16-byte loads of x a lane and step
    constexpr int V = RP >= 64 ? 4 : 2;                  // ranks of a TRANS load
    constexpr int WI = TRANS ? RP / V * OCTS / 64 : RP * OCTS / 64;
    extern __shared__ u32x4 lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    u32x4 *lx = lds + wave * shrink_wave_pieces(RP), *lw = lx + U * MB * 64;
    // All of the plan's words for these tiles in one round trip.
    const bool built = plan.built();
    int tile0 = blockIdx.x * T;
    bool alone = false;
    if constexpr (T > 1) {
        const int pairs = (tiles_max + 1) / 2;
        if ((int)blockIdx.x >= pairs) {
            // An adapter whose first tile is the second of its pair.
            if (!built) return;
            const int a = blockIdx.x - pairs;
            tile0 = plan.group_tile0[a];
            alone = true;
            if ((tile0 & 1) == 0 || plan.group_tile0[a + 1] == tile0) return;
        }
    }
    const int32_t *tile_row = plan.tile_row + (int64_t)tile0 * TILE;
    int adapter[T], x_row[XI];
#pragma unroll
    for (int t = 0; t < T; ++t)
        adapter[t] = tile0 + t < tiles_max && (t == 0 || !alone)
                         ? plan.tile_adapter[tile0 + t] : -2;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int at = lane / OCTS + i * (64 / OCTS);
        // (a tile that there is not: its row is never stored)
        x_row[i] = tile_row[tile0 + at / TILE < tiles_max ? at : 0];
    }
    const int a = adapter[0];
    if (!built || a < 0) return;

    const int64_t kw = ((kpart + NW - 1) / NW + STEP - 1) / STEP * STEP;
    const int64_t k0 = blockIdx.y * kpart + wave * kw;
    const int64_t k1 = min(min(k0 + kw, (int64_t)(blockIdx.y + 1) * kpart), C);
    // Every workgroup takes its columns in one order, so that a row's sums do not
    // depend on the tile that it is in.
    const int steps = k0 < k1 ? (int)((k1 - k0 + STEP - 1) / STEP) : 0;
    const int oct = lane % OCTS;
    const DropoutKey key(DROP ? drop.rng : nullptr, DROP);
    const uint16_t *px[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        x_row[i] = (uint32_t)x_row[i] < (uint32_t)plan.rows ? x_row[i] : 0;   // unstored
        px[i] = row_at(src, x_row[i], ld);
    }

    const uint16_t *w = weights + (int64_t)a * R * C;
    u32x4 xr[XI];
    u32x4 wr[TRANS ? 1 : WI];                // TRANS false: as loaded
    Cols<V> tr[TRANS ? WI : 1][8];           // TRANS true: V ranks of 8 columns
    // Past the end both operands read the part's first columns and count as zero;
    // ranks past R read the first ranks, unstored.
    auto load = [&](int64_t kk) {
        const int64_t k = kk + 8 * oct, kc = k < k1 ? k : k0;
#pragma unroll
        for (int i = 0; i < XI; ++i) xr[i] = *reinterpret_cast<const u32x4 *>(px[i] + kc);
        if constexpr (!TRANS) {
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const int j = lane / OCTS + i * (64 / OCTS);
                wr[i] = *reinterpret_cast<const u32x4 *>(w + (j < R ? j : 0) * C + kc);
            }
        } else {
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const int item = lane + 64 * i, j = item % (RP / V) * V;
                const int64_t n = kk + 8 * (item / (RP / V)), nc = n < k1 ? n : k0;
#pragma unroll
                for (int e = 0; e < 8; ++e) tr[i][e].load(w + (nc + e) * R + (j < R ? j : 0));
            }
        }
    };
    auto slot = [](int o, int r) { return 16 * (o & 3) + ((r ^ (2 * o) ^ (r >> 4)) & 15); };
    auto stage = [&](int64_t kk) {
        const int64_t k = kk + 8 * oct;
        const bool tail = kk + STEP > k1;
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int r = lane / OCTS + i * (64 / OCTS);
            u32x4 v = xr[i];
            if constexpr (DROP)
                v = keep_chunk(v, key, (uint64_t)(x_row[i] * (C >> 3) + (k >> 3)), drop.threshold);
            if (tail)
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = k < k1 ? v[d] : 0u;
            lx[((oct >> 2) * MB + (r >> 4)) * 64 + slot(oct, r)] = v;
        }
        if constexpr (!TRANS) {
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const int j = lane / OCTS + i * (64 / OCTS);
                u32x4 v = wr[i];
                if (tail)
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[d] = k < k1 ? v[d] : 0u;
                lw[((oct >> 2) * J + (j >> 4)) * 64 + slot(oct, j)] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const int item = lane + 64 * i, j0 = item % (RP / V) * V, o = item / (RP / V);
#pragma unroll
                for (int t = 0; t < V; ++t) {
                    u32x4 v;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t a = tr[i][2 * d].d[t >> 1], b = tr[i][2 * d + 1].d[t >> 1];
                        v[d] = (t & 1) ? high_halves(a, b) : low_halves(a, b);
                    }
                    if (tail)
#pragma unroll
                        for (int d = 0; d < 4; ++d) v[d] = kk + 8 * o < k1 ? v[d] : 0u;
                    lw[((o >> 2) * J + ((j0 + t) >> 4)) * 64 + slot(o, j0 + t)] = v;
                }
            }
        }
    };

    f32x4 acc[MB][J];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int jb = 0; jb < J; ++jb) acc[mb][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (steps > 0) load(k0);
    for (int s = 0; s < steps; ++s) {
        stage(k0 + (int64_t)s * STEP);
        if (s + 1 < steps) load(k0 + (int64_t)(s + 1) * STEP);
        // A wave's LDS operations complete in issue order, so its reads see
        // every lane's writes and the next writes come after them; the
        // fences keep the compiler from moving them across.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int u = 0; u < U; ++u) {
            u32x4 xs[MB];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                xs[mb] = lx[(u * MB + mb) * 64 + slot(4 * u + g, 16 * mb + col)];
#pragma unroll
            for (int jb = 0; jb < J; ++jb) {
                const u32x4 b = lw[(u * J + jb) * 64 + slot(4 * u + g, 16 * jb + col)];
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[mb][jb] = mfma(xs[mb], b, acc[mb][jb]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    }
    // The waves' sums of 16 rows at a time, added in wave order, four ranks a
    // thread.
    float *red = reinterpret_cast<float *>(lds);
    const float scale = alpha[a] * drop.factor;
    constexpr int OUTS = (4 * RP + 64 * NW - 1) / (64 * NW);
    int out_row[MB][OUTS];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < OUTS; ++i)
            out_row[mb][i] =
                adapter[mb / 2] == a
                    ? tile_row[16 * mb + min((tid + 64 * NW * i) / (RP / 4), 15)] : -1;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        if (adapter[mb / 2] != a) continue;
        __syncthreads();
#pragma unroll
        for (int jb = 0; jb < J; ++jb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wave * 16 * RP + (4 * g + i) * RP + jb * 16 + col] = acc[mb][jb][i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < OUTS; ++i) {
            const int e = 4 * (tid + 64 * NW * i), j = e % RP;
            if (e >= 16 * RP) continue;
            f32x4 sum = *reinterpret_cast<const f32x4 *>(red + e);
#pragma unroll
            for (int n = 1; n < NW; ++n)
                sum += *reinterpret_cast<const f32x4 *>(red + n * 16 * RP + e);
            if (j < R && out_row[mb][i] >= 0)
                *reinterpret_cast<f32x4 *>(sums + blockIdx.y * part_stride +
                                           (int64_t)out_row[mb][i] * R + j) = scale * sum;
        }
    }
}

// ---- expand: out = base + f keep (h W) ---------------------------------------

// The dropout's numbers of L columns c .. (c a multiple of L).
template <int L>
__device__ __forceinline__ void numbers_of(const DropoutKey &key, int64_t row, int64_t c, int64_t C,
                                           uint32_t (&n)[L / 2]) {
    uint32_t w[4];
    dropout_words(key, (uint64_t)(row * (C >> 3) + (c >> 3)), w);
#pragma unroll
    for (int d = 0; d < L / 2; ++d) n[d] = L == 8 ? w[d] : (c & 4) ? w[2 + d] : w[d];
}

// Columns of an expand lane and threads of a workgroup of 512 columns.  Rank 128
// takes half the columns a lane, so that its weights and the tile ahead fit two
// waves' registers on a SIMD.
constexpr int expand_lane_cols(int rp) { return rp >= 128 ? 4 : 8; }
constexpr int expand_threads(int rp) { return kAdapterCols / expand_lane_cols(rp) * 4; }

// The weights of a lane's L columns c .. as MFMA columns of L blocks (block t:
// column c + t), S contraction steps of 32 ranks each.
//   TRANS false, W [C, R] (B in the forward): 8 ranks of a column are 16 bytes.
//   TRANS true, W [R, C] (A in the backward): a lane reads its L columns of its
//   8 ranks and turns them in registers.
template <int RP, bool TRANS, int S, int L>
__device__ __forceinline__ void load_expand_weights(const uint16_t *w, int64_t C, int R, int64_t c,
                                                    int g, u32x4 (&ws)[L][S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int j = RP == 16 ? 8 * (g & 1) : 32 * s + 8 * g;
        const bool ok = j < R;
        const int js = ok ? j : 0;
        if constexpr (!TRANS) {
#pragma unroll
            for (int t = 0; t < L; ++t)
                ws[t][s] = *reinterpret_cast<const u32x4 *>(w + (c + t) * R + js);
        } else {
            Cols<L> in[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) in[i].load(w + (int64_t)(js + i) * C + c);
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    ws[t][s][d] = (t & 1)
                                      ? high_halves(in[2 * d].d[t >> 1], in[2 * d + 1].d[t >> 1])
                                      : low_halves(in[2 * d].d[t >> 1], in[2 * d + 1].d[t >> 1]);
        }
        if (RP > 16 || R < 16) {
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d) ws[t][s][d] = ok ? ws[t][s][d] : 0u;
        }
    }
}

// Which chunk of tiles a workgroup takes: column blocks are the grid's fastest
// dimension, so that workgroups in flight together cover whole rows and with
// them all memory channels; the chunks are spread over the other two.
constexpr int64_t GRID_Y = 32768;
__device__ __forceinline__ int64_t chunk_of_block() {
    return (int64_t)blockIdx.z * GRID_Y + blockIdx.y;
}
dim3 grid_of(int64_t blocks, int64_t chunks) {
    return dim3((unsigned)blocks, (unsigned)std::min(chunks, GRID_Y),
                (unsigned)((chunks + GRID_Y - 1) / GRID_Y));
}

// The short operands of the weight gradients, split into bf16 parts and laid
// out as MFMA operands once for all column blocks that read them:
// packed [tile][part][16 ranks][lane], lane l of a tile holding rank l % 16 of
// rows 8 (l / 16) ...
struct PackSide {
    const float *h;             // [parts][rows][R]
    int parts;
    u32x4 *packed;
};

__device__ __forceinline__ void pack_tile(const PackSide &side, const int32_t *tile_row,
                                          int64_t tile, int R, int64_t part_stride, int blocks) {
    for (int item = threadIdx.x; item < blocks * 64; item += blockDim.x) {
        const int jb = item >> 6, l = item & 63, j = 16 * jb + (l & 15);
        const int4 *q = reinterpret_cast<const int4 *>(tile_row + tile * TILE + 8 * (l >> 4));
        const int4 lo = q[0], hi = q[1];
        const int r[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        const float *p = side.h + (j < R ? j : 0);
        for (int s = 0; s < side.parts; ++s, p += part_stride)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += p[(int64_t)max(r[i], 0) * R];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r[i] >= 0 && j < R ? v[i] : 0.0f;
        u32x4 part[kAdapterGradParts];
        split8(v, part);
#pragma unroll
        for (int n = 0; n < kAdapterGradParts; ++n)
            side.packed[((tile * kAdapterGradParts + n) * blocks + jb) * 64 + l] = part[n];
    }
}

struct PackArgs {
    PackSide g, h;
    int64_t rows;               // rows of the expand's grid that pack; 0: nothing to pack
};

// Grid: (blocks of 512 columns, chunks of tiles); in the backward rows of
// workgroups before them pack both short operands of the weight gradients.
// h is the MFMA's row operand and a lane's L adjacent columns are L column
// blocks, so a lane holds L adjacent columns of rows 4 g .. 4 g + 3 of the result
// and the sixteen lanes of a row load the base and store the output in one run of
// 256 (rank 128: 128) bytes.  The workgroup sums h's parts, splits h and lays it
// out in LDS as MFMA operands once for its waves (each wave reading it from
// memory by itself made the L1 the bound: 2.3 GB through it for 200 MB of base
// and output).  A wave keeps the weights of its columns while its tiles' adapter
// stays the same.
// Bound by base and output: [8192, 8192] at rank 16 49 us (268 MB, 5.5 TB/s),
// [8192, 6144] at rank 64 48 (201 MB, 4.2 TB/s).  [16384, 8192] at rank 128 137 to
// 143 (537 MB, 3.8 TB/s): there the two bf16 parts' 69 GFLOP take a fifth of the
// cycles and the vector work of a tile (h's split, addresses, sums) a third.
template <int RP, bool TRANS, bool DROP>
__global__ __launch_bounds__(expand_threads(RP), 2) void adapter_expand_kernel(
    PlanView plan, int tiles_max, int chunk, const float *h, int parts, int64_t part_stride,
    const uint16_t *__restrict__ weights, int R, int64_t C, const uint16_t *base, uint32_t ldbase,
    uint16_t *out, uint32_t ldo, float *h_out, PackArgs pack, DropoutArgs drop) {
    // RP = 16: one contraction step, ranks 0 .. 15 of h's high part in its
    // first half and of the low part in its second.
    constexpr int S = RP == 16 ? 1 : RP / 32;
    constexpr int P = RP == 16 ? 1 : 2;
    constexpr int OCTS = RP / 8;                               // groups of 8 ranks in a row
    constexpr int L = expand_lane_cols(RP), NT = expand_threads(RP);
    constexpr int ITEMS = (TILE * OCTS + NT - 1) / NT;
    // Ranks up to 32: one tile a workgroup and more of those on a CU instead.
    constexpr bool AHEAD = RP >= 64;
    __shared__ u32x4 hs[AHEAD ? 2 : 1][2][S][P][64];     // [buffer][half][step][part][lane]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int64_t c_lane = (int64_t)blockIdx.x * kAdapterCols + wave * (16 * L) + L * col;
    const bool c_ok = c_lane < C;
    const int64_t c = c_ok ? c_lane : 0;     // lanes past the end compute column 0, unstored
    int64_t part = chunk_of_block();
    if constexpr (TRANS) {
        // The first pack.rows rows of the grid pack a tile each (they start
        // first: a late one would be the kernel's tail).
        if (part < pack.rows) {
            const int64_t tile = part * gridDim.x + blockIdx.x;
            if (tile >= tiles_max || !plan.built() || plan.tile_adapter[tile] < 0) return;
            pack_tile(pack.g, plan.tile_row, tile, R, part_stride, RP / 16);
            pack_tile(pack.h, plan.tile_row, tile, R, 0, RP / 16);
            return;
        }
        part -= pack.rows;
    }
    const int64_t tile0 = part * chunk;
    const int tile1 = (int)min(tile0 + chunk, (int64_t)tiles_max);
    if (tile0 >= tile1 || out == nullptr) return;

    // A tile's words of the plan: its adapter, the rows of h that this thread
    // stages and the rows of the result that this lane holds.
    struct Ids {
        int a, h[ITEMS];
        int4 rows[2];
    };
    auto load_ids = [&](int64_t tile) {
        Ids d;
        const int32_t *p = plan.tile_row + tile * TILE;
        d.a = plan.tile_adapter[tile];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) d.h[it] = p[min((tid + it * NT) / OCTS, TILE - 1)];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
            d.rows[mb] = *reinterpret_cast<const int4 *>(p + 16 * mb + 4 * g);
        return d;
    };
    Ids next = load_ids(tile0), after{};
    if (AHEAD && tile0 + 1 < tile1) after = load_ids(tile0 + 1);
    if (!plan.built()) return;
    const bool in_place = base == out && ldbase == ldo;
    const DropoutKey key(DROP ? drop.rng : nullptr, DROP);

    // The tile ahead: its values of h (the first K part) and its base, as loaded:
    // nothing is done to them before their tile's turn, so nothing waits.  (A
    // position without a row reads row 0; without a base all read the output's
    // row 0, which stays in the caches.)
    f32x4 h_ahead[ITEMS][2];
    Cols<L> ahead[2][4];
    const uint16_t *bases_at = base ? base : out;
    const uint32_t ld_bases = base ? ldbase : 0u;
    auto h_at = [&](int row, int it) {
        const int j = 8 * ((tid + it * NT) % OCTS);
        return h + (int64_t)max(row, 0) * R + (j < R ? j : 0);
    };
    auto load_data = [&](const Ids &d) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const float *p = h_at(d.h[it], it);
            h_ahead[it][0] = *reinterpret_cast<const f32x4 *>(p);
            h_ahead[it][1] = *reinterpret_cast<const f32x4 *>(p + 4);
        }
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
            const int rows[4] = {d.rows[mb].x, d.rows[mb].y, d.rows[mb].z, d.rows[mb].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ahead[mb][i].load_once(row_at(bases_at + c, max(rows[i], 0), ld_bases));
        }
    };

    if (next.a != -2) load_data(next);
    u32x4 ws[L][S];
    int a_held = -1, buf = 0;
    for (int tile = (int)tile0; tile < tile1; ++tile) {
        const Ids now = next;
        const int a = now.a;
        if (a == -2) return;
        // The plan's words two tiles ahead, the data one.
        next = after;
        if (AHEAD && tile + 2 < tile1) after = load_ids(tile + 2);
        if (a >= 0 && a != a_held) {
            load_expand_weights<RP, TRANS, S, L>(weights + (int64_t)a * R * C, C, R, c, g, ws);
            a_held = a;
        }
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const int item = tid + it * NT, p = item / OCTS, o = item % OCTS;
            const bool ok = a >= 0 && now.h[it] >= 0 && 8 * o < R;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = ok ? h_ahead[it][i >> 2][i & 3] : 0.0f;
            // Few rows: the other parts, three in flight at a time.
            for (int s0 = 1; s0 < parts; s0 += 3) {
                const float *first = h_at(now.h[it], it);
                f32x4 q[3][2];
#pragma unroll
                for (int s = 0; s < 3; ++s) {
                    const float *at = first + min(s0 + s, parts - 1) * part_stride;
                    q[s][0] = *reinterpret_cast<const f32x4 *>(at);
                    q[s][1] = *reinterpret_cast<const f32x4 *>(at + 4);
                }
#pragma unroll
                for (int s = 0; s < 3; ++s)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] += ok && s0 + s < parts ? q[s][i >> 2][i & 3] : 0.0f;
            }
            if (h_out != nullptr && (a < 0 || parts > 1) && blockIdx.x == 0 &&
                item < TILE * OCTS && now.h[it] >= 0 && 8 * o < R) {
                float *to = h_out + (int64_t)now.h[it] * R + 8 * o;
                *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4 *>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
            u32x4 part[2];
            split8<2>(v, part);
            if (a >= 0 && item < TILE * OCTS) {
                if constexpr (RP == 16) {
                    hs[buf][p >> 4][0][0][16 * o + (p & 15)] = part[0];
                    hs[buf][p >> 4][0][0][32 + 16 * o + (p & 15)] = part[1];
                } else {
                    hs[buf][p >> 4][o >> 2][0][16 * (o & 3) + (p & 15)] = part[0];
                    hs[buf][p >> 4][o >> 2][P - 1][16 * (o & 3) + (p & 15)] = part[1];
                }
            }
        }
        Cols<L> bases[2][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int i = 0; i < 4; ++i) bases[mb][i] = ahead[mb][i];
        if (base == nullptr) {
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                for (int i = 0; i < 4; ++i) bases[mb][i].clear_unless(false);
        }
        // Before this tile's stores: a load that follows a store waits for it.
        if (AHEAD && tile + 1 < tile1 && next.a != -2) load_data(next);
        int rows[2][4];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
            rows[mb][0] = now.rows[mb].x, rows[mb][1] = now.rows[mb].y;
            rows[mb][2] = now.rows[mb].z, rows[mb][3] = now.rows[mb].w;
        }
        if (a < 0) {
            // Rows without an adapter: out = base.
            if (!in_place && c_ok) {
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (rows[mb][i] >= 0)
                            bases[mb][i].store(row_at(out + c, rows[mb][i], ldo));
            }
            if constexpr (!AHEAD) return;
            continue;
        }
        // Two buffers: the next tile is staged while slower waves still read
        // this one.
        __syncthreads();
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
            f32x4 acc[L];
#pragma unroll
            for (int t = 0; t < L; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            // The next step's operands are read while this one's are used.
            u32x4 operand[2][P];
#pragma unroll
            for (int p = 0; p < P; ++p) operand[0][p] = hs[buf][mb][0][p][lane];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (s + 1 < S)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        operand[(s + 1) & 1][p] = hs[buf][mb][s + 1][p][lane];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int t = 0; t < L; ++t)
                        acc[t] = mfma(operand[s & 1][p], ws[t][s], acc[t]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = rows[mb][i];
                if (row < 0 || !c_ok) continue;
                uint32_t n[L / 2];
                if constexpr (DROP) numbers_of<L>(key, row, c, C, n);
                Cols<L> o;
#pragma unroll
                for (int d = 0; d < L / 2; ++d) {
                    float lo = acc[2 * d][i], hi = acc[2 * d + 1][i];
                    if constexpr (DROP) {
                        lo = (n[d] & 0xFFFFu) >= drop.threshold ? lo * drop.factor : 0.0f;
                        hi = (n[d] >> 16) >= drop.threshold ? hi * drop.factor : 0.0f;
                    }
                    lo += __uint_as_float(bases[mb][i].d[d] << 16);
                    hi += __uint_as_float(bases[mb][i].d[d] & 0xFFFF0000u);
                    o.d[d] = pack_bf16(lo, hi);
                }
                o.store(row_at(out + c, row, ldo));
            }
        }
        if constexpr (!AHEAD) return;        // its only tile
        buf ^= 1;
    }
}

// ---- few rows: shrink and expand in one launch ----------------------------------

// A of an adapter [R, K] as the MFMA's columns, read straight from memory (few
// rows): 8 contraction indices are 16 bytes.  Ranks past R read rank 0: their
// result columns are not used.
template <int RP>
__device__ __forceinline__ void load_small_weights(const uint16_t *w, int64_t K, int R, int64_t k,
                                                   int col, u32x4 (&out)[RP / 16]) {
#pragma unroll
    for (int jb = 0; jb < RP / 16; ++jb) {
        const int j = jb * 16 + col;
        out[jb] = *reinterpret_cast<const u32x4 *>(w + (j < R ? j : 0) * K + k);
    }
}

// A decode step's batch is bound by the launches and by the chain of loads, not
// by the bytes.  Here every column block of a tile computes the tile's whole h
// by itself (the adapter's A comes from the L2) and goes on to its columns of
// the output; the base and B are on their way while h is computed.
// Grid: (blocks of 512 columns, tiles).  Lane layouts as in the two kernels.
template <int RP, bool DROP>
__global__ __launch_bounds__(THREADS, 2) void adapter_small_kernel(
    PlanView plan, const uint16_t *__restrict__ x, uint32_t ldx, int64_t K,
    const uint16_t *__restrict__ wa, const uint16_t *__restrict__ wb,
    const float *__restrict__ alpha, int R, int64_t C, const uint16_t *base, uint32_t ldbase,
    uint16_t *out, uint32_t ldo, float *h_out, DropoutArgs drop) {
    constexpr int S = RP == 16 ? 1 : RP / 32, P = RP == 16 ? 1 : 2, L = 8, OCTS = RP / 8;
    __shared__ float red[WAVES][TILE * RP];
    __shared__ u32x4 hs[2][S][P][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int64_t c_lane = (int64_t)blockIdx.x * kAdapterCols + wave * (16 * L) + L * col;
    const bool c_ok = c_lane < C;
    const int64_t c = c_ok ? c_lane : 0;
    const int64_t tile = chunk_of_block();
    const int32_t *tile_row = plan.tile_row + tile * TILE;
    const int a = plan.tile_adapter[tile];
    int h_row[2], rows[2][4];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        h_row[mb] = tile_row[16 * mb + col];
        const int4 r = *reinterpret_cast<const int4 *>(tile_row + 16 * mb + 4 * g);
        rows[mb][0] = r.x, rows[mb][1] = r.y, rows[mb][2] = r.z, rows[mb][3] = r.w;
    }
    const int stage_row = tile_row[min(tid / OCTS, TILE - 1)];
    const bool two = tile_row[16] >= 0;                  // rows in the tile's second half
    if (!plan.built() || a == -2) return;

    Cols<L> bases[2][4];
    const bool in_place = base == out && ldbase == ldo;
    const bool read_base = base != nullptr && !(in_place && a < 0);
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (read_base && (mb == 0 || two))
                bases[mb][i].load(row_at(base + c, max(rows[mb][i], 0), ldbase));
            else
                bases[mb][i].clear_unless(false);
        }
    const int so = tid % OCTS, sp = tid / OCTS;          // the 8 ranks of a row this thread sums
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    auto store_h = [&]() {
        if (h_out != nullptr && blockIdx.x == 0 && sp < TILE && stage_row >= 0 && 8 * so < R) {
            float *to = h_out + (int64_t)stage_row * R + 8 * so;
            *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4 *>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    };
    if (a < 0) {
        store_h();
        if (in_place || !c_ok) return;
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (rows[mb][i] >= 0) bases[mb][i].store(row_at(out + c, rows[mb][i], ldo));
        return;
    }
    u32x4 ws[L][S];
    load_expand_weights<RP, false, S, L>(wb + (int64_t)a * R * C, C, R, c, g, ws);

    const DropoutKey key(DROP ? drop.rng : nullptr, DROP);
    const uint16_t *w = wa + (int64_t)a * R * K;
    const int64_t kw = ((K + WAVES - 1) / WAVES + 31) / 32 * 32;
    const int64_t k0 = wave * kw, k1 = min(k0 + kw, K);
    const uint16_t *px[2];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        h_row[mb] = max(h_row[mb], 0);
        px[mb] = row_at(x, h_row[mb], ldx);
    }
    f32x4 acc[2][RP / 16];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int jb = 0; jb < RP / 16; ++jb) acc[mb][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = RP >= 64 ? 4 : 8;
    for (int64_t kk = k0; kk < k1; kk += 32 * U) {
        u32x4 xs[U][2], as[U][RP / 16];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = kk + 32 * u + 8 * g, kc = k < k1 ? k : k0;
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
                if (mb == 0 || two) xs[u][mb] = *reinterpret_cast<const u32x4 *>(px[mb] + kc);
            load_small_weights<RP>(w, K, R, kc, col, as[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = kk + 32 * u + 8 * g;
            if (kk + 32 * U > k1) {
#pragma unroll
                for (int jb = 0; jb < RP / 16; ++jb)
#pragma unroll
                    for (int d = 0; d < 4; ++d) as[u][jb][d] = k < k1 ? as[u][jb][d] : 0u;
            }
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                if (mb == 1 && !two) continue;
                if constexpr (DROP)
                    xs[u][mb] = keep_chunk(xs[u][mb], key,
                                           (uint64_t)(h_row[mb] * (K >> 3) + (k >> 3)),
                                           drop.threshold);
#pragma unroll
                for (int d = 0; d < 4; ++d) xs[u][mb][d] = k < k1 ? xs[u][mb][d] : 0u;
#pragma unroll
                for (int jb = 0; jb < RP / 16; ++jb)
                    acc[mb][jb] = mfma(xs[u][mb], as[u][jb], acc[mb][jb]);
            }
        }
    }
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int jb = 0; jb < RP / 16; ++jb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wave][(16 * mb + 4 * g + i) * RP + jb * 16 + col] = acc[mb][jb][i];
    __syncthreads();
    const float scale = alpha[a] * drop.factor;
    if (sp < TILE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = sp * RP + 8 * so + i;
            v[i] = scale * (((red[0][e] + red[1][e]) + red[2][e]) + red[3][e]);
            v[i] = stage_row >= 0 && 8 * so < R ? v[i] : 0.0f;
        }
        u32x4 part[2];
        split8<2>(v, part);
        if constexpr (RP == 16) {
            hs[sp >> 4][0][0][16 * so + (sp & 15)] = part[0];
            hs[sp >> 4][0][0][32 + 16 * so + (sp & 15)] = part[1];
        } else {
            hs[sp >> 4][so >> 2][0][16 * (so & 3) + (sp & 15)] = part[0];
            hs[sp >> 4][so >> 2][P - 1][16 * (so & 3) + (sp & 15)] = part[1];
        }
    }
    store_h();
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        if (mb == 1 && !two) break;
        f32x4 sum[L];
#pragma unroll
        for (int t = 0; t < L; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const u32x4 operand = hs[mb][s][p][lane];
#pragma unroll
                for (int t = 0; t < L; ++t) sum[t] = mfma(operand, ws[t][s], sum[t]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (rows[mb][i] < 0 || !c_ok) continue;
            Cols<L> o;
#pragma unroll
            for (int d = 0; d < L / 2; ++d)
                o.d[d] = pack_bf16(sum[2 * d][i] + __uint_as_float(bases[mb][i].d[d] << 16),
                                   sum[2 * d + 1][i] +
                                       __uint_as_float(bases[mb][i].d[d] & 0xFFFF0000u));
            o.store(row_at(out + c, rows[mb][i], ldo));
        }
    }
}

// ---- weight gradients ---------------------------------------------------------

// One long operand of the weight gradients and the short one beside it:
// partial [slot][R][C] = sum over a chunk's rows of short[row, j] * src[row, c].
struct WgradSide {
    const uint16_t *src;
    uint32_t ld;                // bytes
    int64_t C;
    const u32x4 *packed;        // the short operand (pack_tile)
    float *partial;
    int drop;                   // src takes the dropout's mask
};

// Columns of a lane and threads of a workgroup of 512 columns.  Rank 128 takes
// half the columns a lane, so that its sums fit two waves' registers on a SIMD.
constexpr int wgrad_lane_cols(int rp) { return rp >= 128 ? 4 : 8; }
constexpr int wgrad_threads(int rp) { return kAdapterCols / wgrad_lane_cols(rp) * 4; }

// Grid: (column blocks of both sides, chunks of tiles).  Per tile of 32 rows a
// lane reads L columns of its 8 rows and turns them in registers into the
// operands of L MFMA row blocks (row q of block t is column L q + t of the
// wave's 16 L); the short operand comes through LDS, once for the workgroup.
// The next tile's loads of both are in flight while the current one is
// multiplied.
// Bound by x and dy at low rank: [8192, 2048 + 8192] at rank 16 40 us (168 MB,
// 4.2 TB/s), at rank 32 45, at rank 64 62 (10 registers spill, 16 with dropout).  At
// rank 128, [16384, 2048 + 8192], 144 to 155 us: three bf16 parts make 129 GFLOP of
// 43, 0.83 to 0.89 PFLOP/s where a large library product reaches 1.24.
template <int RP, bool DROP>
__global__ __launch_bounds__(wgrad_threads(RP), 2) void adapter_wgrad_kernel(
    PlanView plan, WgradSide left, WgradSide right, int left_blocks, int R, int chunk,
    DropoutArgs drop) {
    constexpr int L = wgrad_lane_cols(RP), NT = wgrad_threads(RP);
    constexpr int PARTS = kAdapterGradParts, J = RP / 16, PIECES = PARTS * J * 64;
    constexpr int ITEMS = (PIECES + NT - 1) / NT;
    __shared__ u32x4 hs[2][PIECES];
    if (!plan.built()) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const bool first = (int)blockIdx.x < left_blocks;
    const WgradSide side = first ? left : right;
    const int block = first ? blockIdx.x : blockIdx.x - left_blocks;
    const int64_t C = side.C;
    const int64_t c_lane = (int64_t)block * kAdapterCols + wave * (16 * L) + L * col;
    const bool c_ok = c_lane < C;
    const int64_t c = c_ok ? c_lane : 0;     // lanes past the end compute column 0, unstored
    const uint16_t *src = side.src + c;
    const int live = plan.header[4];
    const int64_t slot = chunk_of_block();
    int tile = (int)min(slot * chunk, (int64_t)live);
    const int tile_end = min(tile + chunk, live);
    const DropoutKey key(DROP ? drop.rng : nullptr, DROP);

    // A lane's rows are read two tiles ahead, the operands one.
    struct Rows {
        int4 lo, hi;
        __device__ __forceinline__ int operator[](int i) const {
            const int r[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            return r[i];
        }
    };
    auto rows_of = [&](int t) {
        const int4 *p = reinterpret_cast<const int4 *>(plan.tile_row + (int64_t)t * TILE + 8 * g);
        return Rows{p[0], p[1]};
    };
    Rows rows, rows_next, rows_after;
    Cols<L> in[8], in_next[8];
    u32x4 h_next[ITEMS];
    auto load_tile = [&](int t, const Rows &r) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
            h_next[it] = side.packed[(int64_t)t * PIECES + min(tid + it * NT, PIECES - 1)];
#pragma unroll
        for (int i = 0; i < 8; ++i) in_next[i].load_once(row_at(src, max(r[i], 0), side.ld));
    };
    auto stage_short = [&](int buf) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
            if (PIECES % NT == 0 || tid + it * NT < PIECES) hs[buf][tid + it * NT] = h_next[it];
    };

    while (tile < tile_end) {
        const int a = plan.tile_adapter[tile];
        const int stop = min(tile_end, plan.group_tile0[a + 1]);
        f32x4 acc[L][J];
#pragma unroll
        for (int t = 0; t < L; ++t)
#pragma unroll
            for (int jb = 0; jb < J; ++jb) acc[t][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
        rows_next = rows_of(tile);
        rows_after = rows_of(min(tile + 1, stop - 1));
        load_tile(tile, rows_next);
        int buf = 0;
        __syncthreads();                     // the run before has read both buffers
        stage_short(0);
        __syncthreads();
        for (; tile < stop; ++tile, buf ^= 1) {
            rows = rows_next;
            rows_next = rows_after;
            if (tile + 2 < stop) rows_after = rows_of(tile + 2);
            // A position without a row: its short operand is zero, and its
            // long one may not be an infinity.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                in[i] = in_next[i];
                in[i].clear_unless(rows[i] >= 0);
            }
            if constexpr (DROP) {
                if (side.drop) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t n[L / 2];
                        numbers_of<L>(key, rows[i], c, C, n);
#pragma unroll
                        for (int d = 0; d < L / 2; ++d)
                            in[i].d[d] &= dropout_keep2(n[d], drop.threshold);
                    }
                }
            }
            const bool more = tile + 1 < stop;
            if (more) load_tile(tile + 1, rows_next);
            u32x4 xs[L];
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    xs[t][d] = (t & 1)
                                   ? high_halves(in[2 * d].d[t >> 1], in[2 * d + 1].d[t >> 1])
                                   : low_halves(in[2 * d].d[t >> 1], in[2 * d + 1].d[t >> 1]);
            // The operands are read two steps ahead of their use (a rank block ahead
            // takes twice the registers and at rank 64 a fifth longer).
            constexpr int STEPS = J * PARTS, RING = 3;
            auto operand = [&](int q) { return hs[buf][(q % PARTS * J + q / PARTS) * 64 + lane]; };
            u32x4 b[RING];
#pragma unroll
            for (int q = 0; q < min(RING - 1, STEPS); ++q) b[q] = operand(q);
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                if (q + RING - 1 < STEPS) b[(q + RING - 1) % RING] = operand(q + RING - 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < L; ++t)
                    acc[t][q / PARTS] = mfma(xs[t], b[q % RING], acc[t][q / PARTS]);
            }
            if (more) stage_short(buf ^ 1);
            __syncthreads();
        }
        float *out = side.partial + (slot + plan.group_rank[a]) * R * C;
        const int64_t n0 = c_lane - L * col;
#pragma unroll
        for (int jb = 0; jb < J; ++jb) {
            const int j = jb * 16 + col;
            if (j >= R) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t n = n0 + L * (4 * g + i);
                if (n >= C) continue;
                float *p = out + (int64_t)j * C + n;
#pragma unroll
                for (int t = 0; t < L; t += 4)
                    *reinterpret_cast<f32x4 *>(p + t) = f32x4{acc[t][jb][i], acc[t + 1][jb][i],
                                                              acc[t + 2][jb][i], acc[t + 3][jb][i]};
            }
        }
    }
}

template <int OUT>
__device__ __forceinline__ void store4(void *out, int64_t at, const float v[4]) {
    if constexpr (OUT == FP8_DTYPE_FP32) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + at) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(out) + at) =
            u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
    }
}

// Partial sums that a thread of the sum has in flight.
constexpr int SUM_UNROLL = 8;

// Adds an adapter's partial sums in chunk order; an adapter without rows gets
// zeros.  Grid: (blocks, adapters); a thread owns four results: of dA
// [R, in] (scaled by the dropout's factor) four columns of a rank; of dB
// [out, R], turned on the way, four ranks of a column.
template <int OUT>
__global__ __launch_bounds__(THREADS) void adapter_wgrad_sum_kernel(
    PlanView plan, const float *__restrict__ part_a, const float *__restrict__ part_b, int R,
    int64_t in, int64_t outs, int chunk, float factor, int64_t a_blocks, void *__restrict__ da,
    void *__restrict__ db) {
    if (!plan.built()) return;
    const int a = blockIdx.y;
    const int t0 = plan.group_tile0[a], t1 = plan.group_tile0[a + 1];
    const int slots = t1 > t0 ? (t1 - 1) / chunk - t0 / chunk + 1 : 0;
    const int64_t slot0 = t0 / chunk + (slots ? plan.group_rank[a] : 0);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if ((int64_t)blockIdx.x < a_blocks) {
        const int64_t e = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * 4;
        if (e >= R * in) return;
        const float *p = part_a + slot0 * R * in + e;
        const int64_t step = R * in;
        for (int s0 = 0; s0 < slots; s0 += SUM_UNROLL) {
            f32x4 q[SUM_UNROLL];
#pragma unroll
            for (int s = 0; s < SUM_UNROLL; ++s)
                q[s] = *reinterpret_cast<const f32x4 *>(p + min(s0 + s, slots - 1) * step);
#pragma unroll
            for (int s = 0; s < SUM_UNROLL; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += s0 + s < slots ? q[s][i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= factor;
        store4<OUT>(da, (int64_t)a * R * in + e, v);
    } else {
        const int64_t e = ((int64_t)blockIdx.x - a_blocks) * THREADS + threadIdx.x;
        const int64_t quads = R / 4;
        // Lanes over the columns within a quad of ranks: contiguous reads.
        const int64_t n = e % outs, q = e / outs;
        if (q >= quads) return;
        const float *p = part_b + slot0 * R * outs + q * 4 * outs + n;
        const int64_t step = R * outs;
        for (int s0 = 0; s0 < slots; s0 += SUM_UNROLL) {
            float w[SUM_UNROLL][4];
#pragma unroll
            for (int s = 0; s < SUM_UNROLL; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[s][i] = p[min(s0 + s, slots - 1) * step + i * outs];
#pragma unroll
            for (int s = 0; s < SUM_UNROLL; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += s0 + s < slots ? w[s][i] : 0.0f;
        }
        store4<OUT>(db, ((int64_t)a * outs + n) * R + q * 4, v);
    }
}

__global__ __launch_bounds__(THREADS) void adapter_clear_kernel(u32x4 *__restrict__ p,
                                                               int64_t pieces) {
    const int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (i < pieces) p[i] = u32x4{0u, 0u, 0u, 0u};
}

// ---- launches -----------------------------------------------------------------

uint32_t row_bytes(int64_t ld) { return (uint32_t)(2 * ld); }

template <typename F>
hipError_t by_rank(int rank, F f) {
    if (rank <= 16) f(std::integral_constant<int, 16>{});
    else if (rank <= 32) f(std::integral_constant<int, 32>{});
    else if (rank <= 64) f(std::integral_constant<int, 64>{});
    else f(std::integral_constant<int, 128>{});
    return hipGetLastError();
}

int64_t part_columns(int64_t C, int parts) { return ((C + parts - 1) / parts + 63) / 64 * 64; }

template <bool TRANS>
hipError_t launch_shrink(const AdapterArgs &w, const AdapterPlanShape &shape, const int32_t *plan,
                         const DropoutArgs &drop, const uint16_t *src, int64_t ld, int64_t C,
                         float *sums, int parts, hipStream_t stream) {
    const PlanView v = view_of(shape, plan);
    hipError_t enabled = hipSuccess;
    const hipError_t e = by_rank(w.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value, bytes = shrink_lds_bytes(RP), T = shrink_tiles(RP);
        const dim3 grid((unsigned)(T > 1 ? (shape.tiles_max + 1) / 2 + shape.adapters
                                         : shape.tiles_max), (unsigned)parts);
        auto go = [&](auto dropped) {
            const auto kernel = adapter_shrink_kernel<RP, TRANS, decltype(dropped)::value>;
            static std::atomic<uint64_t> done{0};
            enabled = enable_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes, done);
            if (enabled) return;
            hipLaunchKernelGGL(kernel, grid, dim3(shrink_threads(RP)), bytes, stream, v,
                               (int)shape.tiles_max, src, row_bytes(ld), C, TRANS ? w.b : w.a, w.alpha,
                               w.rank, sums, shape.rows * w.rank, part_columns(C, parts), drop);
        };
        if constexpr (!TRANS) {
            if (drop.rng) return go(std::true_type{});
        }
        go(std::false_type{});
    });
    return enabled ? enabled : e;
}

template <bool TRANS>
hipError_t launch_expand(const AdapterArgs &w, const AdapterPlanShape &shape, const int32_t *plan,
                         const DropoutArgs &drop, const float *h, int parts, int64_t C,
                         const uint16_t *base, int64_t ldbase, uint16_t *out, int64_t ldo,
                         float *h_out, const PackArgs &pack, hipStream_t stream) {
    const PlanView v = view_of(shape, plan);
    return by_rank(w.rank, [&](auto rp) {
        const int64_t blocks = (C + kAdapterCols - 1) / kAdapterCols;
        const int64_t chunk = adapter_expand_chunk(shape.tiles_max, C, w.rank);
        PackArgs packing = pack;
        packing.rows = pack.g.packed ? (shape.tiles_max + blocks - 1) / blocks : 0;
        // Without an output only the packing is done.
        const dim3 grid =
            grid_of(blocks, packing.rows + (out ? (shape.tiles_max + chunk - 1) / chunk : 0));
        auto go = [&](auto dropped) {
            hipLaunchKernelGGL((adapter_expand_kernel<decltype(rp)::value, TRANS,
                                                      decltype(dropped)::value>),
                               grid, dim3(expand_threads(decltype(rp)::value)), 0, stream, v,
                               (int)shape.tiles_max, (int)chunk, h, parts, shape.rows * w.rank,
                               TRANS ? w.a : w.b, w.rank, C, base, row_bytes(ldbase), out,
                               row_bytes(ldo), h_out, packing, drop);
        };
        if constexpr (TRANS) {
            if (drop.rng) return go(std::true_type{});
        }
        go(std::false_type{});
    });
}

// Whether the forward runs in one launch (adapter_small_kernel).  Its column
// blocks read each tile's A again, 16 rows at a time.  Measured against the two
// launches (us, in a graph and, in brackets, of an eager call):
//   A of 64 KiB, one token                           5.7 : 7.3   (10.5 : 13.4)
//   64 tokens, 32 adapters, 8 MiB of A read in all   6.5 : 7.9   (10.7 : 13.6)
//     16.5 MiB                                       6.6 : 7.9   (10.2 : 13.2)
//     33 MiB                                         9.7 : 9.2   (10.7 : 13.3)
//   64 tokens, 64 adapters, 64 MiB                  14.4 : 10.2  (14.8 : 13.5)
//   A of 128 KiB, 8 adapters, 4.5 MiB                8.5 : 8.6   (10.6 : 13.4)
//     20 MiB                                         9.1 : 8.9   (10.4 : 13.2)
// A bound of 34 MiB takes what an eager call gains, 3 us of the host's time for the
// launch saved, against 0.5 that a graph loses between 17 and 34 MiB.  A of 256 KiB
// is a third slower, and so are 64 rows an adapter from 128 KiB on.
bool one_launch(const AdapterArgs &w, const AdapterPlanShape &shape) {
    const int64_t blocks = (w.out + kAdapterCols - 1) / kAdapterCols;
    const int64_t a_bytes = adapter_padded_rank(w.rank) * w.in * 2;
    const int64_t most = a_bytes > (64 << 10) ? 17 << 20 : 34 << 20;
    return w.rank <= 64 && shape.rows <= 16 * shape.adapters && shape.tiles_max <= GRID_Y &&
           a_bytes <= (128 << 10) && shape.tiles_max * blocks * a_bytes <= most;
}

hipError_t launch_small(const AdapterArgs &w, const AdapterPlanShape &shape, const int32_t *plan,
                        const DropoutArgs &drop, const uint16_t *x, int64_t ldx,
                        const uint16_t *base, int64_t ldbase, uint16_t *y, int64_t ldy, float *h,
                        hipStream_t stream) {
    const PlanView v = view_of(shape, plan);
    const dim3 grid = grid_of((w.out + kAdapterCols - 1) / kAdapterCols, shape.tiles_max);
    auto go = [&](auto rp, auto dropped) {
        hipLaunchKernelGGL((adapter_small_kernel<decltype(rp)::value, decltype(dropped)::value>),
                           grid, dim3(THREADS), 0, stream, v, x, row_bytes(ldx), w.in, w.a, w.b,
                           w.alpha, w.rank, w.out, base, row_bytes(ldbase), y, row_bytes(ldy), h,
                           drop);
    };
    auto by_drop = [&](auto rp) {
        if (drop.rng) go(rp, std::true_type{});
        else go(rp, std::false_type{});
    };
    if (w.rank <= 16) by_drop(std::integral_constant<int, 16>{});
    else if (w.rank <= 32) by_drop(std::integral_constant<int, 32>{});
    else by_drop(std::integral_constant<int, 64>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_plan(const int32_t *row_adapter, const AdapterPlanShape &shape,
                               int32_t *plan, hipStream_t stream) {
    hipLaunchKernelGGL(adapter_plan_groups_kernel, dim3(1), dim3(PLAN_THREADS), 0, stream,
                       row_adapter, (int32_t)shape.rows, (int32_t)shape.adapters, plan,
                       plan + shape.group_tile0, plan + shape.group_rank);
    hipLaunchKernelGGL(adapter_plan_rows_kernel, dim3((unsigned)(shape.adapters + 1)),
                       dim3(THREADS), 0, stream, row_adapter, (int32_t)shape.rows,
                       (int32_t)shape.adapters, (int32_t)shape.tiles_max,
                       plan + shape.group_tile0, plan + shape.tile_adapter, plan + shape.tile_row);
    return hipGetLastError();
}

hipError_t launch_adapter_clear_grads(const AdapterArgs &w, void *da, void *db, int out_dtype,
                                      hipStream_t stream) {
    const int64_t size = out_dtype == FP8_DTYPE_FP32 ? 4 : 2;
    for (int side = 0; side < 2; ++side) {
        // An adapter's elements are a multiple of 64: whole 16-byte pieces.
        const int64_t per = (side ? w.out : w.in) * w.rank * size / 16;
        char *p = static_cast<char *>(side ? db : da);
        const int64_t step = (int64_t)1 << 30;     // pieces of one launch
        for (int64_t at = 0, all = per * w.count; at < all; at += step) {
            const int64_t n = std::min(step, all - at);
            hipLaunchKernelGGL(adapter_clear_kernel, dim3((unsigned)((n + THREADS - 1) / THREADS)),
                               dim3(THREADS), 0, stream, reinterpret_cast<u32x4 *>(p) + at, n);
        }
    }
    return hipGetLastError();
}

hipError_t launch_adapter_fwd(const AdapterArgs &w, const AdapterPlanShape &shape,
                              const int32_t *plan, const DropoutArgs &drop, const uint16_t *x,
                              int64_t ldx, const uint16_t *base, int64_t ldbase, uint16_t *y,
                              int64_t ldy, float *h, void *ws, hipStream_t stream) {
    if (one_launch(w, shape))
        return launch_small(w, shape, plan, drop, x, ldx, base, ldbase, y, ldy, h, stream);
    const int parts = adapter_parts(shape.tiles_max, w.in, w.rank);
    float *sums = parts == 1 && h ? h : static_cast<float *>(ws);
    if (hipError_t e =
            launch_shrink<false>(w, shape, plan, drop, x, ldx, w.in, sums, parts, stream))
        return e;
    const DropoutArgs none = {nullptr, 0, 1.0f};
    return launch_expand<false>(w, shape, plan, none, sums, parts, w.out, base, ldbase, y, ldy, h,
                                PackArgs{}, stream);
}

hipError_t launch_adapter_backward(const AdapterArgs &w, const AdapterPlanShape &shape,
                                   const int32_t *plan, const DropoutArgs &drop,
                                   const uint16_t *x, int64_t ldx, const uint16_t *dy,
                                   int64_t lddy, const float *h, const uint16_t *base,
                                   int64_t ldbase, uint16_t *dx, int64_t lddx, void *da, void *db,
                                   int out_dtype, void *ws, hipStream_t stream) {
    const AdapterWorkspace layout(shape, w.rank, w.in, w.out);
    const int parts = adapter_parts(shape.tiles_max, w.out, w.rank);
    float *g = static_cast<float *>(ws);
    const DropoutArgs none = {nullptr, 0, 1.0f};
    if (hipError_t e = launch_shrink<true>(w, shape, plan, none, dy, lddy, w.out, g, parts, stream))
        return e;
    const int64_t packed = layout.packed / 2;
    char *at = static_cast<char *>(ws) + layout.sums;
    PackArgs pack{};
    if (da) {
        pack.g = {g, parts, reinterpret_cast<u32x4 *>(at)};
        pack.h = {h, 1, reinterpret_cast<u32x4 *>(at + packed)};
    }
    if (hipError_t e = launch_expand<true>(w, shape, plan, drop, g, parts, w.in, base, ldbase, dx,
                                           lddx, nullptr, pack, stream))
        return e;
    if (!da) return hipSuccess;
    const PlanView v = view_of(shape, plan);
    const int64_t chunk = adapter_chunk(shape.tiles_max, w.rank, w.in, w.out);
    const int64_t chunks = (shape.tiles_max + chunk - 1) / chunk;
    const int64_t slots = adapter_slots(shape, chunk);
    float *part_a = reinterpret_cast<float *>(at + layout.packed);
    float *part_b = part_a + slots * w.rank * w.in;
    const WgradSide left = {x, row_bytes(ldx), w.in, pack.g.packed, part_a, 1};
    const WgradSide right = {dy, row_bytes(lddy), w.out, pack.h.packed, part_b, 0};
    const int left_blocks = (int)((w.in + kAdapterCols - 1) / kAdapterCols);
    const int right_blocks = (int)((w.out + kAdapterCols - 1) / kAdapterCols);
    const dim3 grid = grid_of(left_blocks + right_blocks, chunks);
    hipError_t e = by_rank(w.rank, [&](auto rp) {
        auto go = [&](auto dropped) {
            hipLaunchKernelGGL((adapter_wgrad_kernel<decltype(rp)::value, decltype(dropped)::value>),
                               grid, dim3(wgrad_threads(decltype(rp)::value)), 0, stream, v, left,
                               right, left_blocks, w.rank, (int)chunk, drop);
        };
        if (drop.rng) go(std::true_type{});
        else go(std::false_type{});
    });
    if (e) return e;
    const int64_t a_blocks = (w.rank * w.in / 4 + THREADS - 1) / THREADS;
    const int64_t b_blocks = (w.rank * w.out / 4 + THREADS - 1) / THREADS;
    const dim3 sum_grid((unsigned)(a_blocks + b_blocks), (unsigned)w.count);
    if (out_dtype == FP8_DTYPE_FP32)
        hipLaunchKernelGGL(adapter_wgrad_sum_kernel<FP8_DTYPE_FP32>, sum_grid, dim3(THREADS), 0,
                           stream, v, part_a, part_b, w.rank, w.in, w.out, (int)chunk, drop.factor,
                           a_blocks, da, db);
    else
        hipLaunchKernelGGL(adapter_wgrad_sum_kernel<FP8_DTYPE_BF16>, sum_grid, dim3(THREADS), 0,
                           stream, v, part_a, part_b, w.rank, w.in, w.out, (int)chunk, drop.factor,
                           a_blocks, da, db);
    return hipGetLastError();
}

}  // namespace fp8dsl
