// Tokens sorted by expert, and back.
//
//   plan      a stable counting sort of the (token, choice) pairs by expert;
//   gather    y[slot(t, k)] = x[t], and zeros in the segments' other rows;
//   combine   y[t] = base[t] + sum over k of w[t, k] x[slot(t, k)];
//   backward  dw[t, k] = dy[t] . x[slot(t, k)], dx[slot(t, k)] = w[t, k] dy[t].
//
// (The gather with the cast is in the cast's file, whose tile it uses.)
//
// The rows' kernels move bytes: a token's row is read once for all its choices (gather,
// backward), an expert's row once (combine), and written in whole.  Everything about a
// pair comes from the plan, so no kernel searches.
//
// Measured on MI355X, where a large copy moves 5.1 TB/s (us a call on inputs that are not
// in the caches, and in brackets its bytes at that rate): gather of 4096 tokens x 2048
// to 8 of 64 experts 27.4 (27.0), combine of 16384 x 4096 with 4 choices onto a residual
// 161 (158), backward of 8192 x 2048 with 2 choices 34.1 (33.0), its weights alone of
// 1037 x 1160 with 6 choices 7.5 (3.0); in a graph, combine of 16 x 2048 2.7, plan of 64
// tokens with 8 of 64 experts 5.5 (one launch), of 65536 with 4 of 128 10.9 (two).
#include "expert.h"

#include "bf16.h"
#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- the plan ----------------------------------------------------------------

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_WAVES = PLAN_THREADS / 64;

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ int wave_inclusive(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d, 64);
        v += lane >= d ? up : 0;
    }
    return v;
}

// Ids that a lane reads at once.
constexpr int PLAN_IDS = 4;

// Calls what(id) for the ids of p0 .. p1 - 1, `stride` of them side by side, and for
// some that name no expert behind them.
template <typename What>
__device__ __forceinline__ void for_ids(const int32_t *__restrict__ ids, int64_t p0, int64_t p1,
                                        int lane, int stride, What what) {
    for (int64_t p = p0 + lane; p < p1; p += PLAN_IDS * stride) {
        uint32_t id[PLAN_IDS];
#pragma unroll
        for (int i = 0; i < PLAN_IDS; ++i)
            id[i] = p + i * stride < p1 ? (uint32_t)ids[p + i * stride] : 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < PLAN_IDS; ++i) what(id[i]);
    }
}

// Pairs of each expert in the workgroup's piece of the ids.
__global__ __launch_bounds__(PLAN_THREADS) void expert_count_kernel(
    const int32_t *__restrict__ ids, int64_t pairs, int64_t piece, int experts,
    int32_t *__restrict__ hist) {
    __shared__ int count[kExpertsMax];
    for (int e = threadIdx.x; e < experts; e += PLAN_THREADS) count[e] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * piece, p1 = min(pairs, p0 + piece);
    for_ids(ids, p0, p1, threadIdx.x, PLAN_THREADS, [&](uint32_t e) {
        if (e < (uint32_t)experts) atomicAdd(&count[e], 1);
    });
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += PLAN_THREADS)
        hist[(int64_t)blockIdx.x * experts + e] = count[e];
}

// Places the pairs of the workgroup's piece.  Each wave takes a run of the piece
// and counts its pairs per expert (LDS counters: a count does not depend on their
// order); the runs before it, in this piece and the earlier ones (hist), give the
// first place of each expert's pairs.  It then walks its run 64 pairs at a time:
// lanes that name the same expert find each other by ballots over the id's bits,
// and their order among these is their order in the batch.
//
// Bound by latency: a chain of loads, LDS passes and barriers.  Every workgroup adds
// up the counts of all pieces for itself (64 KB from the L2 at 128 experts), spread
// over all its threads with 16 loads in flight each: 65536 tokens with 4 of 128
// experts 10.9 us, 37 with a thread an expert and a load at a time.
__global__ __launch_bounds__(PLAN_THREADS) void expert_place_kernel(
    const int32_t *__restrict__ ids, int64_t pairs, int64_t piece, int pieces, int tokens,
    int top_k, int experts, int capacity, int rows, const int32_t *__restrict__ hist,
    int32_t *__restrict__ header, int32_t *__restrict__ offsets, int32_t *__restrict__ counts,
    int32_t *__restrict__ slots, int32_t *__restrict__ sources, int4 *__restrict__ tiles) {
    extern __shared__ int lds[];
    int *run = lds;                              // [waves][experts]
    int *all = run + PLAN_WAVES * experts;       // [experts] pairs of all pieces
    int *first = all + experts;                  // [experts + 1] first row
    int *tile0 = first + experts + 1;            // [experts + 1] first tile
    __shared__ int2 wave_sum[PLAN_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t p0 = (int64_t)blockIdx.x * piece, p1 = min(pairs, p0 + piece);
    const int64_t per_wave = ((p1 - p0 + PLAN_WAVES - 1) / PLAN_WAVES + 63) / 64 * 64;
    const int64_t w0 = min(p1, p0 + wave * per_wave), w1 = min(p1, w0 + per_wave);

    // run, all and (as the pairs of the earlier pieces) first.
    int *earlier = first;
    for (int i = tid; i < (PLAN_WAVES + 2) * experts; i += PLAN_THREADS) run[i] = 0;
    __syncthreads();
    // The first ids of the run, read once for both passes.
    uint32_t ids_of[PLAN_IDS];
    const auto read = [&](int64_t pw) {
#pragma unroll
        for (int i = 0; i < PLAN_IDS; ++i) {
            const int64_t p = pw + 64 * i + lane;
            ids_of[i] = p < w1 ? (uint32_t)ids[p] : 0xFFFFFFFFu;
        }
    };
    read(w0);
    if (pieces > 1) {
        int wide = 64;                           // threads side by side over the experts
        while (wide < experts && wide < PLAN_THREADS) wide *= 2;
        const int parts = PLAN_THREADS / wide, part = tid / wide;
        const int g0 = pieces * part / parts, g1 = pieces * (part + 1) / parts;
        for (int e = tid % wide; e < experts; e += wide) {
            int before = 0, total = 0;
            for (int g = g0; g < g1; g += 16) {
                int c[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    c[i] = g + i < g1 ? hist[(int64_t)(g + i) * experts + e] : 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    total += c[i];
                    before += g + i < (int)blockIdx.x ? c[i] : 0;
                }
            }
            atomicAdd(&all[e], total);
            atomicAdd(&earlier[e], before);
        }
    }
    const auto count = [&](uint32_t e) {
        if (e < (uint32_t)experts) atomicAdd(&run[wave * experts + e], 1);
    };
#pragma unroll
    for (int i = 0; i < PLAN_IDS; ++i) count(ids_of[i]);
    for_ids(ids, w0 + 64 * PLAN_IDS, w1, lane, 64, count);
    __syncthreads();
    // Pairs before each wave's run, and all pairs, of each expert.
    for (int e = tid; e < experts; e += PLAN_THREADS) {
        int before = earlier[e], c[PLAN_WAVES];
#pragma unroll
        for (int w = 0; w < PLAN_WAVES; ++w) c[w] = run[w * experts + e];
#pragma unroll
        for (int w = 0; w < PLAN_WAVES; ++w) {
            run[w * experts + e] = before;
            before += c[w];
        }
        if (pieces == 1) all[e] = before;
    }
    __syncthreads();
    // First row and tile of each segment: a scan over the experts, two a thread.
    static_assert(kExpertsMax <= 2 * PLAN_THREADS, "two experts a thread");
    int2 length[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * tid + i;
        const int l = e >= experts ? 0 : capacity ? capacity : (all[e] + 15) / 16 * 16;
        length[i] = int2{l, (l + kExpertTile - 1) / kExpertTile};
    }
    const int2 mine = {length[0].x + length[1].x, length[0].y + length[1].y};
    int2 sum = {wave_inclusive(mine.x, lane), wave_inclusive(mine.y, lane)};
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        sum.x += wave_sum[w].x;
        sum.y += wave_sum[w].y;
    }
    int2 at = {sum.x - mine.x, sum.y - mine.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * tid + i;
        if (e < experts) {
            first[e] = at.x;
            tile0[e] = at.y;
        }
        at.x += length[i].x;
        at.y += length[i].y;
        if (e == experts - 1) {
            first[experts] = at.x;
            tile0[experts] = at.y;
        }
    }
    __syncthreads();

    const int end = first[experts], ntiles = tile0[experts];
    if (blockIdx.x == 0) {
        if (tid == 0) {
            header[0] = kExpertMagic;
            header[1] = tokens;
            header[2] = top_k;
            header[3] = experts;
            header[4] = capacity;
            header[5] = ntiles;
            header[6] = end;
        }
        for (int e = tid; e <= experts; e += PLAN_THREADS) {
            offsets[e] = first[e];
            if (e < experts) counts[e] = capacity ? min(all[e], capacity) : all[e];
        }
    }
    // The tiles, spread over the workgroups; a tile's expert by bisection.
    for (int t = blockIdx.x * PLAN_THREADS + tid; t < ntiles; t += gridDim.x * PLAN_THREADS) {
        int lo = 0, hi = experts;                // tile0[lo] <= t < tile0[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (tile0[mid] <= t) lo = mid;
            else hi = mid;
        }
        tiles[t] = int4{(t - tile0[lo]) * kExpertTile, first[lo + 1] - first[lo], first[lo], 0};
    }
    // Slots without a pair: the ends of the segments (16 lanes each) and what lies
    // behind the last one.  Without a capacity an end is under 16 rows.  With one it is up
    // to all of them, and few long ends are slow: 8192 tokens with 2 of 8 experts 8.7 us
    // without, 13.0 at a capacity of 2560, 27.9 at 10240.
    for (int i = blockIdx.x * PLAN_THREADS + tid; i < 16 * experts; i += gridDim.x * PLAN_THREADS) {
        const int e = i / 16, kept = capacity ? min(all[e], capacity) : all[e];
        for (int r = first[e] + kept + (i & 15); r < first[e + 1]; r += 16) sources[r] = -1;
    }
    for (int64_t r = end + (int64_t)blockIdx.x * PLAN_THREADS + tid; r < rows;
         r += (int64_t)gridDim.x * PLAN_THREADS)
        sources[r] = -1;

    int *next = run + wave * experts;
    for (int64_t pw = w0; pw < w1; pw += PLAN_IDS * 64) {
        if (pw > w0) read(pw);
#pragma unroll
        for (int i = 0; i < PLAN_IDS; ++i) {
            const int64_t p = pw + 64 * i + lane;
            const uint32_t id = ids_of[i];
            const bool named = id < (uint32_t)experts;
            uint64_t same = __ballot(named);
            for (int b = 0; (1 << b) < experts; ++b) {
                const bool bit = (id >> b) & 1;
                const uint64_t votes = __ballot(bit);
                same &= bit ? votes : ~votes;
            }
            int slot = -1;
            if (named) {
                const int base = next[id];
                const int rank = base + __popcll(same & ((1ull << lane) - 1));
                wave_fence();
                if ((same >> lane) == 1ull) next[id] = rank + 1;     // the last of them
                if (!capacity || rank < capacity) slot = first[id] + rank;
            }
            wave_fence();
            if (p < w1) {
                slots[p] = slot;
                if (slot >= 0) sources[slot] = (int32_t)p;
            }
        }
    }
}

// ---- rows --------------------------------------------------------------------

constexpr int THREADS = 256;

// Row `row` (not negative) of a bf16 matrix with its stride in bytes.
__device__ __forceinline__ const char *row_at(const void *p, int row, uint32_t ld_bytes) {
    return static_cast<const char *>(p) + (uint64_t)(uint32_t)row * ld_bytes;
}
__device__ __forceinline__ char *row_at(void *p, int row, uint32_t ld_bytes) {
    return static_cast<char *>(p) + (uint64_t)(uint32_t)row * ld_bytes;
}

// Zeros in the rows of the segments that have no pair: the workgroups behind
// those of the tokens, ZERO_ROWS slots each (few, as a small batch is mostly such rows:
// with 256 slots 16 tokens of 8192 columns over 8 experts took 13.9 us, now 4.2).
constexpr int ZERO_ROWS = 16;
__device__ __forceinline__ void zero_rows(const ExpertView &plan, int64_t block, void *y,
                                          uint32_t ldy, int64_t groups) {
    const int row0 = (int)(block * ZERO_ROWS), end = plan.offsets[plan.experts];
    const int lane = threadIdx.x & 63, row = row0 + lane;
    // Every wave looks for itself.
    const bool none = lane < ZERO_ROWS && row < end && plan.sources[row] < 0;
    for (uint64_t left = __ballot(none); left; left &= left - 1) {
        char *to = row_at(y, row0 + __builtin_ctzll(left), ldy);
        for (int64_t g = threadIdx.x; g < groups; g += THREADS)
            *reinterpret_cast<u32x4 *>(to + 16 * g) = u32x4{0u, 0u, 0u, 0u};
    }
}

// A workgroup covers 2^tx_log2 groups of 8 columns of 256 / 2^tx_log2 tokens; a lane
// reads its 16 bytes once and writes them to each of the token's slots.
__global__ __launch_bounds__(THREADS) void expert_gather_kernel(
    ExpertView plan, const uint16_t *__restrict__ x, uint32_t ldx, uint16_t *__restrict__ y,
    uint32_t ldy, int64_t groups, int tx_log2, int64_t token_blocks) {
    if (!plan.built()) return;
    if (blockIdx.x >= token_blocks) {
        if (blockIdx.y == 0) zero_rows(plan, blockIdx.x - token_blocks, y, ldy, groups);
        return;
    }
    const int tx = 1 << tx_log2;
    const int64_t g = (int64_t)blockIdx.y * tx + (threadIdx.x & (tx - 1));
    const int64_t t = (int64_t)blockIdx.x * (THREADS >> tx_log2) + (threadIdx.x >> tx_log2);
    if (g >= groups || t >= plan.tokens) return;
    const u32x4 v = *reinterpret_cast<const u32x4 *>(row_at(x, (int)t, ldx) + 16 * g);
    for (int k = 0; k < plan.top_k; ++k) {
        const int slot = plan.slots[t * plan.top_k + k];
        if (slot >= 0) *reinterpret_cast<u32x4 *>(row_at(y, slot, ldy) + 16 * g) = v;
    }
}

// The same split; a lane keeps the fp32 sums of its 8 columns.
template <bool WEIGHTS>
__global__ __launch_bounds__(THREADS) void expert_combine_kernel(
    ExpertView plan, const uint16_t *__restrict__ x, uint32_t ldx,
    const float *__restrict__ weights, const uint16_t *base, uint32_t ldbase, uint16_t *y,
    uint32_t ldy, int64_t groups, int tx_log2) {
    if (!plan.built()) return;
    const int tx = 1 << tx_log2;
    const int64_t g = (int64_t)blockIdx.y * tx + (threadIdx.x & (tx - 1));
    const int64_t t = (int64_t)blockIdx.x * (THREADS >> tx_log2) + (threadIdx.x >> tx_log2);
    if (g >= groups || t >= plan.tokens) return;
    float sum[8];
    u32x4 b = {0u, 0u, 0u, 0u};
    if (base) b = *reinterpret_cast<const u32x4 *>(row_at(base, (int)t, ldbase) + 16 * g);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        sum[2 * d] = bf16_lo(b[d]);
        sum[2 * d + 1] = bf16_hi(b[d]);
    }
    for (int k = 0; k < plan.top_k; ++k) {
        const int64_t pair = t * plan.top_k + k;
        const int slot = plan.slots[pair];
        if (slot < 0) continue;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(row_at(x, slot, ldx) + 16 * g);
        const float w = WEIGHTS ? weights[pair] : 1.0f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            sum[2 * d] += w * bf16_lo(v[d]);
            sum[2 * d + 1] += w * bf16_hi(v[d]);
        }
    }
    u32x4 out;
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d] = bf16_bits(sum[2 * d]) | (bf16_bits(sum[2 * d + 1]) << 16);
    *reinterpret_cast<u32x4 *>(row_at(y, (int)t, ldy) + 16 * g) = out;
}

// dy[t] . x[slot] for up to PAIRS choices of a token at once, so that dy is read once
// for them and all their rows are in flight together.  2^tx_log2 lanes (64 or 256) take
// a token; their sums meet in a butterfly, and those of four waves in LDS in wave order.
//
// Bound by its bytes where tokens are many: 8192 x 2048, two choices, with dx 34 us (168
// MB, 4.9 TB/s; eight choices at once 40, a workgroup for each four 37), and by the chain
// plan, slots, rows where they are few (256 x 2048: 3.9 us in a graph).
constexpr int PAIRS = 4;
template <bool DX>
__global__ __launch_bounds__(THREADS) void expert_combine_backward_kernel(
    ExpertView plan, const uint16_t *__restrict__ dy, uint32_t lddy, const uint16_t *x,
    uint32_t ldx, const float *__restrict__ weights, float *__restrict__ dweights, uint16_t *dx,
    uint32_t lddx, int64_t groups, int tx_log2, int64_t token_blocks) {
    const bool built = plan.built();
    if (blockIdx.x >= token_blocks) {
        if (built) zero_rows(plan, blockIdx.x - token_blocks, dx, lddx, groups);
        return;
    }
    __shared__ float part[THREADS / 64][PAIRS];
    const int tx = 1 << tx_log2, lane = threadIdx.x & (tx - 1);
    // The same for the wave.
    const int t = __builtin_amdgcn_readfirstlane(
        (int)(blockIdx.x * (THREADS >> tx_log2) + (threadIdx.x >> tx_log2)));
    if (t >= plan.tokens) return;                        // with 256 lanes, the workgroup
    const char *row = row_at(dy, t, lddy);
    for (int k0 = 0; k0 < plan.top_k; k0 += PAIRS) {
        const int64_t pair = (int64_t)t * plan.top_k + k0;
        int slot[PAIRS];
        float w[PAIRS], sum[PAIRS];
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const bool there = k0 + j < plan.top_k;
            slot[j] = there ? plan.slots[pair + j] : -1;
            w[j] = DX && there ? weights[pair + j] : 0.0f;    // not used without a slot
            sum[j] = 0.0f;
        }
        if (!built) return;                              // read beside the slots
        for (int64_t g = lane; g < groups; g += tx) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(row + 16 * g);
            u32x4 v[PAIRS];
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
                if (slot[j] >= 0)
                    v[j] = *reinterpret_cast<const u32x4 *>(row_at(x, slot[j], ldx) + 16 * g);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                if (slot[j] < 0) continue;
                u32x4 out;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    sum[j] += bf16_lo(a[d]) * bf16_lo(v[j][d]);
                    sum[j] += bf16_hi(a[d]) * bf16_hi(v[j][d]);
                    out[d] = bf16_bits(w[j] * bf16_lo(a[d])) |
                             (bf16_bits(w[j] * bf16_hi(a[d])) << 16);
                }
                if constexpr (DX)
                    *reinterpret_cast<u32x4 *>(row_at(dx, slot[j], lddx) + 16 * g) = out;
            }
        }
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) sum[j] += __shfl_xor(sum[j], m, 64);
        if (tx > 64) {
            if (k0 > 0) __syncthreads();                 // the earlier sums have been read
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) part[threadIdx.x >> 6][j] = sum[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
                sum[j] = ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j];
        }
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
                if (k0 + j < plan.top_k) dweights[pair + j] = sum[j];
    }
}

// Lanes of a workgroup along the columns: a power of two that covers them, or 256.
int lanes_log2(int64_t groups) {
    int tx_log2 = 3;
    while (tx_log2 < 8 && (int64_t(1) << tx_log2) < groups) ++tx_log2;
    return tx_log2;
}

int64_t zero_blocks(const ExpertShape &shape) { return (shape.rows + ZERO_ROWS - 1) / ZERO_ROWS; }

}  // namespace

hipError_t launch_expert_plan(const ExpertShape &s, const int32_t *ids, int32_t *plan,
                              hipStream_t stream) {
    const int64_t piece = (s.pairs + s.pieces - 1) / s.pieces;
    if (s.pieces > 1) {
        hipLaunchKernelGGL(expert_count_kernel, dim3((unsigned)s.pieces), dim3(PLAN_THREADS), 0,
                           stream, ids, s.pairs, piece, s.experts, plan + s.hist);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int lds_bytes = (int)sizeof(int) * ((PLAN_WAVES + 3) * s.experts + 2);
    hipLaunchKernelGGL(expert_place_kernel, dim3((unsigned)s.pieces), dim3(PLAN_THREADS),
                       lds_bytes, stream, ids, s.pairs, piece, (int)s.pieces, (int)s.tokens,
                       s.top_k, s.experts, (int)s.capacity, (int)s.rows, plan + s.hist, plan,
                       plan + s.offsets, plan + s.counts, plan + s.slots, plan + s.sources,
                       reinterpret_cast<int4 *>(plan + s.tiles));
    return hipGetLastError();
}

hipError_t launch_expert_gather(const ExpertShape &s, const int32_t *plan, const uint16_t *x,
                                int64_t ldx, uint16_t *y, int64_t ldy, int64_t cols,
                                hipStream_t stream) {
    const int64_t groups = cols / 8;
    const int tx_log2 = lanes_log2(groups), tokens = THREADS >> tx_log2;
    const int64_t token_blocks = (s.tokens + tokens - 1) / tokens;
    const int64_t tx = int64_t(1) << tx_log2;
    const dim3 grid((unsigned)(token_blocks + zero_blocks(s)), (unsigned)((groups + tx - 1) / tx));
    hipLaunchKernelGGL(expert_gather_kernel, grid, dim3(THREADS), 0, stream, ExpertView(s, plan), x,
                       (uint32_t)(2 * ldx), y, (uint32_t)(2 * ldy), groups, tx_log2, token_blocks);
    return hipGetLastError();
}

hipError_t launch_expert_combine(const ExpertShape &s, const int32_t *plan, const uint16_t *x,
                                 int64_t ldx, const float *weights, const uint16_t *base,
                                 int64_t ldbase, uint16_t *y, int64_t ldy, int64_t cols,
                                 hipStream_t stream) {
    const int64_t groups = cols / 8;
    const int tx_log2 = lanes_log2(groups), tokens = THREADS >> tx_log2;
    const int64_t tx = int64_t(1) << tx_log2;
    const dim3 grid((unsigned)((s.tokens + tokens - 1) / tokens),
                    (unsigned)((groups + tx - 1) / tx));
    const auto kernel = weights ? expert_combine_kernel<true> : expert_combine_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, stream, ExpertView(s, plan), x,
                       (uint32_t)(2 * ldx), weights, base, (uint32_t)(2 * ldbase), y,
                       (uint32_t)(2 * ldy), groups, tx_log2);
    return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const ExpertShape &s, const int32_t *plan,
                                          const uint16_t *dy, int64_t lddy, const uint16_t *x,
                                          int64_t ldx, const float *weights, float *dweights,
                                          uint16_t *dx, int64_t lddx, int64_t cols,
                                          hipStream_t stream) {
    const int64_t groups = cols / 8;
    // A wave per token, or a workgroup where its row is longer than 1024 columns, with and
    // without dx: the weights' gradient has the same bits in both.  us with a wave / a
    // workgroup, two choices, with dx and without:
    //   1024 columns  16384 tokens 34.5 / 41.9, 19.4 / 28.3    1037 tokens 5.0 / 5.1, 3.7 / 4.2
    //   1160          14463        39.5 / 40.8, 19.7 / 26.6                6.1 / 5.7, 4.4 / 4.4
    //   1536          10922        36.6 / 35.9, 19.1 / 23.1                6.5 / 6.0, 4.6 / 4.6
    //   2048           8192        38.3 / 34.5, 19.5 / 21.5                7.7 / 7.1, 5.6 / 5.7
    //   4096           4096        39.2 / 35.0, 19.2 / 18.8               11.4 / 10.1, 8.0 / 8.0
    //   8192           2048        40.3 / 38.3, 20.9 / 19.6               23.1 / 17.5, 12.6 / 11.8
    // six choices, 1037 tokens: 1160 columns 12.6 / 10.6, 8.6 / 8.0; 2048 15.0 / 12.5, 10.0 /
    // 9.2.  So many tokens without dx pay for it up to 2048 columns.
    const int tx_log2 = groups > 128 ? 8 : 6, tokens = THREADS >> tx_log2;
    const int64_t token_blocks = (s.tokens + tokens - 1) / tokens;
    const dim3 grid((unsigned)(token_blocks + (dx ? zero_blocks(s) : 0)));
    const auto kernel = dx ? expert_combine_backward_kernel<true>
                           : expert_combine_backward_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, stream, ExpertView(s, plan), dy,
                       (uint32_t)(2 * lddy), x, (uint32_t)(2 * ldx), weights, dweights, dx,
                       (uint32_t)(2 * lddx), groups, tx_log2, token_blocks);
    return hipGetLastError();
}

}  // namespace fp8dsl
