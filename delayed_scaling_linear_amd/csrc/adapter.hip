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
// into bf16 parts that add up to them: two (the error is 2^-17 of h) where
// the result is rounded to bf16, three (2^-24) where it is stored in fp32.
// Dropout multiplies by the mask on the operand (exact) and by f in fp32 on
// the sums.
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
// rounded.  An infinity or NaN goes to the first part alone.
template <int PARTS>
__device__ __forceinline__ void split8(const float v[8], u32x4 (&out)[PARTS]) {
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
                const bool special = (u & 0x7F800000u) == 0x7F800000u;
                if (special && r != r) bits[k] |= 0x00400000u;
                r = special ? 0.0f : r - __uint_as_float(bits[k]);
            }
            out[p][d] = high_halves(bits[0], bits[1]);
        }
    }
}

// ---- the plan ---------------------------------------------------------------

struct PlanView {
    const int32_t *header, *group_tile0, *group_rank, *tile_adapter, *tile_row;
    int32_t rows, adapters;
    // A buffer that no plan of these sizes was written to has no work in it.
    __device__ __forceinline__ bool built() const {
        return header[0] == kPlanMagic && header[1] == rows && header[2] == adapters;
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

// W of adapter a as the contraction sees it: TRANS false, [R, C] (A in the
// forward): a lane's 8 contraction indices are 16 contiguous bytes; TRANS
// true, [C, R] (B in the backward): a lane reads RP / 16 adjacent ranks of
// its 8 rows and turns them in registers, so result column l % 16 of block jb
// is rank (l % 16) * (RP / 16) + jb.
template <int RP, bool TRANS>
__device__ __forceinline__ int shrink_rank(int jb, int col) {
    return TRANS ? col * (RP / 16) + jb : jb * 16 + col;
}

template <int RP, bool TRANS>
__device__ __forceinline__ void load_shrink_weights(const uint16_t *w, int64_t C, int R, int64_t k,
                                                    bool k_ok, int col, u32x4 (&out)[RP / 16]) {
    constexpr int W = RP / 16;
    if constexpr (!TRANS) {
#pragma unroll
        for (int jb = 0; jb < W; ++jb) {
            const int j = jb * 16 + col;
            out[jb] = u32x4{0u, 0u, 0u, 0u};
            if (k_ok && j < R) out[jb] = *reinterpret_cast<const u32x4 *>(w + j * C + k);
        }
    } else {
        uint32_t t[8][(W + 1) / 2];
        const int j = col * W;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int d = 0; d < (W + 1) / 2; ++d) t[i][d] = 0u;
            if (k_ok && j < R) {
                const uint16_t *p = w + (k + i) * R + j;
                if constexpr (W == 1) {
                    t[i][0] = *p;
                } else if constexpr (W == 2) {
                    t[i][0] = *reinterpret_cast<const uint32_t *>(p);
                } else if constexpr (W == 4) {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
                    t[i][0] = v.x;
                    t[i][1] = v.y;
                } else {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
                    for (int d = 0; d < 4; ++d) t[i][d] = v[d];
                }
            }
        }
#pragma unroll
        for (int jb = 0; jb < W; ++jb)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                out[jb][d] = (jb & 1) ? high_halves(t[2 * d][jb >> 1], t[2 * d + 1][jb >> 1])
                                      : low_halves(t[2 * d][jb >> 1], t[2 * d + 1][jb >> 1]);
    }
}

__device__ __forceinline__ u32x4 keep_chunk(u32x4 v, const DropoutKey &key, uint64_t e,
                                            uint32_t threshold) {
    uint32_t w[4];
    dropout_words(key, e, w);
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] &= dropout_keep2(w[d], threshold);
    return v;
}

// Grid: (tiles, K parts); part y sums columns [y * kpart, (y + 1) * kpart) and
// writes sums[y][row][0 .. R).
template <int RP, bool TRANS, bool DROP>
__global__ __launch_bounds__(THREADS) void adapter_shrink_kernel(
    PlanView plan, const uint16_t *__restrict__ src, int64_t ld, int64_t C,
    const uint16_t *__restrict__ weights, const float *__restrict__ alpha, int R,
    float *__restrict__ sums, int64_t part_stride, int64_t kpart, DropoutArgs drop) {
    __shared__ float red[WAVES][16 * RP];
    __shared__ int rows[TILE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    if (!plan.built()) return;
    const int tile = blockIdx.x, a = plan.tile_adapter[tile];
    if (a < 0) return;
    if (tid < TILE) rows[tid] = plan.tile_row[tile * TILE + tid];
    __syncthreads();
    const uint16_t *w = weights + (int64_t)a * R * C;

    int64_t kw = ((kpart + WAVES - 1) / WAVES + 31) / 32 * 32;   // a wave's columns
    const int64_t k0 = blockIdx.y * kpart + wave * kw;
    const int64_t k1 = min(min(k0 + kw, (int64_t)(blockIdx.y + 1) * kpart), C);

    const uint16_t *px[2];
    int64_t row[2];
    bool row_ok[2];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        const int r = rows[mb * 16 + col];
        row_ok[mb] = r >= 0;
        row[mb] = max(r, 0);
        px[mb] = src + row[mb] * ld;
    }
    f32x4 acc[2][RP / 16];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int jb = 0; jb < RP / 16; ++jb) acc[mb][jb] = f32x4{0.f, 0.f, 0.f, 0.f};

    constexpr int U = RP >= 128 ? 2 : 4;
    for (int64_t kk = k0; kk < k1; kk += 32 * U) {
        u32x4 xs[U][2], ws[U][RP / 16];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = kk + 32 * u + 8 * g;
            const bool ok = k < k1;
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                xs[u][mb] = u32x4{0u, 0u, 0u, 0u};
                if (ok && row_ok[mb]) xs[u][mb] = *reinterpret_cast<const u32x4 *>(px[mb] + k);
            }
            load_shrink_weights<RP, TRANS>(w, C, R, k, ok, col, ws[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (DROP) {
                const DropoutKey key(drop.rng);
                const int64_t k = kk + 32 * u + 8 * g;
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
                    xs[u][mb] = keep_chunk(xs[u][mb], key, (uint64_t)(row[mb] * (C >> 3) + (k >> 3)),
                                           drop.threshold);
            }
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                for (int jb = 0; jb < RP / 16; ++jb)
                    acc[mb][jb] = mfma(xs[u][mb], ws[u][jb], acc[mb][jb]);
        }
    }
    const float scale = alpha[a] * drop.factor;
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        if (mb) __syncthreads();
#pragma unroll
        for (int jb = 0; jb < RP / 16; ++jb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wave][(4 * g + i) * RP + shrink_rank<RP, TRANS>(jb, col)] = acc[mb][jb][i];
        __syncthreads();
        for (int e = tid; e < 16 * RP; e += THREADS) {
            const int r = rows[16 * mb + e / RP], j = e % RP;
            if (j < R && r >= 0)
                sums[blockIdx.y * part_stride + (int64_t)r * R + j] =
                    scale * (((red[0][e] + red[1][e]) + red[2][e]) + red[3][e]);
        }
    }
}

// ---- expand: out = base + f keep (h W) ---------------------------------------

// Eight ranks j .. j + 7 of one row of h, the K parts added in order.
__device__ __forceinline__ void load_h8(const float *h, int parts, int64_t part_stride, int R,
                                        int64_t row, int j, bool ok, float v[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (!ok) return;
    const float *p = h + row * R + j;
    for (int s = 0; s < parts; ++s, p += part_stride) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
        }
    }
}

// out = base + f keep v for eight columns of a row.
template <bool DROP>
__device__ __forceinline__ void add_store8(const float v[8], const uint16_t *base, uint16_t *out,
                                           uint64_t e, const DropoutArgs &drop) {
    u32x4 b = {0u, 0u, 0u, 0u}, o;
    if (base != nullptr) b = *reinterpret_cast<const u32x4 *>(base);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (DROP) {
        const DropoutKey key(drop.rng);
        dropout_words(key, e, w);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        float lo = v[2 * d], hi = v[2 * d + 1];
        if constexpr (DROP) {
            lo = (w[d] & 0xFFFFu) >= drop.threshold ? lo * drop.factor : 0.0f;
            hi = (w[d] >> 16) >= drop.threshold ? hi * drop.factor : 0.0f;
        }
        lo += __uint_as_float(b[d] << 16);
        hi += __uint_as_float(b[d] & 0xFFFF0000u);
        o[d] = bf16_rne(lo) | (bf16_rne(hi) << 16);
    }
    *reinterpret_cast<u32x4 *>(out) = o;
}

// Grid: (tiles, blocks of 512 columns).  The product is taken transposed
// (weights' columns are the MFMA rows), so a lane holds adjacent columns of
// one row of the output.  TRANS false: W [C, R] (B in the forward), MFMA row q
// of block t is column 8 (q / 4) + 4 t + q % 4 of 32: a lane holds 8 columns.
// TRANS true: W [R, C] (A in the backward): a lane reads 8 columns of its 8
// ranks and turns them in registers; row q of block t is column
// 32 (q % 4) + 8 (q / 4) + t of 128: a lane holds 4 x 8 columns.
template <int RP, bool TRANS, bool DROP>
__global__ __launch_bounds__(THREADS) void adapter_expand_kernel(
    PlanView plan, const float *h, int parts, int64_t part_stride,
    const uint16_t *__restrict__ weights, int R, int64_t C, const uint16_t *base, int64_t ldbase,
    uint16_t *out, int64_t ldo, float *h_out, DropoutArgs drop) {
    __shared__ int rows[TILE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    if (!plan.built()) return;
    const int tile = blockIdx.x, a = plan.tile_adapter[tile];
    if (a == -2) return;
    if (tid < TILE) rows[tid] = plan.tile_row[tile * TILE + tid];
    __syncthreads();
    if (h_out != nullptr && blockIdx.y == 0 && (a < 0 || parts > 1)) {
        for (int e = tid; e < TILE * (R / 8); e += THREADS) {
            const int r = rows[e / (R / 8)], j = e % (R / 8) * 8;
            if (r < 0) continue;
            float v[8];
            load_h8(h, parts, part_stride, R, r, j, a >= 0, v);
            float *p = h_out + (int64_t)r * R + j;
            *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
    const int64_t c0 = (int64_t)blockIdx.y * kAdapterCols;
    if (a < 0) {
        // Rows without an adapter: out = base.
        if (base == out && ldbase == ldo) return;
        const int64_t c = c0 + 8 * lane;
        if (c >= C) return;
        for (int p = wave; p < TILE; p += WAVES) {
            if (rows[p] < 0) break;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (base) v = *reinterpret_cast<const u32x4 *>(base + rows[p] * ldbase + c);
            *reinterpret_cast<u32x4 *>(out + rows[p] * ldo + c) = v;
        }
        return;
    }
    const uint16_t *w = weights + (int64_t)a * R * C;

    // h as the MFMA columns: S contraction steps of 32 ranks, high and low
    // parts.  RP = 16: one step, ranks 0 .. 15 of the high part in its first
    // half and of the low part in its second.
    constexpr int S = RP == 16 ? 1 : RP / 32;
    constexpr int P = RP == 16 ? 1 : 2;
    u32x4 hs[2][S][P];
    int64_t row[2];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        row[mb] = rows[mb * 16 + col];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = RP == 16 ? 8 * (g & 1) : 32 * s + 8 * g;
            float v[8];
            load_h8(h, parts, part_stride, R, row[mb], j, row[mb] >= 0 && j < R, v);
            u32x4 part[2];
            split8<2>(v, part);
            if constexpr (RP == 16)
                hs[mb][s][0] = g < 2 ? part[0] : part[1];
            else {
                hs[mb][s][0] = part[0];
                hs[mb][s][P - 1] = part[1];
            }
        }
    }

    const int64_t cw = c0 + wave * (kAdapterCols / WAVES);
    if constexpr (!TRANS) {
#pragma unroll 2
        for (int step = 0; step < 4; ++step) {
            const int64_t c = cw + 32 * step;
            if (c >= C) return;
            f32x4 acc[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t n = c + 8 * (col >> 2) + 4 * t + (col & 3);
                u32x4 ws[S];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int j = RP == 16 ? 8 * (g & 1) : 32 * s + 8 * g;
                    ws[s] = u32x4{0u, 0u, 0u, 0u};
                    if (n < C && j < R) ws[s] = *reinterpret_cast<const u32x4 *>(w + n * R + j);
                }
#pragma unroll
                for (int mb = 0; mb < 2; ++mb) {
                    acc[mb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            acc[mb][t] = mfma(ws[s], hs[mb][s][p], acc[mb][t]);
                }
            }
            const int64_t n = c + 8 * g;
            if (n < C) {
#pragma unroll
                for (int mb = 0; mb < 2; ++mb) {
                    if (row[mb] < 0) continue;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = acc[mb][0][i];
                        v[4 + i] = acc[mb][1][i];
                    }
                    add_store8<DROP>(v, base ? base + row[mb] * ldbase + n : nullptr,
                                     out + row[mb] * ldo + n,
                                     (uint64_t)(row[mb] * (C >> 3) + (n >> 3)), drop);
                }
            }
        }
    } else {
        if (cw >= C) return;
        f32x4 acc[2][8];
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[mb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t k = cw + 32 * (col & 3) + 8 * (col >> 2);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = RP == 16 ? 8 * (g & 1) : 32 * s + 8 * g;
            u32x4 in[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                in[i] = u32x4{0u, 0u, 0u, 0u};
                if (k < C && j < R)
                    in[i] = *reinterpret_cast<const u32x4 *>(w + (int64_t)(j + i) * C + k);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u32x4 ws;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    ws[d] = (t & 1) ? high_halves(in[2 * d][t >> 1], in[2 * d + 1][t >> 1])
                                    : low_halves(in[2 * d][t >> 1], in[2 * d + 1][t >> 1]);
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[mb][t] = mfma(ws, hs[mb][s][p], acc[mb][t]);
            }
        }
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
            if (row[mb] < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t n = cw + 32 * i + 8 * g;
                if (n >= C) continue;
                float v[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = acc[mb][t][i];
                add_store8<DROP>(v, base ? base + row[mb] * ldbase + n : nullptr,
                                 out + row[mb] * ldo + n,
                                 (uint64_t)(row[mb] * (C >> 3) + (n >> 3)), drop);
            }
        }
    }
}

// ---- weight gradients ---------------------------------------------------------

// One long operand of the weight gradients and the short one beside it:
// part [slot][R][C] = sum over a chunk's rows of short[row, j] * src[row, c].
struct WgradSide {
    const uint16_t *src;
    int64_t ld, C;
    const float *h;             // [parts][rows][R]
    int parts;
    int64_t part_stride;
    float *partial;
    int drop;                   // src takes the dropout's mask
};

// Grid: (chunks, column blocks of both sides).  A wave owns 128 columns: a
// lane reads 8 columns of its 8 rows and turns them in registers into the
// operands of eight MFMA row blocks (row q of block t is column 8 q + t).
template <int RP, int PARTS, bool DROP>
__global__ __launch_bounds__(THREADS) void adapter_wgrad_kernel(PlanView plan, WgradSide left,
                                                               WgradSide right, int left_blocks,
                                                               int R, int chunk,
                                                               DropoutArgs drop) {
    if (!plan.built()) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const bool first = (int)blockIdx.y < left_blocks;
    const WgradSide side = first ? left : right;
    const int block = first ? blockIdx.y : blockIdx.y - left_blocks;
    const int64_t cw = (int64_t)block * kAdapterCols + wave * (kAdapterCols / WAVES);
    const int64_t C = side.C;
    if (cw >= C) return;
    const int live = plan.header[4];
    int tile = blockIdx.x * chunk;
    const int tile_end = min(tile + chunk, live);
    const int64_t c = cw + 8 * col;
    const bool c_ok = c < C;

    while (tile < tile_end) {
        const int a = plan.tile_adapter[tile];
        const int stop = min(tile_end, plan.group_tile0[a + 1]);
        f32x4 acc[8][RP / 16];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int jb = 0; jb < RP / 16; ++jb) acc[t][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (; tile < stop; ++tile) {
            int rows[8];
            u32x4 in[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) rows[i] = plan.tile_row[tile * TILE + 8 * g + i];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                in[i] = u32x4{0u, 0u, 0u, 0u};
                if (c_ok && rows[i] >= 0)
                    in[i] = *reinterpret_cast<const u32x4 *>(side.src + rows[i] * side.ld + c);
            }
            if constexpr (DROP) {
                if (side.drop) {
                    const DropoutKey key(drop.rng);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        in[i] = keep_chunk(in[i], key,
                                           (uint64_t)((int64_t)rows[i] * (C >> 3) + (c >> 3)),
                                           drop.threshold);
                }
            }
            u32x4 hs[RP / 16][PARTS];
#pragma unroll
            for (int jb = 0; jb < RP / 16; ++jb) {
                const int j = jb * 16 + col;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = 0.0f;
                    if (rows[i] >= 0 && j < R) {
                        const float *p = side.h + (int64_t)rows[i] * R + j;
                        for (int s = 0; s < side.parts; ++s) v[i] += p[s * side.part_stride];
                    }
                }
                split8<PARTS>(v, hs[jb]);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u32x4 xs;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    xs[d] = (t & 1) ? high_halves(in[2 * d][t >> 1], in[2 * d + 1][t >> 1])
                                    : low_halves(in[2 * d][t >> 1], in[2 * d + 1][t >> 1]);
#pragma unroll
                for (int jb = 0; jb < RP / 16; ++jb)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) acc[t][jb] = mfma(xs, hs[jb][p], acc[t][jb]);
            }
        }
        float *out = side.partial + (int64_t)(blockIdx.x + plan.group_rank[a]) * R * C;
#pragma unroll
        for (int jb = 0; jb < RP / 16; ++jb) {
            const int j = jb * 16 + col;
            if (j >= R) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t n = cw + 8 * (4 * g + i);
                if (n >= C) continue;
                float *p = out + (int64_t)j * C + n;
                *reinterpret_cast<f32x4 *>(p) =
                    f32x4{acc[0][jb][i], acc[1][jb][i], acc[2][jb][i], acc[3][jb][i]};
                *reinterpret_cast<f32x4 *>(p + 4) =
                    f32x4{acc[4][jb][i], acc[5][jb][i], acc[6][jb][i], acc[7][jb][i]};
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
        for (int s = 0; s < slots; ++s, p += R * in) {
            const f32x4 q = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += q[i];
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
        for (int s = 0; s < slots; ++s, p += R * outs)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += p[i * outs];
        store4<OUT>(db, ((int64_t)a * outs + n) * R + q * 4, v);
    }
}

__global__ __launch_bounds__(THREADS) void adapter_clear_kernel(u32x4 *__restrict__ p,
                                                               int64_t pieces) {
    const int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (i < pieces) p[i] = u32x4{0u, 0u, 0u, 0u};
}

// ---- launches -----------------------------------------------------------------

template <typename F>
hipError_t by_rank(int rank, F f) {
    if (rank <= 16) f(std::integral_constant<int, 16>{});
    else if (rank <= 32) f(std::integral_constant<int, 32>{});
    else if (rank <= 64) f(std::integral_constant<int, 64>{});
    else f(std::integral_constant<int, 128>{});
    return hipGetLastError();
}

int64_t part_columns(int64_t C, int parts) { return ((C + parts - 1) / parts + 31) / 32 * 32; }

template <bool TRANS>
hipError_t launch_shrink(const AdapterArgs &w, const AdapterPlanShape &shape, const int32_t *plan,
                         const DropoutArgs &drop, const uint16_t *src, int64_t ld, int64_t C,
                         float *sums, int parts, hipStream_t stream) {
    const PlanView v = view_of(shape, plan);
    const dim3 grid((unsigned)shape.tiles_max, (unsigned)parts);
    return by_rank(w.rank, [&](auto rp) {
        auto go = [&](auto dropped) {
            hipLaunchKernelGGL((adapter_shrink_kernel<decltype(rp)::value, TRANS,
                                                      decltype(dropped)::value>),
                               grid, dim3(THREADS), 0, stream, v, src, ld, C, TRANS ? w.b : w.a,
                               w.alpha, w.rank, sums, shape.rows * w.rank, part_columns(C, parts),
                               drop);
        };
        if constexpr (!TRANS) {
            if (drop.rng) return go(std::true_type{});
        }
        go(std::false_type{});
    });
}

template <bool TRANS>
hipError_t launch_expand(const AdapterArgs &w, const AdapterPlanShape &shape, const int32_t *plan,
                         const DropoutArgs &drop, const float *h, int parts, int64_t C,
                         const uint16_t *base, int64_t ldbase, uint16_t *out, int64_t ldo,
                         float *h_out, hipStream_t stream) {
    const PlanView v = view_of(shape, plan);
    const dim3 grid((unsigned)shape.tiles_max, (unsigned)((C + kAdapterCols - 1) / kAdapterCols));
    return by_rank(w.rank, [&](auto rp) {
        auto go = [&](auto dropped) {
            hipLaunchKernelGGL((adapter_expand_kernel<decltype(rp)::value, TRANS,
                                                      decltype(dropped)::value>),
                               grid, dim3(THREADS), 0, stream, v, h, parts, shape.rows * w.rank,
                               TRANS ? w.a : w.b, w.rank, C, base, ldbase, out, ldo, h_out, drop);
        };
        if constexpr (TRANS) {
            if (drop.rng) return go(std::true_type{});
        }
        go(std::false_type{});
    });
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
    const int parts = adapter_parts(shape.tiles_max, w.in);
    float *sums = parts == 1 && h ? h : static_cast<float *>(ws);
    if (hipError_t e = launch_shrink<false>(w, shape, plan, drop, x, ldx, w.in, sums, parts, stream))
        return e;
    const DropoutArgs none = {nullptr, 0, 1.0f};
    return launch_expand<false>(w, shape, plan, none, sums, parts, w.out, base, ldbase, y, ldy, h,
                                stream);
}

hipError_t launch_adapter_backward(const AdapterArgs &w, const AdapterPlanShape &shape,
                                   const int32_t *plan, const DropoutArgs &drop,
                                   const uint16_t *x, int64_t ldx, const uint16_t *dy,
                                   int64_t lddy, const float *h, const uint16_t *base,
                                   int64_t ldbase, uint16_t *dx, int64_t lddx, void *da, void *db,
                                   int out_dtype, void *ws, hipStream_t stream) {
    const AdapterWorkspace layout(shape, w.rank, w.in, w.out);
    const int parts = adapter_parts(shape.tiles_max, w.out);
    float *g = static_cast<float *>(ws);
    const DropoutArgs none = {nullptr, 0, 1.0f};
    if (hipError_t e = launch_shrink<true>(w, shape, plan, none, dy, lddy, w.out, g, parts, stream))
        return e;
    if (dx) {
        if (hipError_t e = launch_expand<true>(w, shape, plan, drop, g, parts, w.in, base, ldbase,
                                               dx, lddx, nullptr, stream))
            return e;
    }
    if (!da) return hipSuccess;
    const PlanView v = view_of(shape, plan);
    const int64_t chunk = adapter_chunk(shape.tiles_max, w.rank, w.in, w.out);
    const int64_t chunks = (shape.tiles_max + chunk - 1) / chunk;
    const int64_t slots = adapter_slots(shape, chunk);
    float *part_a = reinterpret_cast<float *>(static_cast<char *>(ws) + layout.sums);
    float *part_b = part_a + slots * w.rank * w.in;
    const WgradSide left = {x, ldx, w.in, g, parts, shape.rows * w.rank, part_a, 1};
    const WgradSide right = {dy, lddy, w.out, h, 1, 0, part_b, 0};
    const int left_blocks = (int)((w.in + kAdapterCols - 1) / kAdapterCols);
    const int right_blocks = (int)((w.out + kAdapterCols - 1) / kAdapterCols);
    const dim3 grid((unsigned)chunks, (unsigned)(left_blocks + right_blocks));
    hipError_t e = by_rank(w.rank, [&](auto rp) {
        auto go = [&](auto split, auto dropped) {
            hipLaunchKernelGGL((adapter_wgrad_kernel<decltype(rp)::value, decltype(split)::value,
                                                     decltype(dropped)::value>),
                               grid, dim3(THREADS), 0, stream, v, left, right, left_blocks, w.rank,
                               (int)chunk, drop);
        };
        using Two = std::integral_constant<int, 2>;
        using Three = std::integral_constant<int, 3>;
        auto by_drop = [&](auto split) {
            if (drop.rng) go(split, std::true_type{});
            else go(split, std::false_type{});
        };
        if (out_dtype == FP8_DTYPE_FP32) by_drop(Three{});
        else by_drop(Two{});
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
