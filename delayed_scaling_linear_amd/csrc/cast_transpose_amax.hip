// Fused scaled cast + cached transpose + amax: one HBM pass over a bf16/fp32
// tensor.
//
// What is computed follows the FP8 casts of "Accelerating PyTorch Training
// Workloads with FP8 -- Part 2" (round to nearest even onto the
// float8_e4m3fn / float8_e5m2 grids of its finfo table, here with
// saturation), the Float8Tensor of "[PyTorch] Refactor FP8 workspaces in
// linear modules" (codes, a transpose cache and a private scale-inverse
// snapshot), and the per-tensor amax of "support delayed scaling of weight in
// float8 all-gather" (taken on the unscaled source, in the same read as the
// cast, which is why delayed scaling needs fewer memory reads than dynamic
// scaling).
//
// Work decomposition (gfx950, wave64):
//   * 128 x 128 tiles, 256 threads per tile; persistent workgroups (up to
//     three per CU for bf16, two for fp32) walk the tiles with the next
//     tile's loads in flight while the current one is encoded and stored;
//   * lane l of wave w owns rows 4*rg .. 4*rg+3 (rg = 8w + l/8) of the tile.
//     A bf16 lane (cc = l%8) loads the 8-column chunks cc and 8+cc of each
//     row (16-byte loads: the eight lanes of a row cover one whole 128-byte
//     line per instruction), encodes them, and swaps half of its codes with
//     its neighbour lane (l^1) so that it then holds the 16 columns
//     16*cq .. 16*cq+15, cq = 4*(cc%2) + cc/2.  An fp32 lane loads the
//     4-column chunks cc, 8+cc, 16+cc and 24+cc (again whole lines per
//     instruction) and trades its codes through a per-wave row staging in
//     LDS for the 16 columns 16*cc .. 16*cc+15 (cq = cc);
//   * each lane scales, clamps to +-fp8_max and converts with the hardware
//     OCP FP8 converter (v_cvt_pk_fp8_f32 / v_cvt_pk_bf8_f32, round to
//     nearest even), writes its four 16-byte row-major code rows directly,
//     transposes its 4x16 byte block in registers (v_perm_b32) into sixteen
//     4-row column words and stores them to LDS;
//   * the tile is read back from LDS as 16-row column segments (ds_read_b128)
//     and written as 128-byte transposed row segments;
//   * amax: packed 16-bit max over sign-cleared bf16 patterns (or 32-bit max
//     for fp32), wave reduction, LDS across waves, one atomicMax per
//     workgroup into the fp32 amax (order-preserving on non-negative floats).
//
// LDS layout of the transposed tile: 128 columns x 32 words (4 rows / word),
// word index of (column c, row group g) = c*32 + (g ^ 4*(c/16)): the XOR keeps
// the sixteen-lane groups that write one column word apiece in distinct banks
// and leaves each 16-byte, 16-row read contiguous and in order.
#include <algorithm>
#include <type_traits>

#include "bf16.h"
#include "dropout.h"
#include "expert.h"
#include "fp8_codec.h"
#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

constexpr int TILE = 128;
constexpr int THREADS = 256;

typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A lane's sixteen source elements of one tile row, as loaded: kChunks
// 16-byte chunks, chunk k at tile column (128 / kChunks) * k + (16 / kChunks)
// * cc for lane chunk cc (src_offsets), so that the eight lanes of a row
// cover whole 128-byte lines with every load instruction.
template <int SRC>
struct SrcRow;

template <>
struct SrcRow<FP8_DTYPE_BF16> {
    static constexpr int kBytes = 2;
    static constexpr int kChunks = 2;        // 8 elements each, 128 bytes apart
    u32x4 v[2];
    // Chunk k at byte offset off[k] of the descriptor (an offset outside it
    // reads zeros and touches no memory); POL is the cache policy (0, or 2 =
    // non-temporal).
    template <int POL>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, const uint32_t (&off)[2]) {
        v[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off[0], 0, POL));
        v[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off[1], 0, POL));
    }
    // Elements 4j .. 4j+3 as fp32 (exact widening): j = 0, 1 from the first
    // chunk, 2, 3 from the second.
    __device__ __forceinline__ void get4(int j, float o[4]) const {
        const u32x4 &q = v[j >> 1];
        const uint32_t d0 = (j & 1) ? q.z : q.x;
        const uint32_t d1 = (j & 1) ? q.w : q.y;
        o[0] = bf16_lo(d0);
        o[1] = bf16_hi(d0);
        o[2] = bf16_lo(d1);
        o[3] = bf16_hi(d1);
    }
    // Largest sign-cleared pattern, widened to the fp32 bit order.
    __device__ __forceinline__ uint32_t amax_key() const {
        ushort2_t m2 = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t d[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(ushort2_t, d[j] & 0x7FFF7FFFu));
        }
        return (uint32_t)max(m2.x, m2.y) << 16;
    }
};

template <>
struct SrcRow<FP8_DTYPE_FP32> {
    static constexpr int kBytes = 4;
    static constexpr int kChunks = 4;        // 4 elements each, 128 bytes apart
    f32x4 v[4];
    template <int POL>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, const uint32_t (&off)[4]) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            v[h] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off[h], 0, POL));
    }
    // Elements 4j .. 4j+3: chunk j.
    __device__ __forceinline__ void get4(int j, float o[4]) const {
        o[0] = v[j].x;
        o[1] = v[j].y;
        o[2] = v[j].z;
        o[3] = v[j].w;
    }
    __device__ __forceinline__ uint32_t amax_key() const {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            m = max(m, __float_as_uint(v[h].x) & 0x7FFFFFFFu);
            m = max(m, __float_as_uint(v[h].y) & 0x7FFFFFFFu);
            m = max(m, __float_as_uint(v[h].z) & 0x7FFFFFFFu);
            m = max(m, __float_as_uint(v[h].w) & 0x7FFFFFFFu);
        }
        return m;
    }
};

constexpr uint32_t SRC_OOB = 0x80000000u;

// Byte offsets (from the tile's first element) of lane chunk cc's source
// chunks in the first of its four rows, 4*rg; a chunk past the tensor's
// columns, or a row past its rows, takes SRC_OOB and reads zeros (columns
// come in groups of 16, so a chunk is wholly inside or outside).
template <int SRC>
__device__ __forceinline__ void src_offsets(bool row_ok, int64_t col0, int64_t cols, int64_t ld,
                                            int rg, int cc,
                                            uint32_t (&off)[SrcRow<SRC>::kChunks]) {
    constexpr int EB = SrcRow<SRC>::kBytes, K = SrcRow<SRC>::kChunks;
    const int64_t rb = (int64_t)(4 * rg) * ld;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int col = (128 / K) * k + (16 / K) * cc;
        off[k] = (row_ok && col0 + col < cols) ? (uint32_t)((rb + col) * EB) : SRC_OOB;
    }
}

// The 16-column chunk whose codes lane chunk cc stores (after the exchange
// in encode_block: bf16 with the neighbour lane, fp32 through LDS).
template <int SRC>
__device__ __forceinline__ int store_chunk(int cc) {
    return SrcRow<SRC>::kChunks == 2 ? 4 * (cc & 1) + (cc >> 1) : cc;
}

// Column (0..127 in the tile) of element k (0..15) of lane chunk cc's source.
template <int SRC>
__device__ __forceinline__ int src_col(int cc, int k) {
    constexpr int K = SrcRow<SRC>::kChunks, E = 16 / K;
    return (128 / K) * (k / E) + E * cc + (k % E);
}

// Words of the per-wave row staging that the fp32 exchange uses: 32 rows of
// 128 code bytes.
constexpr int ROW_STAGE_WORDS = 32 * 32;

// Lane l's value of v on lane l ^ 1 (DPP quad permutation 1, 0, 3, 2).
__device__ __forceinline__ uint32_t from_neighbour(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}

// 4x4 byte transpose: in[r] holds bytes (r, c=0..3); out[c] holds (r=0..3, c).
__device__ __forceinline__ void transpose4x4(const uint32_t in[4], uint32_t out[4]) {
    const uint32_t lo01 = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);
    const uint32_t hi01 = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
    const uint32_t lo23 = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
    const uint32_t hi23 = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
    out[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
    return v;
}

// Encode this lane's 4 x 16 block of the tile held in `src`, store the
// row-major codes of chunk cq (columns c .. c+15, c = col0 + 16*cq) and its
// transposed 4-row words into the LDS tile `lt`.  bf16: the lane encodes its
// two 8-column source chunks, then keeps the codes of the first (even lane)
// or second (odd lane) and takes the neighbour's codes of the same chunk
// parity, which together are chunk cq = store_chunk(cc).  fp32: the lane's
// four 4-column chunks go through the wave's row staging `ls`
// (ROW_STAGE_WORDS words) and come back as the 16 columns of chunk cq = cc.
// Every lane of the wave must call it (the exchanges read other lanes' data).
template <int SRC, int FMT, bool WANT_Q, bool WANT_QT>
__device__ __forceinline__ void encode_block(const SrcRow<SRC> (&src)[4], float s, bool s_special,
                                             bool valid, uint8_t *__restrict__ q, int64_t r,
                                             int64_t c, int64_t cols, int cq, int rg, int lane,
                                             uint32_t *ls, uint32_t *lt, uint32_t &key) {
    uint32_t codes[4][4];                    // [row][word of 4 columns]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row_key = src[i].amax_key();
        key = max(key, row_key);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x4[4];
            src[i].get4(j, x4);
            codes[i][j] = encode4<FMT>(x4[0], x4[1], x4[2], x4[3], s);
        }
        if (s_special || row_key > 0x7F800000u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x4[4];
                src[i].get4(j, x4);
                codes[i][j] = patch_nan4(codes[i][j], x4, s);
            }
        }
    }
    if constexpr (SrcRow<SRC>::kChunks == 4) {
        // Word group g (columns 4g .. 4g+3) of staging row qr at 16-byte
        // chunk (g / 4) ^ (qr / 4), word g % 4 (at most two lanes per bank on
        // the writes).  A wave's LDS operations complete in issue order, so
        // the reads see every lane's writes; the fences keep the compiler
        // from moving them across.
        const int cc = lane & 7, rl = lane >> 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int qr = 4 * rl + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int g = 8 * j + cc;
                ls[qr * 32 + (((g >> 2) ^ rl) << 2) + (g & 3)] = codes[i][j];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 w =
                *reinterpret_cast<const u32x4 *>(&ls[(4 * rl + i) * 32 + ((cq ^ rl) << 2)]);
            codes[i][0] = w.x;
            codes[i][1] = w.y;
            codes[i][2] = w.z;
            codes[i][3] = w.w;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    } else {
        // Even lane: columns 8cc..+7 | neighbour's 8cc+8..+15.  Odd lane:
        // neighbour's 64+8cc-8..+7 | its own 64+8cc..+7.
        const bool odd = lane & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r0 = from_neighbour(odd ? codes[i][0] : codes[i][2]);
            const uint32_t r1 = from_neighbour(odd ? codes[i][1] : codes[i][3]);
            if (odd) {
                codes[i][0] = r0;
                codes[i][1] = r1;
            } else {
                codes[i][2] = r0;
                codes[i][3] = r1;
            }
        }
    }
    if constexpr (WANT_Q) {
        if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4 *dst = reinterpret_cast<u32x4 *>(q + (r + i) * cols + c);
                *dst = u32x4{codes[i][0], codes[i][1], codes[i][2], codes[i][3]};
            }
        }
    }
    if constexpr (WANT_QT) {
        const int swz = 4 * cq;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t in[4] = {codes[0][j], codes[1][j], codes[2][j], codes[3][j]};
            uint32_t out[4];
            transpose4x4(in, out);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int tc = 16 * cq + 4 * j + b;          // tile column
                lt[tc * 32 + (rg ^ swz)] = out[b];
            }
        }
    }
}

// Transposed store of one tile from its LDS transpose `lt`: 8 lanes per
// tile column (16 rows each), 128-byte transposed row segments.
__device__ __forceinline__ void store_transposed(const uint32_t *lt, uint8_t *__restrict__ qt,
                                                 int64_t rows, int64_t cols, int64_t row0,
                                                 int64_t col0, int lane, int wave) {
    const int qd = lane & 7;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int tc = (lane >> 3) + 8 * (wave + 4 * k);
        const int64_t gc = col0 + tc;
        const int64_t gr = row0 + 16 * qd;
        if (gc < cols && gr < rows) {
            const int word = tc * 32 + ((4 * qd) ^ (4 * (tc >> 4)));
            const u32x4 v = *reinterpret_cast<const u32x4 *>(&lt[word]);
            *reinterpret_cast<u32x4 *>(qt + gc * rows + gr) = v;
        }
    }
}

// Fold this workgroup's sign-cleared maximum `key` into *amax_cur: wave
// reduction, LDS across waves, one atomicMax (skipped when the stored value
// already covers it: amax_cur only grows while casts run).
__device__ __forceinline__ void flush_amax(uint32_t key, float *amax_cur, uint32_t *lds_amax,
                                           int lane, int wave, int tid) {
    key = wave_max_u32(key);
    if (lane == 0) lds_amax[wave] = key;
    __syncthreads();
    if (tid == 0) {
        uint32_t k = lds_amax[0];
#pragma unroll
        for (int w = 1; w < THREADS / 64; ++w) k = max(k, lds_amax[w]);
        unsigned int *a = reinterpret_cast<unsigned int *>(amax_cur);
        if (k > __atomic_load_n(a, __ATOMIC_RELAXED)) atomicMax(a, k);
    }
}

// Persistent: workgroup b casts tiles b, b + gridDim.x, ... with the loads of
// its next tile in flight while the current one is encoded and stored, and
// a double-buffered LDS transpose tile (one barrier per tile).
// SRC: FP8_DTYPE_BF16 or FP8_DTYPE_FP32.  The source is read with
// non-temporal loads (unless `cached`): it is read once, and allocating it in
// the last-level cache would push out the codes just written, which the
// matrix products read next.  Measured on MI355X, one linear's forward +
// backward step is 6-9% faster than with normal loads, and the cast alone on
// cold buffers runs at the same speed (within 2%) either way.  Large
// tensors (more than two tiles per resident workgroup) are launched with one
// workgroup per tile, so that the hardware dispatcher balances the last
// round.
// Resident workgroups per CU: the double-buffered source needs 64 (bf16) or
// 128 (fp32) registers per lane.
// The bias-gradient variant needs its 16 column sums on top: two per CU.
template <int SRC>
constexpr int kWavesPerSimd = SRC == FP8_DTYPE_BF16 ? 3 : 2;

// The bias gradient's per-tile column sums of the unscaled source (fp32),
// taken by the one-tile cast: each lane adds its four rows in order, the
// eight row groups of a wave meet in a butterfly of lane exchanges, the four
// waves in LDS in wave order; tile (tr, tc) writes its 128 sums to
// dbias_ws[tr * ws_ld + 128 tc ..].  Every step has a fixed order, so the
// result is the same on every run.
//   tile_col_sums_to_lds: a wave's sums of its 32 rows into d[0 .. 127]
//   (written by the lanes of row group 0); rows past the tensor were loaded
//   as zeros and add nothing.
template <int SRC>
__device__ __forceinline__ void tile_col_sums_to_lds(const SrcRow<SRC> (&src)[4], float *d,
                                                     int lane, int cc) {
    float cs[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float o[4];
        src[0].get4(j, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) cs[4 * j + k] = o[k];
    }
#pragma unroll
    for (int i = 1; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float o[4];
            src[i].get4(j, o);
#pragma unroll
            for (int k = 0; k < 4; ++k) cs[4 * j + k] += o[k];
        }
#pragma unroll
    for (int m = 8; m < 64; m *= 2)
#pragma unroll
        for (int k = 0; k < 16; ++k) cs[k] += __shfl_xor(cs[k], m);
    if ((lane >> 3) == 0) {
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<f32x4 *>(d + src_col<SRC>(cc, k)) =
                f32x4{cs[k], cs[k + 1], cs[k + 2], cs[k + 3]};
    }
}

//   tile_col_sums_out: after a barrier, the four waves' sums (d = the
//   first wave's 128, the others at strides of 128) added in wave order
//   into the tile's workspace row.
__device__ __forceinline__ void tile_col_sums_out(const float *d, int tid, float *dbias_ws,
                                                  int64_t ws_ld, int64_t tr, int64_t tcn) {
    if (tid < TILE) {
        const float sum = ((d[tid] + d[TILE + tid]) + d[2 * TILE + tid]) + d[3 * TILE + tid];
        dbias_ws[tr * ws_ld + tcn * TILE + tid] = sum;
    }
}

template <int SRC, int FMT, bool WANT_Q, bool WANT_QT>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(kWavesPerSimd<SRC>))) void
cast_transpose_amax_kernel(
    const void *__restrict__ xv, int64_t rows, int64_t cols, int64_t ld,
    const float *__restrict__ scale_ptr, uint8_t *__restrict__ q, uint8_t *__restrict__ qt,
    float *__restrict__ amax_cur, float *__restrict__ scale_inv_out,
    const int32_t *__restrict__ noop, int64_t tiles_c, int64_t ntiles, int cached) {
    if (noop != nullptr && *noop != 0) return;

    __shared__ uint32_t lds_t[2][TILE * (TILE / 4)];   // transposed tiles, 2 x 16 KiB
    __shared__ uint32_t lds_amax[THREADS / 64];
    constexpr int K = SrcRow<SRC>::kChunks;
    __shared__ uint32_t lds_rows[K == 4 ? (THREADS / 64) * ROW_STAGE_WORDS : 1];   // fp32 exchange

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int cc = lane & 7;                 // source chunk (src_offsets)
    const int cq = store_chunk<SRC>(cc);     // 16-column chunk of the codes
    const int rg = wave * 8 + (lane >> 3);   // 4-row group of the tile
    constexpr int EB = SrcRow<SRC>::kBytes;
    const int64_t total_bytes = ((rows - 1) * ld + cols) * EB;

    const float s = *scale_ptr;
    // NaN products from a non-NaN source only arise when s is 0, inf or NaN.
    const bool s_special = !(fabsf(s) > 0.0f && fabsf(s) <= 3.402823466e38f);
    if (blockIdx.x == 0 && tid == 0 && scale_inv_out != nullptr) *scale_inv_out = 1.0f / s;

    // Source descriptor of tile t (empty when t is past the last tile) and
    // this lane's byte offsets in it.
    auto tile_rsrc = [&](int64_t t, __amdgpu_buffer_rsrc_t &rs, uint32_t (&off)[K], int64_t &r,
                         int64_t &c, bool &valid) {
        const int64_t tr = t / tiles_c, tcn = t - (t / tiles_c) * tiles_c;
        const int64_t row0 = tr * TILE, col0 = tcn * TILE;
        r = row0 + 4 * rg;
        c = col0 + 16 * cq;
        valid = (t < ntiles) && (r < rows) && (c < cols);
        const int64_t base = (t < ntiles) ? (row0 * ld + col0) * EB : 0;
        const int64_t avail = (t < ntiles) ? total_bytes - base : 0;
        const int32_t nrec = (int32_t)min(avail, (int64_t)0x7FFFFFFF);
        rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(static_cast<const uint8_t *>(xv)) + base, (short)0, nrec,
            0x00020000);
        src_offsets<SRC>((t < ntiles) && (r < rows), col0, cols, ld, rg, cc, off);
    };
    const uint32_t row_step = (uint32_t)(ld * EB);
    // `cached` (wave-uniform) reads the source through the caches instead.
    auto load_tile = [&](SrcRow<SRC> (&dst)[4], __amdgpu_buffer_rsrc_t rs, const uint32_t (&off)[K]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[K];
#pragma unroll
            for (int k = 0; k < K; ++k) o[k] = off[k] == SRC_OOB ? SRC_OOB : off[k] + i * row_step;
            if (cached)
                dst[i].template load<0>(rs, o);
            else
                dst[i].template load<2>(rs, o);
        }
    };
    auto store_t = [&](const uint32_t *lt, int64_t t) {
        const int64_t tr = t / tiles_c, tcn = t - tr * tiles_c;
        store_transposed(lt, qt, rows, cols, tr * TILE, tcn * TILE, lane, wave);
    };

    uint32_t key = 0;                        // sign-cleared max, fp32 bit order
    SrcRow<SRC> src[2][4];
    __amdgpu_buffer_rsrc_t rs_cur, rs_nxt;
    uint32_t off_cur[K], off_nxt[K];
    int64_t r_cur, c_cur, r_nxt, c_nxt;
    bool v_cur, v_nxt;
    int64_t t = blockIdx.x;
    tile_rsrc(t, rs_cur, off_cur, r_cur, c_cur, v_cur);
    load_tile(src[0], rs_cur, off_cur);

    for (; t < ntiles;) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (t < ntiles) {
                const int64_t tn = t + gridDim.x;
                tile_rsrc(tn, rs_nxt, off_nxt, r_nxt, c_nxt, v_nxt);
                load_tile(src[u ^ 1], rs_nxt, off_nxt);           // empty past the end
                encode_block<SRC, FMT, WANT_Q, WANT_QT>(src[u], s, s_special, v_cur, q, r_cur,
                                                        c_cur, cols, cq, rg, lane,
                                                        lds_rows + (K == 4 ? wave * ROW_STAGE_WORDS : 0),
                                                        lds_t[u], key);
                __syncthreads();
                if constexpr (WANT_QT) store_t(lds_t[u], t);
                t = tn;
                r_cur = r_nxt;
                c_cur = c_nxt;
                v_cur = v_nxt;
            }
        }
    }

    if (amax_cur != nullptr) flush_amax(key, amax_cur, lds_amax, lane, wave, tid);
}

// One tile per workgroup, no loop: every lane issues its tile's source loads
// at once, then encodes and stores them.  With no second tile's source in
// registers a workgroup needs half the registers of the persistent kernel,
// so four or more fit on a CU and all tiles of a [4096, 4096] tensor have
// their loads in flight together (a copy of the same bytes needs about that
// many bytes in flight to reach its best rate); the hardware dispatcher
// balances larger tensors.  Used for casts without the bias gradient of
// tensors with more than two tiles per resident persistent workgroup (there
// it beats the persistent kernel; below that the persistent kernel's
// overlap of one tile's loads with the previous tile's stores wins).
// Tile t (row-major over tiles_c tile columns) of one tensor; scale_inv_out,
// if not null, receives 1 / scale (the caller passes it to one workgroup).
template <int SRC, int FMT, bool WANT_Q, bool WANT_QT, bool DBIAS = false>
__device__ __forceinline__ void cast_one_tile(const void *__restrict__ xv, int64_t rows,
                                              int64_t cols, int64_t ld,
                                              const float *__restrict__ scale_ptr,
                                              uint8_t *__restrict__ q, uint8_t *__restrict__ qt,
                                              float *__restrict__ amax_cur,
                                              float *__restrict__ scale_inv_out, int64_t t,
                                              int64_t tiles_c, int cached,
                                              float *__restrict__ dbias_ws = nullptr,
                                              int64_t ws_ld = 0) {
    __shared__ uint32_t lds_t[TILE * (TILE / 4)];      // the transposed tile, 16 KiB
    __shared__ uint32_t lds_amax[THREADS / 64];
    __shared__ float lds_db[DBIAS ? (THREADS / 64) * TILE : 1];   // [wave][column]
    constexpr int K = SrcRow<SRC>::kChunks;
    __shared__ uint32_t lds_rows[K == 4 ? (THREADS / 64) * ROW_STAGE_WORDS : 1];   // fp32 exchange

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int cc = lane & 7;
    const int cq = store_chunk<SRC>(cc);
    const int rg = wave * 8 + (lane >> 3);
    constexpr int EB = SrcRow<SRC>::kBytes;

    const float s = *scale_ptr;
    const bool s_special = !(fabsf(s) > 0.0f && fabsf(s) <= 3.402823466e38f);
    if (tid == 0 && scale_inv_out != nullptr) *scale_inv_out = 1.0f / s;

    const int64_t tr = t / tiles_c, tcn = t - tr * tiles_c;
    const int64_t row0 = tr * TILE, col0 = tcn * TILE;
    const int64_t r = row0 + 4 * rg, c = col0 + 16 * cq;
    const bool valid = (r < rows) && (c < cols);   // rows, cols are multiples of 16
    // The tile's descriptor ends at the tensor's last byte: rows past the
    // end read as zeros.
    const int64_t base = (row0 * ld + col0) * EB;
    const int64_t avail = ((rows - 1) * ld + cols) * EB - base;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(static_cast<const uint8_t *>(xv)) + base, (short)0,
        (int32_t)min(avail, (int64_t)0x7FFFFFFF), 0x00020000);
    uint32_t off[K];
    src_offsets<SRC>(r < rows, col0, cols, ld, rg, cc, off);
    const uint32_t row_step = (uint32_t)(ld * EB);
    SrcRow<SRC> src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t o[K];
#pragma unroll
        for (int k = 0; k < K; ++k) o[k] = off[k] == SRC_OOB ? SRC_OOB : off[k] + i * row_step;
        if (cached)
            src[i].template load<0>(rs, o);
        else
            src[i].template load<2>(rs, o);
    }
    uint32_t key = 0;
    encode_block<SRC, FMT, WANT_Q, WANT_QT>(src, s, s_special, valid, q, r, c, cols, cq, rg, lane,
                                            lds_rows + (K == 4 ? wave * ROW_STAGE_WORDS : 0),
                                            lds_t, key);
    if constexpr (DBIAS) tile_col_sums_to_lds<SRC>(src, &lds_db[wave * TILE], lane, cc);
    __syncthreads();
    if constexpr (WANT_QT) store_transposed(lds_t, qt, rows, cols, row0, col0, lane, wave);
    if constexpr (DBIAS) tile_col_sums_out(lds_db, tid, dbias_ws, ws_ld, tr, tcn);
    if (amax_cur != nullptr) flush_amax(key, amax_cur, lds_amax, lane, wave, tid);
}

template <int SRC, int FMT, bool WANT_Q, bool WANT_QT, bool DBIAS>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(4))) void
cast_tile_kernel(const void *__restrict__ xv, int64_t rows, int64_t cols, int64_t ld,
                 const float *__restrict__ scale_ptr, uint8_t *__restrict__ q,
                 uint8_t *__restrict__ qt, float *__restrict__ amax_cur,
                 float *__restrict__ scale_inv_out, const int32_t *__restrict__ noop,
                 int64_t tiles_c, int cached, float *__restrict__ dbias_ws, int64_t ws_ld) {
    if (noop != nullptr && *noop != 0) return;
    cast_one_tile<SRC, FMT, WANT_Q, WANT_QT, DBIAS>(xv, rows, cols, ld, scale_ptr, q, qt, amax_cur,
                                                    blockIdx.x == 0 ? scale_inv_out : nullptr,
                                                    (int64_t)blockIdx.x, tiles_c, cached,
                                                    dbias_ws, ws_ld);
}

// Several tensors in one launch, one workgroup per 128 x 128 tile of their
// concatenated tile lists: workgroup b casts tile b - first[i] of tensor i,
// first[i] <= b < first[i + 1], exactly as cast_tile_kernel casts it (the
// same codes, transpose, amax and scale-inverse as one launch per tensor).
// The tensors' parameters are kernel arguments (by value), so the launch
// reads no host memory at run time and can be captured in a HIP graph.
template <int SRC, int FMT, bool WANT_Q, bool WANT_QT>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(4))) void
cast_tile_group_kernel(const CastGroupArgs args, const int32_t *__restrict__ noop, int cached) {
    if (noop != nullptr && *noop != 0) return;
    const int64_t b = blockIdx.x;
    int i = 0;
#pragma unroll
    for (int k = 1; k < kCastGroupMax; ++k)
        if (k < args.n && b >= args.first[k]) i = k;
    const CastGroupItem &it = args.item[i];
    const int64_t t = b - args.first[i];
    cast_one_tile<SRC, FMT, WANT_Q, WANT_QT>(it.x, it.rows, it.cols, it.ld, it.scale, it.q,
                                             it.qt, it.amax_cur,
                                             t == 0 ? it.scale_inv : nullptr, t, it.tiles_c,
                                             cached);
}

template <int SRC, int FMT>
hipError_t launch_src_fmt(const void *x, int64_t rows, int64_t cols, int64_t ld,
                          const float *scale, uint8_t *q, uint8_t *qt, float *amax_cur,
                          float *scale_inv_out, const int32_t *noop, float *dbias_ws,
                          int64_t ws_ld, bool cached, hipStream_t stream) {
    int cus = 0;
    if (hipError_t e = current_cu_count(&cus)) return e;
    const int64_t tiles_r = (rows + TILE - 1) / TILE;
    const int64_t tiles_c = (cols + TILE - 1) / TILE;
    const int64_t ntiles = tiles_r * tiles_c;
    // As many workgroups as fit on the chip at once, each looping over tiles
    // with the next tile's loads in flight; tensors with more than two tiles
    // per resident workgroup, and every cast that also sums the bias
    // gradient: one workgroup per tile (cast_tile_kernel).
    const int64_t resident = (int64_t)cus * kWavesPerSimd<SRC>;
    const bool per_tile = ntiles > 2 * resident || dbias_ws != nullptr;
    if (per_tile) {
        auto launch1 = [&](auto wq, auto wqt, auto db) {
            hipLaunchKernelGGL((cast_tile_kernel<SRC, FMT, decltype(wq)::value,
                                                 decltype(wqt)::value, decltype(db)::value>),
                               dim3((unsigned)ntiles), dim3(THREADS), 0, stream, x, rows, cols,
                               ld, scale, q, qt, amax_cur, scale_inv_out, noop, tiles_c,
                               (int)cached, dbias_ws, ws_ld);
        };
        using T1 = std::true_type;
        using F1 = std::false_type;
        auto by_layout1 = [&](auto db) {
            if (q && qt) launch1(T1{}, T1{}, db);
            else if (q) launch1(T1{}, F1{}, db);
            else launch1(F1{}, T1{}, db);
        };
        if (dbias_ws) by_layout1(T1{});
        else by_layout1(F1{});
        return hipGetLastError();
    }
    const dim3 grid((unsigned)std::min<int64_t>(ntiles, resident));
    auto launch = [&](auto wq, auto wqt) {
        hipLaunchKernelGGL((cast_transpose_amax_kernel<SRC, FMT, decltype(wq)::value,
                                                       decltype(wqt)::value>),
                           grid, dim3(THREADS), 0, stream, x, rows, cols, ld, scale, q, qt,
                           amax_cur, scale_inv_out, noop, tiles_c, ntiles, (int)cached);
    };
    using T_ = std::true_type;
    using F_ = std::false_type;
    if (q && qt) launch(T_{}, T_{});
    else if (q) launch(T_{}, F_{});
    else launch(F_{}, T_{});
    return hipGetLastError();
}

// An empty source still takes the scale-inverse snapshot.
__global__ void scale_inv_only_kernel(const float *__restrict__ scale_ptr,
                                      float *__restrict__ scale_inv_out,
                                      const int32_t *__restrict__ noop) {
    if (noop != nullptr && *noop != 0) return;
    *scale_inv_out = 1.0f / *scale_ptr;
}

}  // namespace

hipError_t launch_scale_inv_only(const float *scale, float *scale_inv_out, const int32_t *noop,
                                 hipStream_t stream) {
    hipLaunchKernelGGL(scale_inv_only_kernel, dim3(1), dim3(1), 0, stream, scale, scale_inv_out,
                       noop);
    return hipGetLastError();
}

hipError_t launch_cast_transpose_amax(const void *x, int src, int64_t rows, int64_t cols,
                                      int64_t ld, const float *scale, int fmt, uint8_t *q,
                                      uint8_t *qt, float *amax_cur, float *scale_inv_out,
                                      const int32_t *noop, float *dbias_ws, int64_t ws_ld,
                                      hipStream_t stream, bool cached) {
    if (src == FP8_DTYPE_BF16) {
        if (fmt == FP8_E4M3)
            return launch_src_fmt<FP8_DTYPE_BF16, FP8_E4M3>(x, rows, cols, ld, scale, q, qt,
                                                            amax_cur, scale_inv_out, noop,
                                                            dbias_ws, ws_ld, cached, stream);
        return launch_src_fmt<FP8_DTYPE_BF16, FP8_E5M2>(x, rows, cols, ld, scale, q, qt, amax_cur,
                                                        scale_inv_out, noop, dbias_ws, ws_ld,
                                                        cached, stream);
    }
    if (fmt == FP8_E4M3)
        return launch_src_fmt<FP8_DTYPE_FP32, FP8_E4M3>(x, rows, cols, ld, scale, q, qt, amax_cur,
                                                        scale_inv_out, noop, dbias_ws, ws_ld,
                                                        cached, stream);
    return launch_src_fmt<FP8_DTYPE_FP32, FP8_E5M2>(x, rows, cols, ld, scale, q, qt, amax_cur,
                                                    scale_inv_out, noop, dbias_ws, ws_ld, cached,
                                                    stream);
}

template <int SRC, int FMT>
hipError_t launch_group_src_fmt(const CastGroupArgs &args, int64_t tiles, bool want_q,
                                bool want_qt, const int32_t *noop, bool cached,
                                hipStream_t stream) {
    auto launch = [&](auto wq, auto wqt) {
        hipLaunchKernelGGL((cast_tile_group_kernel<SRC, FMT, decltype(wq)::value,
                                                   decltype(wqt)::value>),
                           dim3((unsigned)tiles), dim3(THREADS), 0, stream, args, noop,
                           (int)cached);
    };
    using T1 = std::true_type;
    using F1 = std::false_type;
    if (want_q && want_qt) launch(T1{}, T1{});
    else if (want_q) launch(T1{}, F1{});
    else launch(F1{}, T1{});
    return hipGetLastError();
}

hipError_t launch_cast_group(const CastGroupArgs &args, int src, int fmt, bool want_q,
                             bool want_qt, const int32_t *noop, bool cached,
                             hipStream_t stream) {
    const int64_t tiles = args.first[args.n];
    if (tiles == 0) return hipSuccess;
    if (src == FP8_DTYPE_BF16) {
        if (fmt == FP8_E4M3)
            return launch_group_src_fmt<FP8_DTYPE_BF16, FP8_E4M3>(args, tiles, want_q, want_qt,
                                                                  noop, cached, stream);
        return launch_group_src_fmt<FP8_DTYPE_BF16, FP8_E5M2>(args, tiles, want_q, want_qt, noop,
                                                              cached, stream);
    }
    if (fmt == FP8_E4M3)
        return launch_group_src_fmt<FP8_DTYPE_FP32, FP8_E4M3>(args, tiles, want_q, want_qt, noop,
                                                              cached, stream);
    return launch_group_src_fmt<FP8_DTYPE_FP32, FP8_E5M2>(args, tiles, want_q, want_qt, noop,
                                                          cached, stream);
}

// Producer-fused cast.  The toy block of "CPU Overhead of te.Linear FP8
// Layers" (TEBlock.forward) computes each linear's input with an elementwise
// operation in torch (the modulation: the input times one slice of the
// modulation linear's output, divided by another; the residual adds) and
// only then casts it.  Here one pass reads the operands, writes the bf16
// result y and casts y exactly as cast_transpose_amax_kernel would:
//   OP 1 (modulate): y = bf16(a * x / b) (fp32 multiply, correctly rounded
//        fp32 division, round to nearest even); infinities stay infinities,
//        a NaN quotient becomes 0x7FC0, and the cast codes both by its rules;
//   OP 2 (residual add): y = bf16(x + a); a NaN sum becomes 0x7FC0;
//   OP 3 (two residual terms): y = bf16(bf16(x + a) + b), each sum rounded;
//   OP 4 (modulate, finite: this library's addition, not on the pages): as
//        OP 1, then a y that is not finite becomes +0, so a zero divisor
//        cannot put infinities or NaNs into a model's activations.
// One workgroup per 128 x 128 tile, the lane layout of the cast (4 rows x 16
// columns, 16-byte loads and stores).
template <int OP>
__device__ __forceinline__ uint32_t produce_pair(uint32_t xw, uint32_t aw, uint32_t bw) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float xv = __uint_as_float(h ? (xw & 0xFFFF0000u) : (xw << 16));
        const float av = __uint_as_float(h ? (aw & 0xFFFF0000u) : (aw << 16));
        uint32_t y;
        if constexpr (OP == FP8_PRODUCE_MODULATE || OP == FP8_PRODUCE_MODULATE_FINITE) {
            const float bv = __uint_as_float(h ? (bw & 0xFFFF0000u) : (bw << 16));
            const float v = (av * xv) / bv;
            y = bf16_bits(v);
            if constexpr (OP == FP8_PRODUCE_MODULATE_FINITE)
                y = ((y & 0x7F80u) == 0x7F80u) ? 0u : y;
        } else if constexpr (OP == FP8_PRODUCE_ADD) {
            const float v = xv + av;
            y = bf16_bits(v);
        } else {
            // Two terms, added one at a time with a bf16 rounding after each.
            const float bv = __uint_as_float(h ? (bw & 0xFFFF0000u) : (bw << 16));
            const float v1 = xv + av;
            const uint32_t t = bf16_bits(v1);
            const float v = __uint_as_float(t << 16) + bv;
            y = bf16_bits(v);
        }
        out |= y << (16 * h);
    }
    return out;
}

template <int OP, int FMT, bool WANT_Q, bool WANT_QT>
__global__ __launch_bounds__(THREADS) void produce_cast_kernel(
    const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ a, int64_t lda,
    const uint16_t *__restrict__ b, int64_t ldb, uint16_t *__restrict__ y, int64_t rows,
    int64_t cols, const float *__restrict__ scale_ptr, uint8_t *__restrict__ q,
    uint8_t *__restrict__ qt, float *__restrict__ amax_cur, float *__restrict__ scale_inv_out,
    const int32_t *__restrict__ noop, int64_t tiles_c) {
    if (noop != nullptr && *noop != 0) return;
    __shared__ uint32_t lds_t[TILE * (TILE / 4)];
    __shared__ uint32_t lds_amax[THREADS / 64];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int cc = lane & 7;
    const int cq = store_chunk<FP8_DTYPE_BF16>(cc);
    const int rg = wave * 8 + (lane >> 3);
    const float s = *scale_ptr;
    const bool s_special = !(fabsf(s) > 0.0f && fabsf(s) <= 3.402823466e38f);
    if (blockIdx.x == 0 && tid == 0 && scale_inv_out != nullptr) *scale_inv_out = 1.0f / s;

    const int64_t t = blockIdx.x;
    const int64_t tr = t / tiles_c, tcn = t - tr * tiles_c;
    const int64_t row0 = tr * TILE, col0 = tcn * TILE;
    const int64_t r = row0 + 4 * rg, c = col0 + 16 * cq;
    const bool valid = (r < rows) && (c < cols);   // rows, cols are multiples of 16

    // The lane's two 8-column chunks (cc and 8 + cc, as in the cast), each
    // loaded, combined and stored as y only when it lies inside the tensor.
    SrcRow<FP8_DTYPE_BF16> ys[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ys[i].v[0] = u32x4{0u, 0u, 0u, 0u};
        ys[i].v[1] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t ch = col0 + 64 * h + 8 * cc;
        if (r < rows && ch < cols) {
            u32x4 xv[4], av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[i] = *reinterpret_cast<const u32x4 *>(x + (r + i) * ldx + ch);
                av[i] = *reinterpret_cast<const u32x4 *>(a + (r + i) * lda + ch);
                if constexpr (OP != FP8_PRODUCE_ADD)
                    bv[i] = *reinterpret_cast<const u32x4 *>(b + (r + i) * ldb + ch);
                else
                    bv[i] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 X = xv[i], A = av[i], B = bv[i];
                const u32x4 Y = {produce_pair<OP>(X.x, A.x, B.x), produce_pair<OP>(X.y, A.y, B.y),
                                 produce_pair<OP>(X.z, A.z, B.z), produce_pair<OP>(X.w, A.w, B.w)};
                ys[i].v[h] = Y;
                *reinterpret_cast<u32x4 *>(y + (r + i) * cols + ch) = Y;
            }
        }
    }
    uint32_t key = 0;
    encode_block<FP8_DTYPE_BF16, FMT, WANT_Q, WANT_QT>(ys, s, s_special, valid, q, r, c, cols, cq,
                                                       rg, lane, nullptr, lds_t, key);
    __syncthreads();
    if constexpr (WANT_QT) store_transposed(lds_t, qt, rows, cols, row0, col0, lane, wave);
    if (amax_cur != nullptr) flush_amax(key, amax_cur, lds_amax, lane, wave, tid);
}

template <int OP, int FMT>
hipError_t launch_produce_op_fmt(const uint16_t *x, int64_t ldx, const uint16_t *a, int64_t lda,
                                 const uint16_t *b, int64_t ldb, uint16_t *y, int64_t rows,
                                 int64_t cols, const float *scale, uint8_t *q, uint8_t *qt,
                                 float *amax_cur, float *scale_inv_out, const int32_t *noop,
                                 hipStream_t stream) {
    const int64_t tiles_c = (cols + TILE - 1) / TILE;
    const dim3 grid((unsigned)(((rows + TILE - 1) / TILE) * tiles_c));
    if (q && qt)
        hipLaunchKernelGGL((produce_cast_kernel<OP, FMT, true, true>), grid, dim3(THREADS), 0,
                           stream, x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur,
                           scale_inv_out, noop, tiles_c);
    else if (q)
        hipLaunchKernelGGL((produce_cast_kernel<OP, FMT, true, false>), grid, dim3(THREADS), 0,
                           stream, x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur,
                           scale_inv_out, noop, tiles_c);
    else
        hipLaunchKernelGGL((produce_cast_kernel<OP, FMT, false, true>), grid, dim3(THREADS), 0,
                           stream, x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur,
                           scale_inv_out, noop, tiles_c);
    return hipGetLastError();
}

// Dropout in front of a cast, one pass: y = bf16(residual + dropout(x)) (or
// the dropout alone; the arithmetic of dropout.hip), y cast exactly as
// fp8_cast_transpose_amax casts a bf16 source, its column sums as
// fp8_cast_transpose_amax_dbias takes them.  One workgroup per 128 x 128
// tile in the lane layout of the cast: a lane's 8-column source chunk is one
// group of the generator, so a lane makes eight Philox calls for its 64
// elements while its loads are in flight.  A lane stores y where it alone has
// read x and the residual, so y may be either of them.  The sources are read
// once, past the last-level cache, which keeps the codes for the products.
// Bound by its bytes: [8192, 2048] with a residual to E4M3 28 us (134 MB, 4.8
// TB/s; 31 us with ordinary loads; a copy of as much 26), the gradient
// [8192, 8192] to E5M2 with its column sums 61 to 63 us (268 MB, 4.3 TB/s) and 5
// for the sums of the tile rows.
template <int FMT, bool WANT_Q, bool WANT_QT, bool DBIAS>
__global__ __launch_bounds__(THREADS) void dropout_cast_kernel(
    const uint16_t *x, int64_t ldx, const uint16_t *res, int64_t ldres, uint16_t *y, int64_t ldy,
    int64_t rows, int64_t cols, DropoutArgs drop,
    const float *__restrict__ scale_ptr, uint8_t *__restrict__ q, uint8_t *__restrict__ qt,
    float *__restrict__ amax_cur, float *__restrict__ scale_inv_out,
    const int32_t *__restrict__ noop, int64_t tiles_c, float *__restrict__ dbias_ws,
    int64_t ws_ld) {
#pragma clang fp contract(off)
    if (noop != nullptr && *noop != 0) return;
    __shared__ uint32_t lds_t[TILE * (TILE / 4)];
    __shared__ uint32_t lds_amax[THREADS / 64];
    __shared__ float lds_db[DBIAS ? (THREADS / 64) * TILE : 1];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int cc = lane & 7;
    const int cq = store_chunk<FP8_DTYPE_BF16>(cc);
    const int rg = wave * 8 + (lane >> 3);
    const float s = *scale_ptr;
    const bool s_special = !(fabsf(s) > 0.0f && fabsf(s) <= 3.402823466e38f);
    if (blockIdx.x == 0 && tid == 0 && scale_inv_out != nullptr) *scale_inv_out = 1.0f / s;
    const DropoutKey dkey(drop.rng);

    const int64_t t = blockIdx.x;
    const int64_t tr = t / tiles_c, tcn = t - tr * tiles_c;
    const int64_t row0 = tr * TILE, col0 = tcn * TILE;
    const int64_t r = row0 + 4 * rg, c = col0 + 16 * cq;
    const bool valid = (r < rows) && (c < cols);   // rows, cols are multiples of 16
    const bool add = res != nullptr;

    // All loads first: the lane's two chunks of its four rows.
    u32x4 xs[4][2], rs[4][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t ch = col0 + 64 * h + 8 * cc;
        const bool in = r < rows && ch < cols;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xs[i][h] = rs[i][h] = u32x4{0u, 0u, 0u, 0u};
            if (in) {
                xs[i][h] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4 *>(x + (r + i) * ldx + ch));
                if (add)
                    rs[i][h] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(res + (r + i) * ldres + ch));
            }
        }
    }
    SrcRow<FP8_DTYPE_BF16> ys[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t ch = col0 + 64 * h + 8 * cc;
        const bool in = r < rows && ch < cols;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
            dropout_words(dkey, (uint64_t)((r + i) * (cols >> 3) + (ch >> 3)), w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t xw = xs[i][h][k], rw = rs[i][h][k];
                const bool keep0 = (w[k] & 0xFFFFu) >= drop.threshold;
                const bool keep1 = (w[k] >> 16) >= drop.threshold;
                float v0 = keep0 ? bf16_lo(xw) * drop.factor : 0.0f;
                float v1 = keep1 ? bf16_hi(xw) * drop.factor : 0.0f;
                if (add) {
                    v0 = bf16_lo(rw) + v0;
                    v1 = bf16_hi(rw) + v1;
                }
                const uint32_t y0 = bf16_bits(v0);
                const uint32_t y1 = bf16_bits(v1);
                ys[i].v[h][k] = y0 | (y1 << 16);
            }
            if (y != nullptr && in) *reinterpret_cast<u32x4 *>(y + (r + i) * ldy + ch) = ys[i].v[h];
        }
    }
    uint32_t key = 0;
    encode_block<FP8_DTYPE_BF16, FMT, WANT_Q, WANT_QT>(ys, s, s_special, valid, q, r, c, cols, cq,
                                                       rg, lane, nullptr, lds_t, key);
    if constexpr (DBIAS) tile_col_sums_to_lds<FP8_DTYPE_BF16>(ys, &lds_db[wave * TILE], lane, cc);
    __syncthreads();
    if constexpr (WANT_QT) store_transposed(lds_t, qt, rows, cols, row0, col0, lane, wave);
    if constexpr (DBIAS) tile_col_sums_out(lds_db, tid, dbias_ws, ws_ld, tr, tcn);
    if (amax_cur != nullptr) flush_amax(key, amax_cur, lds_amax, lane, wave, tid);
}

template <int FMT>
hipError_t launch_dropout_cast_fmt(const uint16_t *x, int64_t ldx, const uint16_t *res,
                                   int64_t ldres, uint16_t *y, int64_t ldy, int64_t rows,
                                   int64_t cols, const DropoutArgs &drop, const float *scale,
                                   uint8_t *q, uint8_t *qt, float *amax_cur, float *scale_inv_out,
                                   const int32_t *noop, float *dbias_ws, int64_t ws_ld,
                                   hipStream_t stream) {
    const int64_t tiles_c = (cols + TILE - 1) / TILE;
    const dim3 grid((unsigned)(((rows + TILE - 1) / TILE) * tiles_c));
    auto launch = [&](auto wq, auto wqt, auto db) {
        hipLaunchKernelGGL((dropout_cast_kernel<FMT, decltype(wq)::value, decltype(wqt)::value,
                                                decltype(db)::value>),
                           grid, dim3(THREADS), 0, stream, x, ldx, res, ldres, y, ldy, rows, cols,
                           drop, scale, q, qt, amax_cur, scale_inv_out, noop, tiles_c, dbias_ws,
                           ws_ld);
    };
    using T1 = std::true_type;
    using F1 = std::false_type;
    auto by_layout = [&](auto db) {
        if (q && qt) launch(T1{}, T1{}, db);
        else if (q) launch(T1{}, F1{}, db);
        else launch(F1{}, T1{}, db);
    };
    if (dbias_ws) by_layout(T1{});
    else by_layout(F1{});
    return hipGetLastError();
}

// Rows gathered into expert order in front of a cast: y[slot(t, k)] = x[t], or
// bf16(weights[t, k] * x[t]), cast as fp8_cast_transpose_amax casts y, each
// segment of the plan with a transpose of its own.  One workgroup per 128 x 128
// tile in the lane layout of the cast; a tile lies within one segment, and a lane
// finds the tokens of its four rows in the plan's sources.  Rows without a pair are
// zeros.  Workgroups behind the plan's last tile have nothing to do.
//
// A source row is read once for each of its pairs, from the last-level cache after the
// first (ordinary loads: they have to stay there).  8192 tokens of 2048 columns, two
// choices, to E4M3: 24 to 26 us a call for 101 MB that it cannot do without (4 TB/s; 134 MB
// with the second reads, the rate of a plain cast of as many rows).  Small calls are the
// chain plan, sources, rows, stores: 16 tokens 4.3 us in a graph.
template <int FMT, bool WANT_Q, bool WANT_QT, bool WEIGHTS>
__global__ __launch_bounds__(THREADS) void expert_gather_cast_kernel(
    ExpertView plan, const uint16_t *__restrict__ x, uint32_t ldx, int64_t cols,
    const float *__restrict__ weights, const float *__restrict__ scale_ptr,
    uint8_t *__restrict__ q, uint8_t *__restrict__ qt, float *__restrict__ amax_cur,
    float *__restrict__ scale_inv_out, const int32_t *__restrict__ noop, int64_t tiles_c) {
    if (noop != nullptr && *noop != 0) return;
    __shared__ uint32_t lds_t[TILE * (TILE / 4)];
    __shared__ uint32_t lds_amax[THREADS / 64];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int cc = lane & 7;
    const int cq = store_chunk<FP8_DTYPE_BF16>(cc);
    const int rg = wave * 8 + (lane >> 3);
    // The plan's header, the tile and the scale in one go (the grid ends with the
    // plan's space for tiles).
    const int64_t tr = blockIdx.x / tiles_c, tcn = blockIdx.x - tr * tiles_c;
    const int4 tile = plan.tiles[tr];
    const bool used = tr < plan.header[5];
    const float s = *scale_ptr;
    const bool s_special = !(fabsf(s) > 0.0f && fabsf(s) <= 3.402823466e38f);
    if (!plan.built()) return;
    if (blockIdx.x == 0 && tid == 0 && scale_inv_out != nullptr) *scale_inv_out = 1.0f / s;
    if (!used) return;
    const int64_t rows = tile.y, first = tile.z;         // the segment
    const int64_t row0 = tile.x, col0 = tcn * TILE;
    const int64_t r = row0 + 4 * rg, c = col0 + 16 * cq;
    const bool valid = (r < rows) && (c < cols);   // rows, cols are multiples of 16
    q += first * cols;
    qt += first * cols;

    int4 source = {-1, -1, -1, -1};
    if (r < rows) source = *reinterpret_cast<const int4 *>(plan.sources + first + r);
    const int pair[4] = {source.x, source.y, source.z, source.w};
    SrcRow<FP8_DTYPE_BF16> ys[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = WEIGHTS && pair[i] >= 0 ? weights[pair[i]] : 0.0f;
        const char *row = reinterpret_cast<const char *>(x) +
                          (uint64_t)plan.token_of((uint32_t)max(pair[i], 0)) * ldx;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t ch = col0 + 64 * h + 8 * cc;
            ys[i].v[h] = u32x4{0u, 0u, 0u, 0u};
            if (pair[i] >= 0 && ch < cols)
                ys[i].v[h] = *reinterpret_cast<const u32x4 *>(row + 2 * ch);
        }
    }
    if constexpr (WEIGHTS) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // Past the columns 0 * 0 as well, whatever the weight.
                const float wh = col0 + 64 * h + 8 * cc < cols ? w[i] : 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t xw = ys[i].v[h][k];
                    const float v0 = wh * bf16_lo(xw), v1 = wh * bf16_hi(xw);
                    const uint32_t y0 = bf16_bits(v0);
                    const uint32_t y1 = bf16_bits(v1);
                    ys[i].v[h][k] = y0 | (y1 << 16);     // +0 without a pair: 0 * 0
                }
            }
    }
    uint32_t key = 0;
    encode_block<FP8_DTYPE_BF16, FMT, WANT_Q, WANT_QT>(ys, s, s_special, valid, q, r, c, cols, cq,
                                                       rg, lane, nullptr, lds_t, key);
    __syncthreads();
    if constexpr (WANT_QT) store_transposed(lds_t, qt, rows, cols, row0, col0, lane, wave);
    if (amax_cur != nullptr) flush_amax(key, amax_cur, lds_amax, lane, wave, tid);
}

template <int FMT, bool WEIGHTS>
hipError_t launch_expert_gather_cast_fmt(const ExpertShape &shape, const int32_t *plan,
                                         const uint16_t *x, int64_t ldx, int64_t cols,
                                         const float *weights, const float *scale, uint8_t *q,
                                         uint8_t *qt, float *amax_cur, float *scale_inv_out,
                                         const int32_t *noop, hipStream_t stream) {
    const int64_t tiles_c = (cols + TILE - 1) / TILE;
    const dim3 grid((unsigned)(shape.tiles_max * tiles_c));
    // By registers a CU holds seven workgroups, six with weights; codes alone run so.  A
    // tile with a transpose keeps 17 KB of LDS, and 12 KB more leave five: better in a grid
    // of more than seven a CU, with weights more than eight.  us with 7 / 6 / 5 to E4M3 and
    // 6 / 5 with weights to E5M2, two choices: 1664 tiles (6144 x 2048) 16.1 / 16.2 / 17.0
    // and 19.7 / 20.8, 1920 (7168 x 2048) 21.1 to 22.5 / 20.2 / 20.9 and 23.2 / 24.8, 2176
    // (8192 x 2048) 28.3 / 27.5 / 26.4 and 29.7 / 29.3, 2560 (2048 x 8192) 30.0 / 28.9 / 27.9
    // and 30.7 / 29.9.
    unsigned lds = 0;
    if (qt) {
        int cus = 0;
        if (hipError_t e = current_cu_count(&cus)) return e;
        if (shape.tiles_max * tiles_c > (WEIGHTS ? 8 : 7) * (int64_t)cus) lds = 12 * 1024;
    }
    auto launch = [&](auto wq, auto wqt) {
        hipLaunchKernelGGL((expert_gather_cast_kernel<FMT, decltype(wq)::value,
                                                      decltype(wqt)::value, WEIGHTS>),
                           grid, dim3(THREADS), lds, stream, ExpertView(shape, plan), x,
                           (uint32_t)(2 * ldx), cols, weights, scale, q, qt, amax_cur,
                           scale_inv_out, noop, tiles_c);
    };
    using T1 = std::true_type;
    using F1 = std::false_type;
    if (q && qt) launch(T1{}, T1{});
    else if (q) launch(T1{}, F1{});
    else launch(F1{}, T1{});
    return hipGetLastError();
}

// Gradient of the modulation producer y = a * x / b (FP8_PRODUCE_MODULATE,
// or _FINITE) with respect to x, a and b, for the output gradient dy of y.
// fp32 on the widened bf16 inputs, each step rounded to nearest even:
// u = (a * x) / b (the forward's quotient), t = dy / b, then
// dx = bf16(t * a), da = bf16(t * x), db = bf16(-(t * u)); a NaN is written
// 0x7FC0.  FINITE: +0 in all three where the forward's bf16(u) is infinite
// or NaN (the forward wrote the constant +0 there).
template <bool FINITE>
__device__ __forceinline__ void modulate_grad_pair(uint32_t gw, uint32_t xw, uint32_t aw,
                                                   uint32_t bw, uint32_t &ox, uint32_t &oa,
                                                   uint32_t &ob) {
    ox = oa = ob = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        auto wide = [h](uint32_t w) { return __uint_as_float(h ? (w & 0xFFFF0000u) : (w << 16)); };
        const float gv = wide(gw), xv = wide(xw), av = wide(aw), bv = wide(bw);
        const float u = (av * xv) / bv;
        const float t = gv / bv;
        uint32_t rx = bf16_bits(t * av), ra = bf16_bits(t * xv), rb = bf16_bits(-(t * u));
        if constexpr (FINITE) {
            if ((bf16_bits(u) & 0x7F80u) == 0x7F80u) rx = ra = rb = 0u;
        }
        ox |= rx << (16 * h);
        oa |= ra << (16 * h);
        ob |= rb << (16 * h);
    }
}

// One lane per 8 consecutive columns of one row: four 16-byte loads, three
// 16-byte stores.  vec_per_row = cols / 8.
template <bool FINITE>
__global__ __launch_bounds__(THREADS) void modulate_backward_kernel(
    const uint16_t *__restrict__ dy, int64_t lddy, const uint16_t *__restrict__ x, int64_t ldx,
    const uint16_t *__restrict__ a, int64_t lda, const uint16_t *__restrict__ b, int64_t ldb,
    uint16_t *__restrict__ dx, int64_t lddx, uint16_t *__restrict__ da, int64_t ldda,
    uint16_t *__restrict__ db, int64_t lddb, int64_t rows, int64_t vec_per_row) {
    const int64_t v = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (v >= rows * vec_per_row) return;
    const int64_t r = v / vec_per_row;
    const int64_t c = (v - r * vec_per_row) * 8;
    const u32x4 G = *reinterpret_cast<const u32x4 *>(dy + r * lddy + c);
    const u32x4 X = *reinterpret_cast<const u32x4 *>(x + r * ldx + c);
    const u32x4 A = *reinterpret_cast<const u32x4 *>(a + r * lda + c);
    const u32x4 B = *reinterpret_cast<const u32x4 *>(b + r * ldb + c);
    const uint32_t g[4] = {G.x, G.y, G.z, G.w}, xs[4] = {X.x, X.y, X.z, X.w},
                   as[4] = {A.x, A.y, A.z, A.w}, bs[4] = {B.x, B.y, B.z, B.w};
    uint32_t ox[4], oa[4], ob[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        modulate_grad_pair<FINITE>(g[k], xs[k], as[k], bs[k], ox[k], oa[k], ob[k]);
    *reinterpret_cast<u32x4 *>(dx + r * lddx + c) = u32x4{ox[0], ox[1], ox[2], ox[3]};
    *reinterpret_cast<u32x4 *>(da + r * ldda + c) = u32x4{oa[0], oa[1], oa[2], oa[3]};
    *reinterpret_cast<u32x4 *>(db + r * lddb + c) = u32x4{ob[0], ob[1], ob[2], ob[3]};
}

// Bias gradient, second pass: dbias[c] = sum over tile rows tr of
// ws[tr * ws_ld + c].  A workgroup takes 64 columns; its four 64-thread
// parts add the tile rows of four contiguous ranges (loads issued sixteen at
// a time, added in row order) and part 0 adds the four part sums in part
// order, so the order is fixed.  tiles_r = 0 writes zeros.
__global__ __launch_bounds__(256) void dbias_reduce_kernel(const float *__restrict__ ws,
                                                           int64_t tiles_r, int64_t ws_ld,
                                                           int64_t cols, float *__restrict__ dbias,
                                                           const int32_t *__restrict__ noop) {
    if (noop != nullptr && *noop != 0) return;
    __shared__ float part_sum[4][64];
    const int cl = threadIdx.x & 63, part = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + cl;
    const int64_t per = (tiles_r + 3) / 4;
    const int64_t r0 = min(tiles_r, part * per), r1 = min(tiles_r, r0 + per);
    float acc = 0.0f;
    if (c < cols) {
        int64_t r = r0;
        for (; r + 16 <= r1; r += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = ws[(r + k) * ws_ld + c];
#pragma unroll
            for (int k = 0; k < 16; ++k) acc += v[k];
        }
        for (; r < r1; ++r) acc += ws[r * ws_ld + c];
    }
    part_sum[part][cl] = acc;
    __syncthreads();
    if (part == 0 && c < cols)
        dbias[c] = ((part_sum[0][cl] + part_sum[1][cl]) + part_sum[2][cl]) + part_sum[3][cl];
}

hipError_t launch_dbias_reduce(const float *ws, int64_t tiles_r, int64_t ws_ld, int64_t cols,
                               float *dbias, const int32_t *noop, hipStream_t stream) {
    if (cols == 0) return hipSuccess;
    hipLaunchKernelGGL(dbias_reduce_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0,
                       stream, ws, tiles_r, ws_ld, cols, dbias, noop);
    return hipGetLastError();
}

hipError_t launch_produce_cast(int op, const uint16_t *x, int64_t ldx, const uint16_t *a,
                               int64_t lda, const uint16_t *b, int64_t ldb, uint16_t *y,
                               int64_t rows, int64_t cols, const float *scale, int fmt,
                               uint8_t *q, uint8_t *qt, float *amax_cur, float *scale_inv_out,
                               const int32_t *noop, hipStream_t stream) {
    if (op == FP8_PRODUCE_MODULATE) {
        if (fmt == FP8_E4M3)
            return launch_produce_op_fmt<FP8_PRODUCE_MODULATE, FP8_E4M3>(
                x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
                stream);
        return launch_produce_op_fmt<FP8_PRODUCE_MODULATE, FP8_E5M2>(
            x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
            stream);
    }
    if (op == FP8_PRODUCE_MODULATE_FINITE) {
        if (fmt == FP8_E4M3)
            return launch_produce_op_fmt<FP8_PRODUCE_MODULATE_FINITE, FP8_E4M3>(
                x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
                stream);
        return launch_produce_op_fmt<FP8_PRODUCE_MODULATE_FINITE, FP8_E5M2>(
            x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
            stream);
    }
    if (op == FP8_PRODUCE_ADD2) {
        if (fmt == FP8_E4M3)
            return launch_produce_op_fmt<FP8_PRODUCE_ADD2, FP8_E4M3>(
                x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
                stream);
        return launch_produce_op_fmt<FP8_PRODUCE_ADD2, FP8_E5M2>(
            x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
            stream);
    }
    if (fmt == FP8_E4M3)
        return launch_produce_op_fmt<FP8_PRODUCE_ADD, FP8_E4M3>(
            x, ldx, a, lda, b, ldb, y, rows, cols, scale, q, qt, amax_cur, scale_inv_out, noop,
            stream);
    return launch_produce_op_fmt<FP8_PRODUCE_ADD, FP8_E5M2>(x, ldx, a, lda, b, ldb, y, rows, cols,
                                                            scale, q, qt, amax_cur, scale_inv_out,
                                                            noop, stream);
}

hipError_t launch_dropout_cast(const uint16_t *x, int64_t ldx, const uint16_t *residual,
                               int64_t ldres, uint16_t *y, int64_t ldy, int64_t rows, int64_t cols,
                               const DropoutArgs &drop, const float *scale, int fmt, uint8_t *q,
                               uint8_t *qt, float *amax_cur, float *scale_inv_out,
                               const int32_t *noop, float *dbias_ws, int64_t ws_ld,
                               hipStream_t stream) {
    if (fmt == FP8_E4M3)
        return launch_dropout_cast_fmt<FP8_E4M3>(x, ldx, residual, ldres, y, ldy, rows, cols, drop,
                                                 scale, q, qt, amax_cur, scale_inv_out, noop,
                                                 dbias_ws, ws_ld, stream);
    return launch_dropout_cast_fmt<FP8_E5M2>(x, ldx, residual, ldres, y, ldy, rows, cols, drop,
                                             scale, q, qt, amax_cur, scale_inv_out, noop, dbias_ws,
                                             ws_ld, stream);
}

hipError_t launch_expert_gather_cast(const ExpertShape &shape, const int32_t *plan,
                                     const uint16_t *x, int64_t ldx, int64_t cols,
                                     const float *weights, const float *scale, int fmt, uint8_t *q,
                                     uint8_t *qt, float *amax_cur, float *scale_inv_out,
                                     const int32_t *noop, hipStream_t stream) {
    const auto launch = fmt == FP8_E4M3 ? (weights ? launch_expert_gather_cast_fmt<FP8_E4M3, true>
                                                   : launch_expert_gather_cast_fmt<FP8_E4M3, false>)
                                        : (weights ? launch_expert_gather_cast_fmt<FP8_E5M2, true>
                                                   : launch_expert_gather_cast_fmt<FP8_E5M2, false>);
    return launch(shape, plan, x, ldx, cols, weights, scale, q, qt, amax_cur, scale_inv_out, noop,
                  stream);
}

hipError_t launch_modulate_backward(bool finite, const uint16_t *dy, int64_t lddy,
                                    const uint16_t *x, int64_t ldx, const uint16_t *a,
                                    int64_t lda, const uint16_t *b, int64_t ldb, uint16_t *dx,
                                    int64_t lddx, uint16_t *da, int64_t ldda, uint16_t *db,
                                    int64_t lddb, int64_t rows, int64_t cols,
                                    hipStream_t stream) {
    const int64_t vec_per_row = cols / 8;
    const dim3 grid((unsigned)((rows * vec_per_row + THREADS - 1) / THREADS));
    if (finite)
        hipLaunchKernelGGL(modulate_backward_kernel<true>, grid, dim3(THREADS), 0, stream, dy,
                           lddy, x, ldx, a, lda, b, ldb, dx, lddx, da, ldda, db, lddb, rows,
                           vec_per_row);
    else
        hipLaunchKernelGGL(modulate_backward_kernel<false>, grid, dim3(THREADS), 0, stream, dy,
                           lddy, x, ldx, a, lda, b, ldb, dx, lddx, da, ldda, db, lddb, rows,
                           vec_per_row);
    return hipGetLastError();
}

}  // namespace fp8dsl
