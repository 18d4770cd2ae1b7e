// The gradients' norm and the AdamW step over many tensors.
//
// The tensors of a launch are kernel arguments (by value, within the 4 KB that a
// launch takes), so a call reads no host memory later and can be captured; their
// tiles are one list, which the workgroups share evenly.
//
// Bound by memory: the step moves 28 bytes a value in fp32, 16 with 8-bit moments, 10
// with bf16 parameters and gradients on top (there the generator, 13 quarter-rate multiplies
// per four values, and the arithmetic come near the memory's time).  Measured on MI355X,
// where a large copy moves 5.1 TB/s: 32 million values in fp32 159 us (5.9 TB/s), with 8-bit
// moments 96 (5.6), all of it in bf16 with them 67 (5.0); the 2.7 billion of the 32-block
// toy stack 13.2 ms (5.7) and 7.8 ms.  The norm reads 2 GiB at 6.0 TB/s, 336 MB at 5.3; behind
// other kernels it pays for the writing back of what they left in the last-level cache.
// Small calls: a step of two adapters (2^19 bf16 values) 6.1 us in a graph.
#include "adamw.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "bf16.h"
#include "dropout.h"
#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;

template <typename V>
__device__ __forceinline__ V load_once(const void *p) {
    return __builtin_nontemporal_load(static_cast<const V *>(p));
}
template <typename V>
__device__ __forceinline__ void store_once(void *p, V v) {
    __builtin_nontemporal_store(v, static_cast<V *>(p));
}

// Four values of a tensor from element i on, `left` of them (1 .. 4) there, past the
// last-level cache: a step touches every value once, and what it would leave there
// are the last tensors' values only.  Measured (all loads and stores of a step so,
// against none): a toy block in fp32 with the norm before it 456 us against 538,
// 67 million values in 8 bits 224 against 263, 16 million fp32 values alone 84
// against 94, 1 million 12.0 against 13.4.  (With the norm, gradients that it has read
// are still in that cache, and the step begins with the last of them.)
template <typename T>
struct Four;
template <>
struct Four<float> {
    static __device__ __forceinline__ void load(const void *p, int64_t i, int left, float (&o)[4]) {
        const float *at = static_cast<const float *>(p) + i;
        if (left >= 4) {
            const u32x4 v = load_once<u32x4>(at);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __uint_as_float(v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = k < left ? at[k] : 0.0f;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, int left, const float (&v)[4]) {
        float *at = static_cast<float *>(p) + i;
        if (left >= 4) {
            store_once(at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                 __float_as_uint(v[2]), __float_as_uint(v[3])});
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < left) at[k] = v[k];
        }
    }
};
// bf16: the bits of a value are the upper half of an fp32's.
template <>
struct Four<uint16_t> {
    static __device__ __forceinline__ void load(const void *p, int64_t i, int left, float (&o)[4]) {
        const uint16_t *at = static_cast<const uint16_t *>(p) + i;
        if (left >= 4) {
            const u32x2 v = load_once<u32x2>(at);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = __uint_as_float(k & 1 ? v[k / 2] & 0xFFFF0000u : v[k / 2] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = k < left ? __uint_as_float((uint32_t)at[k] << 16) : 0.0f;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, int left,
                                                 const uint32_t (&bits)[4]) {
        uint16_t *at = static_cast<uint16_t *>(p) + i;
        if (left >= 4) {
            store_once(at, u32x2{bits[0] | (bits[1] << 16), bits[2] | (bits[3] << 16)});
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < left) at[k] = (uint16_t)bits[k];
        }
    }
};
template <>
struct Four<uint8_t> {
    static __device__ __forceinline__ uint32_t load(const void *p, int64_t i, int left) {
        const uint8_t *at = static_cast<const uint8_t *>(p) + i;
        if (left >= 4) return load_once<uint32_t>(at);
        uint32_t v = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < left) v |= (uint32_t)at[k] << (8 * k);
        return v;
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, int left, uint32_t v) {
        uint8_t *at = static_cast<uint8_t *>(p) + i;
        if (left >= 4) {
            store_once(at, v);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < left) at[k] = (uint8_t)(v >> (8 * k));
        }
    }
};

// ---- the norm ----------------------------------------------------------------

// Pieces of 16 bytes that a lane takes at once; a tile is a workgroup's.
constexpr int NORM_STEPS = 4;
constexpr int64_t NORM_TILE_BYTES = THREADS * 16 * NORM_STEPS;
constexpr int NORM_TENSORS = 100;

struct NormTensor {
    const void *grad;
    int64_t n;
    int32_t first;           // its first tile
    int32_t bf16;
};
struct NormArgs {
    int count, tiles;
    int again;               // earlier launches have left sums in parts
    NormTensor t[NORM_TENSORS];
};
static_assert(sizeof(NormArgs) <= 3584, "kernel arguments");

// The last tensor whose first tile is at most `tile` (wave-uniform).
template <typename Args>
__device__ __forceinline__ int tensor_of(const Args &args, int tile) {
    int lo = 0, hi = args.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (args.t[mid].first <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

__device__ __forceinline__ void add_square(float x, double &sum) {
    sum = fma((double)x, (double)x, sum);
}

// Adds the squares of tile `tile` of a tensor of 4-byte or 2-byte values.
template <bool BF16, bool FULL>
__device__ __forceinline__ void add_tile(const NormTensor &t, int tile, double (&sum)[4]) {
    constexpr int E = BF16 ? 8 : 4;                      // values of 16 bytes
    const int64_t i0 = tile * (NORM_TILE_BYTES / 16 * E) + E * threadIdx.x;
    u32x4 v[NORM_STEPS];
#pragma unroll
    for (int s = 0; s < NORM_STEPS; ++s) {
        const int64_t i = i0 + s * THREADS * E;
        v[s] = u32x4{0u, 0u, 0u, 0u};
        if (FULL || i + E <= t.n) {
            v[s] = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(t.grad) +
                                                    i * (16 / E));
        } else if (BF16) {
            const uint16_t *at = static_cast<const uint16_t *>(t.grad);
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (i + k < t.n) v[s][k / 2] |= (uint32_t)at[i + k] << (16 * (k & 1));
        } else {
            const uint32_t *at = static_cast<const uint32_t *>(t.grad);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < t.n) v[s][k] = at[i + k];
        }
    }
#pragma unroll
    for (int s = 0; s < NORM_STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BF16) {
                add_square(__uint_as_float(v[s][k] << 16), sum[k]);
                add_square(__uint_as_float(v[s][k] & 0xFFFF0000u), sum[k]);
            } else {
                add_square(__uint_as_float(v[s][k]), sum[k]);
            }
        }
}

// Each workgroup takes a run of tiles, so it looks for its first tensor only.
__global__ __launch_bounds__(THREADS) void grad_norm_kernel(const NormArgs args,
                                                            double *__restrict__ parts) {
    __shared__ double waves[WAVES];
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    const int t0 = (int)((int64_t)args.tiles * blockIdx.x / gridDim.x);
    const int t1 = (int)((int64_t)args.tiles * (blockIdx.x + 1) / gridDim.x);
    int item = tensor_of(args, t0);
    for (int tile = t0; tile < t1; ++tile) {
        while (item + 1 < args.count && args.t[item + 1].first <= tile) ++item;
        const NormTensor &t = args.t[item];
        // Loads without branches where the tile is whole.
        const int at = tile - t.first;
        const bool full = t.n >= (at + 1) * (NORM_TILE_BYTES / (t.bf16 ? 2 : 4));
        if (t.bf16) full ? add_tile<true, true>(t, at, sum) : add_tile<true, false>(t, at, sum);
        else full ? add_tile<false, true>(t, at, sum) : add_tile<false, false>(t, at, sum);
    }
    const double all = wave_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        const double mine = (waves[0] + waves[1]) + (waves[2] + waves[3]);
        parts[blockIdx.x] = args.again ? parts[blockIdx.x] + mine : mine;
    }
}

__global__ __launch_bounds__(THREADS) void grad_norm_sum_kernel(const double *__restrict__ parts,
                                                                int count, float max_norm,
                                                                float *__restrict__ norm,
                                                                float *__restrict__ factor,
                                                                int32_t *__restrict__ flag) {
    __shared__ double waves[WAVES];
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += THREADS) sum += parts[i];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        const float all = (float)sqrt((waves[0] + waves[1]) + (waves[2] + waves[3]));
        *norm = all;
        if (factor) *factor = all > max_norm ? max_norm / all : 1.0f;
        if (flag) *flag = fabsf(all) <= 3.402823466e38f ? 0 : 1;
    }
}

// ---- the step ----------------------------------------------------------------

constexpr int BLOCK = FP8DSL_ADAMW_BLOCK;
// Blocks of 256 that a wave takes at once: four, for the bytes in flight, or one where
// that gives a compute unit no more than one workgroup.  us in a graph with 1 / 2 / 4:
// 524288 bf16 values with 8-bit states 6.0 / 6.2 / 7.5, 2^20 7.3 / 7.3 / 7.9, 2^21 10.6 /
// 9.3 / 9.5; 2^20 fp32 values 8.1 / 8.1 / 8.0, 2^21 13.2 / 12.8 / 13.1; a toy block in fp32
// 474 / 450 / 432 (8: 456).
constexpr int STEP_BLOCKS = 4;
constexpr int step_tile(int blocks) { return WAVES * blocks * BLOCK; }
constexpr int STEP_TENSORS = 48;
// Counters behind the step count, 128 bytes apart.
constexpr int TICKET_GROUPS = 64;
static_assert(128 * (1 + TICKET_GROUPS) == FP8DSL_ADAMW_STATE_BYTES, "state");
static_assert(BLOCK == 64 * 4, "a wave's lanes hold four values of a block each");

struct StepTensor {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    uint16_t *copy;
    int64_t n;
    int32_t first;           // its first tile
    float weight_decay;
    int32_t index;           // its place in the call
};
struct StepArgs {
    int count, tiles;
    int last;                // the launch that counts the step
    const float *lr, *grad_scale;
    int64_t *steps;
    double beta1, beta2;
    float b1, c1, b2, c2, eps;
    uint32_t seed_lo, seed_hi;
    StepTensor t[STEP_TENSORS];
};
static_assert(sizeof(StepArgs) <= 4064, "kernel arguments");

__device__ __forceinline__ double power(double x, uint64_t n) {
    double r = 1.0;
    for (; n; n >>= 1) {
        if (n & 1) r *= x;
        x *= x;
    }
    return r;
}

// What the step's values share.
struct Factors {
    float b1, c1, b2, c2, eps, grad, step, root, decay;
};

// Bits of the power of two that scales a block whose largest finite magnitude is
// `most` (bits): the least, 2^-126 or more, that keeps it within 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_bits(uint32_t most) {
    const int e = (int)((most + 0x1FFFFFu) >> 23);      // one more beyond 1.75
    return (uint32_t)max(e - 8, 1) << 23;
}

// The maximum over the wave (all lanes active): within rows of 16, then across.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Four E4M3 codes of x (magnitudes of at most 448), each rounded by the upper half of
// its u: the converter adds u to the 20 bits below a code's three (below 2^-6, to as
// many below the step of 2^-9) and cuts, which is floor(place + u / 2^16).
__device__ __forceinline__ uint32_t convert4(const float (&x)[4], const uint32_t (&u)[4]) {
    int c = __builtin_amdgcn_cvt_sr_fp8_f32(x[0], (int)u[0], 0, 0);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[1], (int)u[1], c, 1);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[2], (int)u[2], c, 2);
    return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(x[3], (int)u[3], c, 3);
}

// Four codes of a moment under the power of two `scale`.  KEEP: a value above 0 gets
// a code above 0.  SPECIAL: what is not finite becomes 0x7F.
template <bool KEEP, bool SPECIAL>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[4], uint32_t scale,
                                             const uint32_t (&u)[4]) {
    // 1 / 2^e: e and its negative are both exponents of normal numbers.
    const float inverse = __uint_as_float((254u << 23) - scale);
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = x[k] * inverse;
    uint32_t codes = convert4(y, u);
    // A byte of zero borrows from the one above; no other code has its upper bit set.
    if (KEEP && ((codes - 0x01010101u) & 0x80808080u)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (y[k] > 0.0f && ((codes >> (8 * k)) & 0xFFu) == 0) codes |= 1u << (8 * k);
    }
    if constexpr (SPECIAL) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((__float_as_uint(x[k]) & 0x7F800000u) == 0x7F800000u)
                codes = (codes & ~(0xFFu << (8 * k))) | (0x7Fu << (8 * k));
    }
    return codes;
}

// The largest magnitude (bits) of the wave's block of a moment.
template <bool SIGNED>
__device__ __forceinline__ uint32_t most_of(const float (&x)[4], bool finite_only) {
    uint32_t mag[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mag[k] = __float_as_uint(x[k]);
        if (SIGNED || finite_only) mag[k] &= 0x7FFFFFFFu;
        if (finite_only && mag[k] >= 0x7F800000u) mag[k] = 0;
    }
    return wave_max(max(max(mag[0], mag[1]), max(mag[2], mag[3])));
}

// The codes of a block's values and its scale; `most` is most_of(x, false).
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode(const float (&x)[4], uint32_t most,
                                           const uint32_t (&u)[4], uint32_t &scale) {
    if (most >= 0x7F800000u) {                           // rare, the same for the wave
        scale = scale_bits(most_of<SIGNED>(x, true));
        return codes_of<!SIGNED, true>(x, scale, u);
    }
    scale = scale_bits(most);
    return codes_of<!SIGNED, false>(x, scale, u);
}

__device__ __forceinline__ void decode(uint32_t codes, float scale, float (&x)[4]) {
    x[0] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 0) * scale;
    x[1] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 1) * scale;
    x[2] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 2) * scale;
    x[3] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 3) * scale;
}
// The code 0x7F of a second moment is an infinity, as an overflowed sum of squares is
// in fp32: it holds its parameter still (a NaN gradient leaves its NaN in m).
__device__ __forceinline__ void decode_square(uint32_t codes, float scale, float (&x)[4]) {
    decode(codes, scale, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = fminf(x[k], __builtin_inff());   // of a NaN: the infinity
}

// sqrt within 2^-23 of itself: the instruction does not take denormal numbers.
__device__ __forceinline__ float root_of(float x) {
    const bool small = x < 0x1p-96f;
    const float r = __builtin_amdgcn_sqrtf(small ? x * 0x1p32f : x);
    return small ? r * 0x1p-16f : r;
}
// The same times 2^12 where x < 2^104.
__device__ __forceinline__ float root_of_scaled(float x) {
    return __builtin_amdgcn_sqrtf(x * 0x1p24f);
}

// Lane l's value of v on lane l ^ 1.
__device__ __forceinline__ uint32_t from_neighbour(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}

// The two words of each of a lane's N fours of parameters.  An even lane has the first
// half of a group of eight, its neighbour the second: of two blocks each makes one
// block's words for both.
template <int N>
__device__ __forceinline__ void param_words(const DropoutKey &key, int index, int64_t i0, int lane,
                                            uint32_t (&out)[N][2]) {
    const bool odd = lane & 1;
    const auto words = [&](int64_t i, uint32_t (&w)[4]) {
        dropout_words(key, ((uint64_t)(2u * (uint32_t)index + 1u) << 32) | (uint64_t)(i / 8), w);
    };
    uint32_t w[4];
    if constexpr (N == 1) {
        words(i0 + 4 * lane, w);
        out[0][0] = odd ? w[2] : w[0];
        out[0][1] = odd ? w[3] : w[1];
    } else {
        static_assert(N % 2 == 0, "pairs of blocks");
#pragma unroll
        for (int s = 0; s < N; s += 2) {
            words(i0 + (s + odd) * BLOCK + 4 * lane, w);
            const uint32_t x0 = from_neighbour(odd ? w[0] : w[2]);
            const uint32_t x1 = from_neighbour(odd ? w[1] : w[3]);
            out[s][0] = odd ? x0 : w[0];
            out[s][1] = odd ? x1 : w[1];
            out[s + 1][0] = odd ? w[2] : x0;
            out[s + 1][1] = odd ? w[3] : x1;
        }
    }
}

// N blocks of 256 values of a tensor, a wave's; FULL: all of their values exist.
template <typename P, typename G, bool STATE8, int N, bool FULL>
__device__ __forceinline__ void step_blocks(const StepTensor &t, const Factors &f,
                                            const DropoutKey &key, int64_t i0) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    float p[N][4], g[N][4], m[N][4], v[N][4], ms[N], vs[N];
    uint32_t mc[N], vc[N], pw[N][2];
    int left[N];
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int64_t b = i0 + s * BLOCK, i = b + 4 * lane;
        left[s] = FULL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - i));
        if (FULL || left[s] > 0) {
            Four<P>::load(t.param, i, left[s], p[s]);
            Four<G>::load(t.grad, i, left[s], g[s]);
            if constexpr (STATE8) {
                mc[s] = Four<uint8_t>::load(t.m, i, left[s]);
                vc[s] = Four<uint8_t>::load(t.v, i, left[s]);
                ms[s] = t.m_scale[b / BLOCK];
                vs[s] = t.v_scale[b / BLOCK];
            } else {
                Four<float>::load(t.m, i, left[s], m[s]);
                Four<float>::load(t.v, i, left[s], v[s]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[s][k] = g[s][k] = m[s][k] = v[s][k] = 0.0f;
            mc[s] = vc[s] = 0;
            ms[s] = vs[s] = 0.0f;
        }
    }
    if constexpr (std::is_same<P, uint16_t>::value) param_words(key, t.index, i0, lane, pw);
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int64_t b = i0 + s * BLOCK, i = b + 4 * lane;
        if constexpr (STATE8) {
            decode(mc[s], ms[s], m[s]);
            decode_square(vc[s], vs[s], v[s]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gk = g[s][k] * f.grad;
            m[s][k] = m[s][k] * f.b1 + gk * f.c1;
            v[s][k] = v[s][k] * f.b2 + (gk * f.c2) * gk;
        }
        uint32_t most = 0xFFFFFFFFu;
        if constexpr (STATE8) most = most_of<false>(v[s], false);
        // A wave of ordinary values needs no look at each for the root.  (The divisor,
        // between eps and 2^101, has a normal reciprocal, or is infinite.)
        float r[4];
        if (most < 0x73000000u) {                        // 2^103
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = root_of_scaled(v[s][k]) * (f.root * 0x1p-12f);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = root_of(v[s][k]) * f.root;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[s][k] = p[s][k] * f.decay -
                      (m[s][k] * f.step) * __builtin_amdgcn_rcpf(r[k] + f.eps);
        uint32_t sm, sv;
        if constexpr (STATE8) {
            uint32_t w[4], um[4], uv[4];
            dropout_words(key, ((uint64_t)(2u * (uint32_t)t.index) << 32) | (uint64_t)(i / 4), w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                um[k] = w[k] << 16;
                uv[k] = w[k] & 0xFFFF0000u;
            }
            mc[s] = encode<true>(m[s], most_of<true>(m[s], false), um, sm);
            vc[s] = encode<false>(v[s], most, uv, sv);
        }
        if (!FULL && left[s] <= 0) continue;
        if constexpr (STATE8) {
            Four<uint8_t>::store(t.m, i, left[s], mc[s]);
            Four<uint8_t>::store(t.v, i, left[s], vc[s]);
            if (lane == 0) {
                t.m_scale[b / BLOCK] = __uint_as_float(sm);
                t.v_scale[b / BLOCK] = __uint_as_float(sv);
            }
        } else {
            Four<float>::store(t.m, i, left[s], m[s]);
            Four<float>::store(t.v, i, left[s], v[s]);
        }
        if constexpr (std::is_same<P, float>::value) {
            Four<float>::store(t.param, i, left[s], p[s]);
            if (t.copy) {
                const uint32_t bits[4] = {bf16_bits(p[s][0]), bf16_bits(p[s][1]),
                                          bf16_bits(p[s][2]), bf16_bits(p[s][3])};
                Four<uint16_t>::store(t.copy, i, left[s], bits);
            }
        } else {
            uint32_t bits[4];
            const uint32_t (&word)[2] = pw[s];
            // An infinity's bits below the upper half are zero: nothing is carried.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = k & 1 ? word[k / 2] >> 16 : word[k / 2] & 0xFFFFu;
                bits[k] = (__float_as_uint(p[s][k]) + u) >> 16;
            }
            const bool nan[4] = {p[s][0] != p[s][0], p[s][1] != p[s][1], p[s][2] != p[s][2],
                                 p[s][3] != p[s][3]};
            if (nan[0] | nan[1] | nan[2] | nan[3]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) bits[k] = nan[k] ? 0x7FC0u : bits[k];
            }
            Four<uint16_t>::store(t.param, i, left[s], bits);
        }
    }
}

template <typename P, typename G, bool STATE8, int N>
__global__ __launch_bounds__(THREADS) void adamw_kernel(const StepArgs args,
                                                        const int32_t *__restrict__ noop) {
    if (noop != nullptr && *noop != 0) return;
    __shared__ int64_t taken;
    if (threadIdx.x == 0) taken = args.steps[0];
    __syncthreads();
    const uint64_t steps = (uint64_t)taken + 1;
    const double lr = *args.lr;
    Factors f = {args.b1, args.c1, args.b2, args.c2, args.eps};
    f.grad = args.grad_scale ? *args.grad_scale : 1.0f;
    f.step = (float)(lr / (1.0 - power(args.beta1, steps)));
    f.root = (float)(1.0 / sqrt(1.0 - power(args.beta2, steps)));
    const DropoutKey key(args.seed_lo, args.seed_hi, steps);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int tile = args.tiles - 1 - (int)blockIdx.x; tile >= 0; tile -= gridDim.x) {
        const StepTensor &t = args.t[tensor_of(args, tile)];
        const int64_t i0 = (int64_t)(tile - t.first) * step_tile(N) + wave * N * BLOCK;
        f.decay = (float)(1.0 - lr * (double)t.weight_decay);
        if (t.n - i0 >= N * BLOCK) {
            step_blocks<P, G, STATE8, N, true>(t, f, key, i0);
        } else {
            for (int64_t i = i0; i < min(t.n, i0 + N * BLOCK); i += BLOCK)
                step_blocks<P, G, STATE8, 1, false>(t, f, key, i);
        }
    }
    // The last workgroup to come here counts the step: all have read the count.  Its
    // tickets are in two levels, as one address takes an addition in 13 ns: 2048
    // workgroups on one counter took 26 us.
    if (args.last && threadIdx.x == 0) {
        const int group = blockIdx.x % TICKET_GROUPS, groups = min(TICKET_GROUPS, (int)gridDim.x);
        const int mine = ((int)gridDim.x - group + TICKET_GROUPS - 1) / TICKET_GROUPS;
        uint32_t *root = reinterpret_cast<uint32_t *>(args.steps + 1);
        uint32_t *ticket = reinterpret_cast<uint32_t *>(args.steps) + 32 * (1 + group);
        if (atomicAdd(ticket, 1u) == (uint32_t)mine - 1u) {
            *ticket = 0;
            if (atomicAdd(root, 1u) == (uint32_t)groups - 1u) {
                *root = 0;
                args.steps[0] = (int64_t)steps;
            }
        }
    }
}

using StepKernel = void (*)(StepArgs, const int32_t *);
template <int N>
StepKernel adamw_kernel_of(int kind) {
    constexpr StepKernel kernels[8] = {
        adamw_kernel<float, float, false, N>,    adamw_kernel<uint16_t, float, false, N>,
        adamw_kernel<float, uint16_t, false, N>, adamw_kernel<uint16_t, uint16_t, false, N>,
        adamw_kernel<float, float, true, N>,     adamw_kernel<uint16_t, float, true, N>,
        adamw_kernel<float, uint16_t, true, N>,  adamw_kernel<uint16_t, uint16_t, true, N>};
    return kernels[kind];
}
StepKernel adamw_kernel_of(int kind, int blocks) {
    return blocks == 1 ? adamw_kernel_of<1>(kind) : adamw_kernel_of<STEP_BLOCKS>(kind);
}

}  // namespace

hipError_t launch_grad_norm(const fp8_grad_t *grads, int count, float max_norm, float *norm,
                            float *factor, int32_t *flag, double *parts, hipStream_t stream) {
    int used = 0, at = 0;                              // parts written, tensors read
    while (at < count) {
        NormArgs args;
        args.count = args.tiles = 0;
        args.again = used > 0;
        for (; at < count && args.count < NORM_TENSORS; ++at) {
            if (grads[at].n == 0) continue;
            args.t[args.count++] = {grads[at].grad, grads[at].n, args.tiles,
                                    grads[at].dtype == FP8_DTYPE_BF16};
            const int64_t bytes = grads[at].n * (grads[at].dtype == FP8_DTYPE_BF16 ? 2 : 4);
            args.tiles += (int)((bytes + NORM_TILE_BYTES - 1) / NORM_TILE_BYTES);
        }
        if (args.count == 0) break;
        // The first launch writes the parts that all have.
        const int grid = args.again ? std::min(used, args.tiles)
                                    : std::min(kNormParts, at < count ? kNormParts : args.tiles);
        used = std::max(used, grid);
        hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)grid), dim3(THREADS), 0, stream, args,
                           parts);
        if (hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL(grad_norm_sum_kernel, dim3(1), dim3(THREADS), 0, stream, parts, used,
                       max_norm, norm, factor, flag);
    return hipGetLastError();
}

hipError_t launch_adamw(const fp8_adamw_t &opt, const fp8_adamw_tensor_t *tensors, int count,
                        const float *grad_scale, const int32_t *noop, hipStream_t stream) {
    const auto kind_of = [](const fp8_adamw_tensor_t &t) {
        return (t.param_dtype == FP8_DTYPE_BF16 ? 1 : 0) | (t.grad_dtype == FP8_DTYPE_BF16 ? 2 : 0) |
               (t.m_scale ? 4 : 0);
    };
    int cus = 0;
    if (hipError_t e = current_cu_count(&cus)) return e;
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i)
        tiles += (tensors[i].n + step_tile(STEP_BLOCKS) - 1) / step_tile(STEP_BLOCKS);
    const int blocks = tiles <= cus ? 1 : STEP_BLOCKS;
    StepArgs args;
    args.lr = opt.lr;
    args.grad_scale = grad_scale;
    args.steps = opt.state;
    args.beta1 = opt.beta1;
    args.beta2 = opt.beta2;
    args.b1 = (float)opt.beta1;
    args.c1 = (float)(1.0 - opt.beta1);
    args.b2 = (float)opt.beta2;
    args.c2 = (float)(1.0 - opt.beta2);
    args.eps = (float)opt.eps;
    args.seed_lo = (uint32_t)opt.seed;
    args.seed_hi = (uint32_t)(opt.seed >> 32);
    // A launch holds tensors of one combination of types; the last one counts the step.
    int kinds[8] = {};
    for (int i = 0; i < count; ++i)
        if (tensors[i].n > 0) ++kinds[kind_of(tensors[i])];
    int left = 0;
    for (int kind = 0; kind < 8; ++kind) left += kinds[kind];
    for (int kind = 0; kind < 8; ++kind) {
        if (kinds[kind] == 0 && !(left == 0 && kind == 0)) continue;
        int at = 0;
        do {
            args.count = args.tiles = 0;
            for (; at < count && args.count < STEP_TENSORS; ++at) {
                const fp8_adamw_tensor_t &t = tensors[at];
                if (t.n == 0 || kind_of(t) != kind) continue;
                args.t[args.count++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n,
                                        args.tiles, t.weight_decay, at};
                args.tiles += (int)((t.n + step_tile(blocks) - 1) / step_tile(blocks));
            }
            kinds[kind] -= args.count;
            left -= args.count;
            args.last = left == 0;
            const int grid = std::max(1, std::min(args.tiles, 16 * cus));
            hipLaunchKernelGGL(adamw_kernel_of(kind, blocks), dim3((unsigned)grid), dim3(THREADS),
                               0, stream, args, noop);
            if (hipError_t e = hipGetLastError()) return e;
        } while (kinds[kind] > 0);
        if (left == 0) break;
    }
    return hipSuccess;
}

}  // namespace fp8dsl
