// The gradients' norm and the AdamW step over many tensors.
//
// The tensors of a launch are kernel arguments (by value, within the 4 KB that a
// launch takes), so a call reads no host memory later and can be captured; their
// tiles are one list, which the workgroups share evenly.
#include "adamw.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "dropout.h"
#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;

__device__ __forceinline__ uint32_t bf16_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return (f != f) ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Four values of a tensor from element i on, `left` of them (1 .. 4) there.
template <typename T>
struct Four;
template <>
struct Four<float> {
    static __device__ __forceinline__ void load(const void *p, int64_t i, int left, float (&o)[4]) {
        const float *at = static_cast<const float *>(p) + i;
        if (left >= 4) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(at);
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
            *reinterpret_cast<u32x4 *>(at) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                   __float_as_uint(v[2]), __float_as_uint(v[3])};
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
            const u32x2 v = *reinterpret_cast<const u32x2 *>(at);
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
            *reinterpret_cast<u32x2 *>(at) = u32x2{bits[0] | (bits[1] << 16),
                                                   bits[2] | (bits[3] << 16)};
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
        if (left >= 4) return *reinterpret_cast<const uint32_t *>(at);
        uint32_t v = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < left) v |= (uint32_t)at[k] << (8 * k);
        return v;
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, int left, uint32_t v) {
        uint8_t *at = static_cast<uint8_t *>(p) + i;
        if (left >= 4) {
            *reinterpret_cast<uint32_t *>(at) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < left) at[k] = (uint8_t)(v >> (8 * k));
        }
    }
};

// ---- the norm ----------------------------------------------------------------

// Values of a tile: a lane takes NORM_LANE of them, four at a time.
constexpr int NORM_STEPS = 8;
constexpr int NORM_TILE = THREADS * 4 * NORM_STEPS;
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

template <typename T>
__device__ __forceinline__ void add_squares(const NormTensor &t, int64_t i0, double (&sum)[4]) {
    float v[NORM_STEPS][4];
#pragma unroll
    for (int s = 0; s < NORM_STEPS; ++s) {
        const int64_t i = i0 + (int64_t)s * THREADS * 4 + 4 * threadIdx.x;
        const int left = (int)min((int64_t)4, t.n - i);
        if (left > 0) {
            Four<T>::load(t.grad, i, left, v[s]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[s][k] = 0.0f;
        }
    }
#pragma unroll
    for (int s = 0; s < NORM_STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = fma((double)v[s][k], (double)v[s][k], sum[k]);
}

__global__ __launch_bounds__(THREADS) void grad_norm_kernel(const NormArgs args,
                                                            double *__restrict__ parts) {
    __shared__ double waves[WAVES];
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    for (int tile = blockIdx.x; tile < args.tiles; tile += gridDim.x) {
        const NormTensor &t = args.t[tensor_of(args, tile)];
        const int64_t i0 = (int64_t)(tile - t.first) * NORM_TILE;
        if (t.bf16) add_squares<uint16_t>(t, i0, sum);
        else add_squares<float>(t, i0, sum);
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
constexpr int STEP_BLOCKS = 2;                         // blocks of 256 a wave takes at once
constexpr int STEP_TILE = WAVES * STEP_BLOCKS * BLOCK;
constexpr int STEP_TENSORS = 48;
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
    int32_t types;           // 1: bf16 param, 2: bf16 grad, 4: states in 8 bits
};
struct StepArgs {
    int count, tiles;
    int base;                // tensors of earlier launches
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

struct Factors {
    float grad, step, root, lr;
};

// Bits of the power of two that scales a block whose largest finite magnitude is
// `most` (bits): the least, 2^-126 or more, that keeps it within 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_bits(uint32_t most) {
    const int e = (int)((most + 0x1FFFFFu) >> 23);      // one more beyond 1.75
    return (uint32_t)max(e - 8, 1) << 23;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m, 64));
    return v;
}

// The E4M3 code of x (|x| <= 448, or not finite), u a 16-bit number.  An fp32 value
// from 2^-6 on has 20 bits below the code's three: adding u there and cutting rounds
// up with the probability of the part cut.  Below 2^-6 the codes are as far
// apart as from 2^-6 to 2^-5: the value is moved there.
template <bool KEEP>
__device__ __forceinline__ uint32_t code_of(float x, uint32_t u) {
    const uint32_t bits = __float_as_uint(x), mag = bits & 0x7FFFFFFFu;
    const float ax = __uint_as_float(mag);
    const bool low = ax < 0x1p-6f;
    const uint32_t y = low ? __float_as_uint(ax + 0x1p-6f) : mag;
    uint32_t code = ((y + (u << 4)) >> 20) - (low ? 968u : 960u);
    if constexpr (KEEP) code = code == 0u && mag != 0u ? 1u : code;
    code |= (bits >> 24) & 0x80u;
    return mag >= 0x7F800000u ? 0x7Fu : code;
}

// One block of 256 values of a tensor: a lane's four begin at element i.
template <typename P, typename G, bool STATE8>
struct Block {
    float p[4], g[4], m[4], v[4];
    uint32_t mc, vc;
    float ms, vs;

    __device__ __forceinline__ void load(const StepTensor &t, int64_t i, int left) {
        if (left <= 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = g[k] = m[k] = v[k] = 0.0f;
            mc = vc = 0;
            ms = vs = 0.0f;
            return;
        }
        Four<P>::load(t.param, i, left, p);
        Four<G>::load(t.grad, i, left, g);
        if constexpr (STATE8) {
            mc = Four<uint8_t>::load(t.m, i, left);
            vc = Four<uint8_t>::load(t.v, i, left);
            ms = t.m_scale[i / BLOCK];
            vs = t.v_scale[i / BLOCK];
        } else {
            Four<float>::load(t.m, i, left, m);
            Four<float>::load(t.v, i, left, v);
        }
    }

    __device__ __forceinline__ void step(const StepArgs &args, const StepTensor &t, int item,
                                         uint64_t steps, const Factors &f, float decay, int64_t i,
                                         int left) {
#pragma clang fp contract(off)
        if constexpr (STATE8) {
            m[0] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 0) * ms;
            m[1] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 1) * ms;
            m[2] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 2) * ms;
            m[3] = __builtin_amdgcn_cvt_f32_fp8((int)mc, 3) * ms;
            v[0] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 0) * vs;
            v[1] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 1) * vs;
            v[2] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 2) * vs;
            v[3] = __builtin_amdgcn_cvt_f32_fp8((int)vc, 3) * vs;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gk = g[k] * f.grad;
            m[k] = m[k] * args.b1 + gk * args.c1;
            v[k] = v[k] * args.b2 + (gk * args.c2) * gk;
            p[k] = p[k] * decay - (m[k] * f.step) / (sqrtf(v[k]) * f.root + args.eps);
        }
        const DropoutKey key(args.seed_lo, args.seed_hi, steps);
        if constexpr (STATE8) {
            uint32_t most_m = 0, most_v = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = __float_as_uint(m[k]) & 0x7FFFFFFFu;
                const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
                most_m = max(most_m, a < 0x7F800000u ? a : 0u);
                most_v = max(most_v, b < 0x7F800000u ? b : 0u);
            }
            const uint32_t sm = scale_bits(wave_max(most_m)), sv = scale_bits(wave_max(most_v));
            // 1 / 2^e: e and its negative are both exponents of normal numbers.
            const float im = __uint_as_float((254u << 23) - sm);
            const float iv = __uint_as_float((254u << 23) - sv);
            uint32_t w[4];
            dropout_words(key, ((uint64_t)(2u * (uint32_t)item) << 32) | (uint64_t)(i / 4), w);
            mc = vc = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mc |= code_of<false>(m[k] * im, w[k] & 0xFFFFu) << (8 * k);
                vc |= code_of<true>(v[k] * iv, w[k] >> 16) << (8 * k);
            }
            if (left <= 0) return;
            Four<uint8_t>::store(t.m, i, left, mc);
            Four<uint8_t>::store(t.v, i, left, vc);
            if (i % BLOCK == 0) {
                t.m_scale[i / BLOCK] = __uint_as_float(sm);
                t.v_scale[i / BLOCK] = __uint_as_float(sv);
            }
        } else {
            if (left <= 0) return;
            Four<float>::store(t.m, i, left, m);
            Four<float>::store(t.v, i, left, v);
        }
        if constexpr (std::is_same<P, float>::value) {
            Four<float>::store(t.param, i, left, p);
            if (t.copy) {
                const uint32_t bits[4] = {bf16_bits(p[0]), bf16_bits(p[1]), bf16_bits(p[2]),
                                          bf16_bits(p[3])};
                Four<uint16_t>::store(t.copy, i, left, bits);
            }
        } else {
            uint32_t w[4], bits[4];
            dropout_words(key, ((uint64_t)(2u * (uint32_t)item + 1u) << 32) | (uint64_t)(i / 8), w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t word = (i & 4) ? w[2 + k / 2] : w[k / 2];
                const uint32_t u = k & 1 ? word >> 16 : word & 0xFFFFu;
                const uint32_t b = __float_as_uint(p[k]);
                const bool finite = (b & 0x7F800000u) != 0x7F800000u;
                bits[k] = p[k] != p[k] ? 0x7FC0u : (b + (finite ? u : 0u)) >> 16;
            }
            Four<uint16_t>::store(t.param, i, left, bits);
        }
    }
};

template <typename P, typename G, bool STATE8>
__device__ __forceinline__ void step_tile(const StepArgs &args, int item, uint64_t steps,
                                          const Factors &f, int64_t i0) {
    const StepTensor &t = args.t[item];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float decay = (float)(1.0 - (double)f.lr * (double)t.weight_decay);
    Block<P, G, STATE8> b[STEP_BLOCKS];
    int64_t i[STEP_BLOCKS];
    int left[STEP_BLOCKS];
#pragma unroll
    for (int s = 0; s < STEP_BLOCKS; ++s) {
        i[s] = i0 + (wave * STEP_BLOCKS + s) * BLOCK + 4 * lane;
        left[s] = (int)max((int64_t)0, min((int64_t)4, t.n - i[s]));
        b[s].load(t, i[s], left[s]);
    }
#pragma unroll
    for (int s = 0; s < STEP_BLOCKS; ++s)
        b[s].step(args, t, args.base + item, steps, f, decay, i[s], left[s]);
}

__global__ __launch_bounds__(THREADS) void adamw_kernel(const StepArgs args,
                                                        const int32_t *__restrict__ noop) {
    if (noop != nullptr && *noop != 0) return;
    __shared__ int64_t taken;
    if (threadIdx.x == 0) taken = args.steps[0];
    __syncthreads();
    const uint64_t steps = (uint64_t)taken + 1;
    Factors f;
    f.lr = *args.lr;
    f.grad = args.grad_scale ? *args.grad_scale : 1.0f;
    f.step = (float)((double)f.lr / (1.0 - power(args.beta1, steps)));
    f.root = (float)(1.0 / sqrt(1.0 - power(args.beta2, steps)));
    for (int tile = blockIdx.x; tile < args.tiles; tile += gridDim.x) {
        const int item = tensor_of(args, tile);
        const int64_t i0 = (int64_t)(tile - args.t[item].first) * STEP_TILE;
        switch (args.t[item].types) {
            case 0: step_tile<float, float, false>(args, item, steps, f, i0); break;
            case 1: step_tile<uint16_t, float, false>(args, item, steps, f, i0); break;
            case 2: step_tile<float, uint16_t, false>(args, item, steps, f, i0); break;
            case 3: step_tile<uint16_t, uint16_t, false>(args, item, steps, f, i0); break;
            case 4: step_tile<float, float, true>(args, item, steps, f, i0); break;
            case 5: step_tile<uint16_t, float, true>(args, item, steps, f, i0); break;
            case 6: step_tile<float, uint16_t, true>(args, item, steps, f, i0); break;
            default: step_tile<uint16_t, uint16_t, true>(args, item, steps, f, i0); break;
        }
    }
    // The last workgroup to come here counts the step: all have read the count.
    if (args.last && threadIdx.x == 0) {
        unsigned long long *tickets = reinterpret_cast<unsigned long long *>(args.steps + 1);
        if (atomicAdd(tickets, 1ull) == gridDim.x - 1) {
            args.steps[0] = (int64_t)steps;
            args.steps[1] = 0;
        }
    }
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
            args.tiles += (int)((grads[at].n + NORM_TILE - 1) / NORM_TILE);
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
    int cus = 0;
    if (hipError_t e = current_cu_count(&cus)) return e;
    StepArgs args;
    args.lr = opt.lr;
    args.grad_scale = grad_scale;
    args.steps = opt.steps;
    args.beta1 = opt.beta1;
    args.beta2 = opt.beta2;
    args.b1 = (float)opt.beta1;
    args.c1 = (float)(1.0 - opt.beta1);
    args.b2 = (float)opt.beta2;
    args.c2 = (float)(1.0 - opt.beta2);
    args.eps = (float)opt.eps;
    args.seed_lo = (uint32_t)opt.seed;
    args.seed_hi = (uint32_t)(opt.seed >> 32);
    args.base = 0;
    do {
        args.count = std::min(STEP_TENSORS, count - args.base);
        args.last = args.base + args.count == count;
        args.tiles = 0;
        for (int i = 0; i < args.count; ++i) {
            const fp8_adamw_tensor_t &t = tensors[args.base + i];
            args.t[i] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n, args.tiles,
                         t.weight_decay,
                         (t.param_dtype == FP8_DTYPE_BF16 ? 1 : 0) |
                             (t.grad_dtype == FP8_DTYPE_BF16 ? 2 : 0) | (t.m_scale ? 4 : 0)};
            args.tiles += (int)((t.n + STEP_TILE - 1) / STEP_TILE);
        }
        const int grid = std::max(1, std::min(args.tiles, 8 * cus));
        hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)grid), dim3(THREADS), 0, stream, args, noop);
        if (hipError_t e = hipGetLastError()) return e;
        args.base += args.count;
    } while (args.base < count);
    return hipSuccess;
}

}  // namespace fp8dsl
