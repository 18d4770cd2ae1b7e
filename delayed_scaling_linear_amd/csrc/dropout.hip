// Elementwise dropout with an optional residual:
//
//   y[r, c] = residual[r, c] + (kept(r, c) ? f * x[r, c] : +0)
//
// in fp32 (the product and the sum each rounded), rounded once to the type of
// x.  A dropped element is +0 whatever x holds there, infinities and NaNs
// included.  The gradient with respect to x is the same call on the output's
// gradient, without the residual.
//
// Memory bound: 2 or 3 passes of the tensor and 1.75 quarter-rate multiplies
// per element.  A lane takes the 8 columns of one Philox call (16 bytes of
// bf16, 32 of fp32); a workgroup covers TX such groups of TY rows at a time
// (TX a power of two that covers the row or 256), so no lane divides, and
// each lane has ROWS_PER_LANE rows' loads in flight.  A lane stores only where
// it alone has read, so y may be x or the residual.  Measured: bf16 [8192, 2048]
// 12.7 us a call, 5.3 TB/s of the 67 MB it reads and writes (a copy of as much:
// 5.1 to 5.4; with non-temporal loads 14.6); fp32 [1037, 1160] with a residual
// 4.7 us on the GPU, 7.1 a call.
#include "dropout.h"
#include "bf16.h"
#include "fp8dsl_internal.h"

namespace fp8dsl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;
constexpr int ROWS_PER_LANE = 4;

// res + (keep ? f * x : 0), the product and the sum each rounded.
__device__ __forceinline__ float drop_add(float x, bool keep, float f, float res, bool add) {
#pragma clang fp contract(off)
    const float t = keep ? x * f : 0.0f;
    return add ? res + t : t;
}

template <int SRC>
__global__ __launch_bounds__(THREADS) void dropout_kernel(
    const void *xv, int64_t ldx, const void *resv, int64_t ldres, void *yv, int64_t ldy,
    int64_t rows, int64_t groups, int tx_log2, DropoutArgs drop) {
    constexpr int V = SRC == FP8_DTYPE_BF16 ? 1 : 2;       // 16-byte pieces per group
    const int tx = 1 << tx_log2, ty = THREADS >> tx_log2;
    const int64_t gcol = (int64_t)blockIdx.y * tx + (threadIdx.x & (tx - 1));
    const int64_t row0 = (int64_t)blockIdx.x * ty * ROWS_PER_LANE + (threadIdx.x >> tx_log2);
    if (gcol >= groups) return;
    const DropoutKey key(drop.rng);
    constexpr int64_t EB = SRC == FP8_DTYPE_BF16 ? 2 : 4;
    const char *x = static_cast<const char *>(xv) + gcol * 8 * EB;
    const char *res = static_cast<const char *>(resv) + gcol * 8 * EB;
    char *y = static_cast<char *>(yv) + gcol * 8 * EB;
    const bool add = resv != nullptr;

    u32x4 xs[ROWS_PER_LANE][V], rs[ROWS_PER_LANE][V];
#pragma unroll
    for (int i = 0; i < ROWS_PER_LANE; ++i) {
        const int64_t r = row0 + (int64_t)i * ty;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xs[i][v] = rs[i][v] = u32x4{0u, 0u, 0u, 0u};
            if (r < rows) {
                xs[i][v] = *reinterpret_cast<const u32x4 *>(x + r * ldx * EB + 16 * v);
                if (add) rs[i][v] = *reinterpret_cast<const u32x4 *>(res + r * ldres * EB + 16 * v);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS_PER_LANE; ++i) {
        const int64_t r = row0 + (int64_t)i * ty;
        if (r >= rows) return;
        uint32_t w[4];
        dropout_words(key, (uint64_t)(r * groups + gcol), w);
        u32x4 out[V];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool k0 = (w[k] & 0xFFFFu) >= drop.threshold, k1 = (w[k] >> 16) >= drop.threshold;
            if constexpr (SRC == FP8_DTYPE_BF16) {
                const uint32_t a = xs[i][0][k], b = rs[i][0][k];
                const float lo = drop_add(__uint_as_float(a << 16), k0, drop.factor,
                                          __uint_as_float(b << 16), add);
                const float hi = drop_add(__uint_as_float(a & 0xFFFF0000u), k1, drop.factor,
                                          __uint_as_float(b & 0xFFFF0000u), add);
                out[0][k] = bf16_bits(lo) | (bf16_bits(hi) << 16);
            } else {
                const int v = k >> 1, at = 2 * (k & 1);
                out[v][at] = __float_as_uint(drop_add(__uint_as_float(xs[i][v][at]), k0,
                                                      drop.factor, __uint_as_float(rs[i][v][at]),
                                                      add));
                out[v][at + 1] = __float_as_uint(
                    drop_add(__uint_as_float(xs[i][v][at + 1]), k1, drop.factor,
                             __uint_as_float(rs[i][v][at + 1]), add));
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            *reinterpret_cast<u32x4 *>(y + r * ldy * EB + 16 * v) = out[v];
    }
}

}  // namespace

hipError_t launch_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldres, void *y,
                          int64_t ldy, int dtype, int64_t rows, int64_t cols,
                          const DropoutArgs &drop, hipStream_t stream) {
    const int64_t groups = cols / 8;
    int tx_log2 = 3;
    while (tx_log2 < 8 && (int64_t(1) << tx_log2) < groups) ++tx_log2;
    const int64_t tx = int64_t(1) << tx_log2, step = (THREADS >> tx_log2) * ROWS_PER_LANE;
    const dim3 grid((unsigned)((rows + step - 1) / step), (unsigned)((groups + tx - 1) / tx));
    if (dtype == FP8_DTYPE_BF16)
        hipLaunchKernelGGL(dropout_kernel<FP8_DTYPE_BF16>, grid, dim3(THREADS), 0, stream, x, ldx,
                           residual, ldres, y, ldy, rows, groups, tx_log2, drop);
    else
        hipLaunchKernelGGL(dropout_kernel<FP8_DTYPE_FP32>, grid, dim3(THREADS), 0, stream, x, ldx,
                           residual, ldres, y, ldy, rows, groups, tx_log2, drop);
    return hipGetLastError();
}

}  // namespace fp8dsl
