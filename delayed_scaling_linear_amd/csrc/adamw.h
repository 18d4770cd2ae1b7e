// Launchers of the optimizer kernels, and the sizes the C-ABI layer checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8dsl.h"

namespace fp8dsl {

// Values of one tensor at most: the random numbers' group fits 32 bits.
constexpr int64_t kTensorMost = (int64_t)1 << 34;
// Partial sums of the norm, one per workgroup at most.
constexpr int kNormParts = 2048;

hipError_t launch_grad_norm(const fp8_grad_t *grads, int count, float max_norm, float *norm,
                            float *factor, int32_t *flag, double *parts, hipStream_t stream);

hipError_t launch_adamw(const fp8_adamw_t &opt, const fp8_adamw_tensor_t *tensors, int count,
                        const float *grad_scale, const int32_t *noop, hipStream_t stream);

}  // namespace fp8dsl
