// bf16 values as the bits of their 16-bit words, two to a 32-bit word.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8dsl {

// The lower and the upper value of a word: a bf16's bits are the upper half of an fp32's.
__device__ __forceinline__ float bf16_lo(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); }

// f rounded to nearest even; a NaN becomes 0x7FC0.
__device__ __forceinline__ uint32_t bf16_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return (f != f) ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

}  // namespace fp8dsl
