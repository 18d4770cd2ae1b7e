// Dropout from a counter-based generator, shared by the kernels that apply
// it (the elementwise dropout, the dropout in front of a cast, and the
// low-rank adapters' input).  No mask is ever stored: every kernel derives
// the elements it keeps from the element's position alone, so the forward
// and the backward agree however their work is split.
//
// Generator: Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011, whose tables give 7 as the
// fewest rounds that pass BigCrush).  One call yields four 32-bit words, here
// eight 16-bit numbers, for the eight consecutive columns of group
// e = (row * cols + col) / 8; the counter is (e, offset), the key the seed.
// The words cost 14 quarter-rate 32 x 32 -> 64 bit multiplies per eight
// elements; 7 instead of 10 rounds and 16 instead of 32 bits per element keep
// that below the time the elements' memory traffic takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8dsl {

// A dropout's arguments as the kernels take them.  Element kept where its
// 16-bit number is >= threshold (0 .. 65535); factor = 65536 / (65536 -
// threshold), rounded once to fp32, is the reciprocal of the exact keep rate.
struct DropoutArgs {
    const int64_t *rng;      // device {seed, offset}, or null: nothing is dropped
    uint32_t threshold;
    float factor;
};

// The generator's key and stream, read once per kernel (wave-uniform).
struct DropoutKey {
    uint32_t seed_lo, seed_hi, off_lo, off_hi;
    // used false: no dropout, rng is not read.
    __device__ __forceinline__ explicit DropoutKey(const int64_t *rng, bool used = true) {
        const uint64_t s = used ? (uint64_t)rng[0] : 0, o = used ? (uint64_t)rng[1] : 0;
        seed_lo = (uint32_t)s;
        seed_hi = (uint32_t)(s >> 32);
        off_lo = (uint32_t)o;
        off_hi = (uint32_t)(o >> 32);
    }
};

// The eight 16-bit numbers of group e: element i in half i % 2 of word i / 2.
__device__ __forceinline__ void dropout_words(const DropoutKey &key, uint64_t e, uint32_t w[4]) {
    uint32_t c0 = (uint32_t)e, c1 = (uint32_t)(e >> 32), c2 = key.off_lo, c3 = key.off_hi;
    uint32_t k0 = key.seed_lo, k1 = key.seed_hi;
#pragma unroll
    for (int r = 0; r < 7; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// Bit masks of the two kept 16-bit halves of word w.
__device__ __forceinline__ uint32_t dropout_keep2(uint32_t w, uint32_t threshold) {
    return ((w & 0xFFFFu) >= threshold ? 0x0000FFFFu : 0u) |
           ((w >> 16) >= threshold ? 0xFFFF0000u : 0u);
}

}  // namespace fp8dsl
