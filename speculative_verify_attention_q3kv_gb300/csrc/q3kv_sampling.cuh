// Device helpers shared by the acceptance kernels: the ordering of (value,
// index) candidates, logit loads and the counter-based noise stream.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace q3kv {

// a beats b: larger value, or the same value at a lower index
__device__ __forceinline__ bool beats(float av, int ai, float bv, int bi) {
    return av > bv || (av == bv && ai < bi);
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// State of output number row * 2^32 + x of the counter-based SplitMix64 stream seeded with
// `seed`; the next outputs' states are kNoiseStep apart.
constexpr uint64_t kNoiseStep = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ uint64_t noise_state(uint64_t seed, uint32_t row, uint32_t x) {
    return seed + ((((uint64_t)row << 32) + x) + 1ull) * kNoiseStep;
}
// z >> 41 of the output z of a state (the last step, z ^= z >> 31, leaves those bits as they
// are), as a float: 23 bits under the exponent of 2^23.
__device__ __forceinline__ float noise_level(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return __uint_as_float((uint32_t)(z >> 41) | 0x4B000000u) - 8388608.0f;
}

// U = ((z >> 41) + 0.5) / 2^23.
__device__ __forceinline__ float noise_uniform(uint64_t seed, uint32_t row, uint32_t x) {
    return (noise_level(noise_state(seed, row, x)) + 0.5f) * (1.0f / 8388608.0f);
}

}  // namespace q3kv
