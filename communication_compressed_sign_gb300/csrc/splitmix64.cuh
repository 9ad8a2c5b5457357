// splitmix64.cuh -- SplitMix64 (Steele, Lea and Flood 2014) as a counter-based
// generator: output number k (from 0) of the generator that starts at `seed`.
#pragma once

#include <stdint.h>

namespace lc {

constexpr uint64_t kSplitMix64Step = 0x9e3779b97f4a7c15ull;  // the state's increment (gamma)

// The output for a state: the state is seed + (k + 1) * kSplitMix64Step.
__host__ __device__ __forceinline__ uint64_t splitmix64_mix(uint64_t z)
{
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
    return z ^ (z >> 31);
}

__host__ __device__ __forceinline__ uint64_t splitmix64(uint64_t seed, uint64_t k)
{
    return splitmix64_mix(seed + (k + 1ull) * kSplitMix64Step);
}

}  // namespace lc
