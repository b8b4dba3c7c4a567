// The fixed-point scale of the samplers' masses.
#pragma once

#include <stdint.h>

namespace llb {

// A token's mass is its exponential (1 for the most likely token) times 2^b,
// rounded: b = 46, less where V masses of 2^46 would not fit 64 bits.  At V =
// 2^18 their sum is 2^64 exactly, so b is the most for which V * 2^b < 2^64.  A
// power of two, so that u * (kept mass) stays exact on rows of equal logits.
__host__ __device__ constexpr int mass_bits(int V) {
    int b = 46;
    while (b > 0 && static_cast<uint64_t>(V) > (~0ull >> b)) --b;
    return b;
}

}  // namespace llb
