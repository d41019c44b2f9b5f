// The angle of a position, for the rotary kernels.  Host code too, so that its arithmetic is tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define LLA_ANGLE_FN __host__ __device__ __forceinline__
#else
#define LLA_ANGLE_FN inline
#endif

namespace lla {
namespace rotary {

// position * turns 2^-64 turns, modulo a turn, in units of 2^-32 of one: the product's upper half.  Unsigned, since the product
// wraps from position 4 on at the fastest pair, and only unsigned products may (the two's complement bits are the same).
LLA_ANGLE_FN int turn_of(long long position, long long turns) {
    const unsigned long long t = static_cast<unsigned long long>(position) * static_cast<unsigned long long>(turns);
    return static_cast<int>(static_cast<unsigned>(t >> 32));
}

}  // namespace rotary
}  // namespace lla
