// prism_e4m3.h - the scale of a block of values held as e4m3 bytes (the norm's 8-bit output, the paged cache).
#pragma once
#include <hip/hip_runtime.h>

namespace prism {
namespace norm {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// Below this a block counts as all zero: 448 / amax would overflow soon after.
constexpr float kTiny = 0x1p-100f;
// The scale of a block from its largest |y| (bits), and the factor that takes y to the bytes' range: NaN for a block
// with a non-finite value, which makes all its bytes NaN.  |y| factor <= 448 (1 + 2^-22) rounds to 448 at most.
__device__ __forceinline__ float block_scale(unsigned amax, float* factor) {
  const float m = __builtin_bit_cast(float, amax);
  if (m < kTiny) {
    *factor = 0.f;
    return 1.f;
  }
  *factor = m < __builtin_inff() ? kE4m3Max / m : __builtin_nanf("");
  return m / kE4m3Max;
}

}  // namespace norm
}  // namespace prism
