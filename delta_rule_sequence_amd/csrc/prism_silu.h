// prism_silu.h - sigmoid of the gates and activations of the state space layer.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

namespace prism {

// 1 / (1 + e^-z) for tensors of type T, from the hardware's 2^t and reciprocal (1 ulp each).
//   bfloat16: t = -z log2(e) is rounded, so the error grows to |z| + 5 half steps of 2^-24, 2^-17 at |z| = 80, where the tensor's
//   own rounding is 2^-8.  (Convolution of 8 x 2048 x 1792: 23.5 us and backward 46.2, with float's form 26.6 and 48.9.)
//   float: what t's rounding and log2(e)'s left out comes in as a factor, 7 half steps at any z.  (16 x 4800 x 160: 17.0 us with
//   bfloat16's form, 17.7 with this, 23.3 with the library's exponential and a division; 8 x 2048 x 1792: 42, 42, 44.5.)
template <class T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (std::is_same<T, float>::value) {
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float t = -z * kLog2e;
    const float left = fmaf(-z, kLog2eLow, fmaf(-z, kLog2e, -t));
    const float f = fmaf(left, kLn2, 1.f);
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t) * (fabsf(t) < 200.f ? f : 1.f));  // past 2^200 an infinity or 0
  } else {
    return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  }
}

}  // namespace prism
