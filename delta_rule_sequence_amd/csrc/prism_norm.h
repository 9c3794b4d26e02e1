// prism_norm.h - root-mean-square norm of rows, with residual, gate and 8-bit output, and its backward (gfx950).
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w silu(z)
//   with u = dy silu(z):  dw = sum_rows u h r,   dz = dy h r w silu'(z)
//   dh = r (u w - h r mean(u w h r)) + dh_in
//
// Bound by its bytes.
#pragma once
#include "prism_ssm_args.h"
#include "prism_tile.h"

namespace prism {
namespace norm {

constexpr int kBlock = 128;        // values that share one scale of the 8-bit output
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
// The largest |value| over the wave; a NaN's pattern lies above infinity's, so it wins.
__device__ __forceinline__ unsigned wave_max_bits(unsigned v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// The scale of a block from its largest |y| (bits).
__device__ __forceinline__ float block_scale(unsigned amax) {
  return amax == 0u ? 1.f : __builtin_bit_cast(float, amax) / kE4m3Max;
}
// y / scale rounded to e4m3 (to nearest even, at most 448); NaN for a block whose scale is not finite.
__device__ __forceinline__ unsigned char to_e4m3(float y, float scale) {
  if (!(scale < __builtin_inff())) return 0x7f;
  const float v = fminf(fmaxf(y / scale, -kE4m3Max), kE4m3Max);
  return (unsigned char)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

__device__ __forceinline__ float block_sum(float v, float* part) {  // 256 threads
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) part[wave_id()] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// One workgroup per row, in 128-value blocks of one wave each.
template <class T>
__global__ __launch_bounds__(256) void fwd_kernel(NormArgs a) {
  __shared__ float part[4];
  const size_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.xs;
  const T* res = a.residual != nullptr ? reinterpret_cast<const T*>(a.residual) + row * a.D : nullptr;
  const T* z = a.gate != nullptr ? reinterpret_cast<const T*>(a.gate) + row * a.gs : nullptr;
  float s = 0.f;
  for (int c = threadIdx.x; c < a.D; c += 256) {
    const float h = (float)x[c] + (res != nullptr ? (float)res[c] : 0.f);
    s += h * h;
  }
  const float r = 1.f / sqrtf(block_sum(s, part) / a.D + a.eps);
  const int nb = (a.D + kBlock - 1) / kBlock;
  for (int blk = wave_id(); blk < nb; blk += 4) {
    float y[2];
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = blk * kBlock + k * 64 + lane_id();
      y[k] = 0.f;
      if (c < a.D) {
        const float h = (float)x[c] + (res != nullptr ? (float)res[c] : 0.f);
        y[k] = h * r * (a.w != nullptr ? a.w[c] : 1.f);
        if (z != nullptr) y[k] *= (float)z[c] * sigmoid_f((float)z[c]);
        if (a.h != nullptr) reinterpret_cast<T*>(a.h)[row * a.D + c] = (T)h;
      }
      m = max(m, abs_bits(y[k]));
    }
    float scale = 1.f;
    if (a.scales != nullptr) {
      scale = block_scale(wave_max_bits(m));
      if (lane_id() == 0) a.scales[row * nb + blk] = scale;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = blk * kBlock + k * 64 + lane_id();
      if (c >= a.D) continue;
      if (a.scales != nullptr) reinterpret_cast<unsigned char*>(a.y)[row * a.D + c] = to_e4m3(y[k], scale);
      else reinterpret_cast<T*>(a.y)[row * a.D + c] = (T)y[k];
    }
  }
}

// Workgroup k takes rows k, k + nblk, ...; its shares of dweight stay in part[k].
template <class T>
__global__ __launch_bounds__(256) void bwd_kernel(NormArgs a) {
  __shared__ float part[4];
  float* dw = a.dw != nullptr ? a.part + (size_t)blockIdx.x * a.D : nullptr;
  for (int row = blockIdx.x; row < a.rows; row += a.nblk) {
    const T* h = reinterpret_cast<const T*>(a.x) + (size_t)row * a.xs;
    const T* dy = reinterpret_cast<const T*>(a.dy) + (size_t)row * a.D;
    const T* z = a.gate != nullptr ? reinterpret_cast<const T*>(a.gate) + (size_t)row * a.gs : nullptr;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float hv = (float)h[c];
      float u = (float)dy[c] * (a.w != nullptr ? a.w[c] : 1.f);
      if (z != nullptr) u *= (float)z[c] * sigmoid_f((float)z[c]);
      s += hv * hv;
      q += u * hv;
    }
    s = block_sum(s, part);
    const float r = 1.f / sqrtf(s / a.D + a.eps);
    const float mean = block_sum(q, part) * r / a.D;
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const size_t at = (size_t)row * a.D + c;
      const float hat = (float)h[c] * r, w = a.w != nullptr ? a.w[c] : 1.f;
      float u = (float)dy[c];
      if (z != nullptr) {
        const float zv = (float)z[c], sg = sigmoid_f(zv);
        reinterpret_cast<T*>(a.dgate)[at] = (T)(u * hat * w * (sg * (1.f + zv * (1.f - sg))));
        u *= zv * sg;
      }
      float dh = r * (u * w - hat * mean);
      if (a.dh_in != nullptr) dh += (float)reinterpret_cast<const T*>(a.dh_in)[at];
      reinterpret_cast<T*>(a.h)[at] = (T)dh;
      if (dw != nullptr) dw[c] = (row == (int)blockIdx.x ? 0.f : dw[c]) + u * hat;
    }
  }
}

// dweight from the workgroups' shares, in float64 and a fixed order.  Grid (columns / 64), four waves.
__global__ __launch_bounds__(256) void wsum_kernel(NormArgs a) {
  __shared__ double part[4][64];
  const int c = blockIdx.x * 64 + threadIdx.x % 64, q = threadIdx.x / 64;
  double s = 0.0;
  if (c < a.D)
    for (int k = q; k < a.nblk; k += 4) s += (double)a.part[(size_t)k * a.D + c];
  part[q][threadIdx.x % 64] = s;
  __syncthreads();
  if (q == 0 && c < a.D) a.dw[c] = (float)((part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]));
}

}  // namespace norm
}  // namespace prism
