// prism_norm.h - root-mean-square norm of rows, with residual, gate and 8-bit output, and its backward (gfx950).
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w silu(z)
//   with u = dy silu(z):  dw = sum_rows u h r,   dz = dy h r w silu'(z)
//   dh = r (u w - h r mean(u w h r)) + dh_in
//
// Bound by its bytes.  A row of up to 32768 bytes stays in the registers of a group of lanes and is read once.  Measured
// (a copy of 1 GiB makes 5.2 TB/s): 16384 x 1536 bfloat16 with residual, 8-bit output 33 us, 4.9 TB/s; 131072 x 64
// gated 10.6 us, 4.7; backward of 16384 x 768 with a residual's gradient 20 us and 4 for dw, 4.3 TB/s; rows of odd
// length, which start anywhere: backward of 4924 x 843, gated, 26 us.
#pragma once
#include "prism_silu.h"
#include "prism_ssm_args.h"
#include "prism_tile.h"

namespace prism {
namespace norm {

constexpr int kBlock = 128;        // values that share one scale of the 8-bit output
constexpr float kE4m3Max = 448.f;

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

__device__ __forceinline__ float block_sum(float v, float* part) {  // 256 threads
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) part[wave_id()] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__device__ __forceinline__ size_t block_id() { return (size_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Longer rows: one workgroup per row, read twice, in 128-value blocks of one wave each.
template <class T>
__global__ __launch_bounds__(256) void fwd_long_kernel(NormArgs a) {
  __shared__ float part[4];
  const size_t row = block_id();
  if (row >= (size_t)a.rows) return;
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
        if (z != nullptr) y[k] *= (float)z[c] * sigmoid<float>((float)z[c]);
        if (a.h != nullptr) reinterpret_cast<T*>(a.h)[row * a.D + c] = (T)h;
      }
      m = max(m, abs_bits(y[k]));
    }
    float factor = 1.f;
    if (a.scales != nullptr) {
      const float scale = block_scale(wave_max_bits(m), &factor);
      if (lane_id() == 0) a.scales[row * nb + blk] = scale;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = blk * kBlock + k * 64 + lane_id();
      if (c >= a.D) continue;
      if (a.scales != nullptr) reinterpret_cast<unsigned char*>(a.y)[row * a.D + c] =
          (unsigned char)(__builtin_amdgcn_cvt_pk_fp8_f32(y[k] * factor, 0.f, 0, false) & 0xff);
      else reinterpret_cast<T*>(a.y)[row * a.D + c] = (T)y[k];
    }
  }
}

// Longer rows: workgroup k takes rows k, k + nblk, ...; its shares of dweight stay in part[k].
template <class T>
__global__ __launch_bounds__(256) void bwd_long_kernel(NormArgs a) {
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
      if (z != nullptr) u *= (float)z[c] * sigmoid<float>((float)z[c]);
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
        const float zv = (float)z[c], sg = sigmoid<float>(zv);
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

// ---- rows of up to 32768 bytes ------------------------------------------------------------------------
// A row lies in the registers of TPR lanes (a part of a wave, a wave or the workgroup), NV 16-byte pieces per lane, and
// is read once: statistics by lane exchanges, then the outputs from the same registers.  Piece k of lane j is number
// k TPR + j of the row, so a 128-value block of the 8-bit output is 128 / V neighbouring lanes.
// Rows may start anywhere: 16-byte accesses need no more than the alignment of their elements here.
template <class T> struct Piece {
  static constexpr int V = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
// The piece at p, of which n values belong to the row (the others, and all for n <= 0, are 0 and not touched).
template <class T>
__device__ __forceinline__ typename Piece<T>::vec load_piece(const T* p, int n) {
  if (n >= Piece<T>::V) return *reinterpret_cast<const typename Piece<T>::vec*>(p);
  typename Piece<T>::vec v = (typename Piece<T>::vec)(0);
#pragma unroll
  for (int e = 0; e < Piece<T>::V; ++e)
    if (e < n) v[e] = p[e];
  return v;
}
template <class T>
__device__ __forceinline__ void store_piece(T* p, const typename Piece<T>::vec& v, int n) {
  if (n >= Piece<T>::V) {
    *reinterpret_cast<typename Piece<T>::vec*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < Piece<T>::V; ++e)
    if (e < n) p[e] = v[e];
}
// V weights from column c on (ones without a weight; 0 past the row).
template <int V>
__device__ __forceinline__ void load_weight(float (&w)[V], const float* p, int c, int n) {
  typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
  if (p != nullptr && n >= V) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const f4 v = *reinterpret_cast<const f4*>(p + c + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[k + e] = v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = e < n ? (p != nullptr ? p[c + e] : 1.f) : 0.f;
  }
}

template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < W; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Lanes of a workgroup whose rows have TPR lanes each.
constexpr int row_threads(int TPR) { return TPR > 256 ? TPR : 256; }
// Sum over a row's lanes; buf (TPR / 64 floats) joins the waves of a row that fills the workgroup.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = lanes_sum<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR >= 256) {
    if (lane_id() == 0) buf[wave_id()] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int k = 0; k < TPR / 64; k += 4) v += (buf[k] + buf[k + 1]) + (buf[k + 2] + buf[k + 3]);
  }
  return v;
}

template <class T, int TPR, int NV>
__global__ __launch_bounds__(row_threads(TPR)) void fwd_row_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, BL = kBlock / V < TPR ? kBlock / V : TPR;  // lanes of a scale block
  typedef typename Piece<T>::vec vec;
  __shared__ float buf[TPR < 256 ? 1 : TPR / 64];
  const int j = threadIdx.x % TPR;
  const size_t row = block_id() * (row_threads(TPR) / TPR) + threadIdx.x / TPR;
  if (row >= (size_t)a.rows) return;  // whole workgroups only where a row fills one
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.xs;
  const T* z = a.gate != nullptr ? reinterpret_cast<const T*>(a.gate) + row * a.gs : nullptr;
  float h[NV][V];
  vec zv[NV];
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + j) * V;
    const vec xv = load_piece(x + c, a.D - c);
#pragma unroll
    for (int e = 0; e < V; ++e) h[k][e] = (float)xv[e];
    if (z != nullptr) zv[k] = load_piece(z + c, a.D - c);
  }
  if (a.residual != nullptr) {
    const T* res = reinterpret_cast<const T*>(a.residual) + row * a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + j) * V;
      const vec rv = load_piece(res + c, a.D - c);
#pragma unroll
      for (int e = 0; e < V; ++e) h[k][e] += (float)rv[e];
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) s += h[k][e] * h[k][e];
  const float r = 1.f / sqrtf(row_sum<TPR>(s, buf) / a.D + a.eps);
  const int nb = (a.D + kBlock - 1) / kBlock;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + j) * V;
    const int left = a.D - c;
    const bool in = left > 0;
    const size_t at = row * a.D + c;
    if (a.h != nullptr) {
      vec o;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = (T)h[k][e];
      store_piece(reinterpret_cast<T*>(a.h) + at, o, left);
    }
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = h[k][e] * r;
    if (a.w != nullptr) {
      float w[V];
      load_weight<V>(w, a.w, c, left);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] *= w[e];
    }
    if (z != nullptr) {
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] *= (float)zv[k][e] * sigmoid<T>((float)zv[k][e]);
    }
    if (a.scales == nullptr) {
      vec o;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = (T)y[e];
      store_piece(reinterpret_cast<T*>(a.y) + at, o, left);
      continue;
    }
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) m = max(m, e < left ? abs_bits(y[e]) : 0u);
#pragma unroll
    for (int o = 1; o < BL; o <<= 1) {
      const unsigned u = __shfl_xor(m, o, 64);
      m = u > m ? u : m;
    }
    float factor;
    const float scale = block_scale(m, &factor);
    if (!in) continue;
    if (j % BL == 0) a.scales[row * nb + c / kBlock] = scale;
    unsigned q[V / 4];
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[e] * factor, y[e + 1] * factor, 0, false);
      q[e / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(y[e + 2] * factor, y[e + 3] * factor, p, true);
    }
    unsigned char* o = reinterpret_cast<unsigned char*>(a.y) + at;
    if (left >= V) {
      typedef unsigned any __attribute__((ext_vector_type(V / 4 > 1 ? V / 4 : 2), aligned(1)));
      typedef unsigned one __attribute__((aligned(1)));
      if constexpr (V == 8) *reinterpret_cast<any*>(o) = any{q[0], q[1]};
      else *reinterpret_cast<one*>(o) = q[0];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) o[e] = (unsigned char)(q[e / 4] >> (e % 4 * 8));
    }
  }
}

// The same for the backward: the workgroup walks rows (256 / TPR at a time) with its lanes' columns of dweight in
// registers, joins them over its row slots in LDS and leaves one share per workgroup.
// Gated bfloat16 rows of 1024 lanes form sigmoid(z) and u again for the outputs: held, with the row in 128 registers per lane,
// they went to scratch (1000 x 8200: 70 us, formed again 33; 1000 x 16384: 99 and 51; in 512 lanes of 256 registers 80 and 116).
template <class T, int TPR, int NV, bool GATE>
__global__ __launch_bounds__(row_threads(TPR)) void bwd_row_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, RPB = row_threads(TPR) / TPR;
  constexpr bool AGAIN = GATE && TPR == 1024 && V == 8;
  typedef typename Piece<T>::vec vec;
  __shared__ float buf[2][2][TPR < 256 ? 1 : TPR / 64];  // taken in turn: no wait for the last row's reads
  __shared__ float sdw[RPB > 1 ? RPB * TPR * V : 1];
  const int j = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  float dw[NV][V], w[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + j) * V;
    load_weight<V>(w[k], a.w, c, a.D - c);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = 0.f;
  }
  int flip = 0;
  for (size_t row = (size_t)blockIdx.x * RPB + slot; row < (size_t)a.rows; row += (size_t)a.nblk * RPB) {
    const T* h = reinterpret_cast<const T*>(a.x) + row * a.xs;
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.D;
    const T* z = GATE ? reinterpret_cast<const T*>(a.gate) + row * a.gs : nullptr;
    const T* din = a.dh_in != nullptr ? reinterpret_cast<const T*>(a.dh_in) + row * a.D : nullptr;
    vec hv[NV], yv[NV], zv[NV], iv[NV];
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + j) * V;
      const int left = a.D - c;
      hv[k] = load_piece(h + c, left);
      yv[k] = load_piece(dy + c, left);
      if constexpr (GATE) zv[k] = load_piece(z + c, left);
      iv[k] = (vec)(0);
      if (din != nullptr) iv[k] = load_piece(din + c, left);
    }
    float u[NV][V], sg[GATE ? NV : 1][V];  // u = dy silu(z)
    const auto through_gate = [&](int k, int e) {
      u[k][e] = (float)yv[k][e];
      if constexpr (GATE) {
        sg[k][e] = sigmoid<T>((float)zv[k][e]);
        u[k][e] *= (float)zv[k][e] * sg[k][e];
      }
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hh = (float)hv[k][e];
        through_gate(k, e);
        s += hh * hh;
        q += u[k][e] * w[k][e] * hh;
      }
    }
    s = row_sum<TPR>(s, buf[flip][0]);
    q = row_sum<TPR>(q, buf[flip][1]);
    flip ^= 1;
    const float r = 1.f / sqrtf(s / a.D + a.eps), mean = q * r / a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + j) * V;
      if (c >= a.D) continue;
      if constexpr (AGAIN) {  // z of unknown origin, so that the compiler does not hold what it has formed from it
        typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
        u32x4 z4 = __builtin_bit_cast(u32x4, zv[k]);
        asm volatile("" : "+v"(z4));
        zv[k] = __builtin_bit_cast(vec, z4);
      }
      vec o, og;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = (float)hv[k][e] * r;
        if constexpr (AGAIN) through_gate(k, e);
        dw[k][e] += u[k][e] * hat;
        o[e] = (T)(r * (u[k][e] * w[k][e] - hat * mean) + (float)iv[k][e]);
        if constexpr (GATE) {
          const float zz = (float)zv[k][e];
          og[e] = (T)((float)yv[k][e] * hat * w[k][e] * (sg[k][e] * (1.f + zz * (1.f - sg[k][e]))));
        }
      }
      store_piece(reinterpret_cast<T*>(a.h) + row * a.D + c, o, a.D - c);
      if constexpr (GATE) store_piece(reinterpret_cast<T*>(a.dgate) + row * a.D + c, og, a.D - c);
    }
  }
  if (a.dw == nullptr) return;
  float* part = a.part + (size_t)blockIdx.x * a.D;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + j) * V;
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) sdw[(slot * V + e) * TPR + j] = dw[k][e];
      __syncthreads();
      for (int i = threadIdx.x; i < TPR * V; i += 256) {  // i = e TPR + lane
        float t = 0.f;
#pragma unroll
        for (int p = 0; p < RPB; ++p) t += sdw[p * V * TPR + i];
        const int col = (k * TPR + i % TPR) * V + i / TPR;
        if (col < a.D) part[col] = t;
      }
    } else if (c < a.D) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < a.D) part[c + e] = dw[k][e];
    }
  }
}

// dweight from the workgroups' shares, in float64 and a fixed order: 32 columns per workgroup, 32 lanes down the shares
// of each.
__global__ __launch_bounds__(1024) void wsum_kernel(NormArgs a) {
  __shared__ double part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, q = threadIdx.x / 32;
  double s = 0.0;
  if (c < a.D) {
#pragma unroll 8
    for (int k = q; k < a.nblk; k += 32) s += (double)a.part[(size_t)k * a.D + c];
  }
  part[q][threadIdx.x % 32] = s;
  __syncthreads();
  if (q == 0 && c < a.D) {
    s = 0.0;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += part[k][threadIdx.x];
    a.dw[c] = (float)s;
  }
}

}  // namespace norm
}  // namespace prism
