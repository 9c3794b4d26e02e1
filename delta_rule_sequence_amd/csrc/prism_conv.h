// prism_conv.h - depthwise causal convolution over the tokens: forward, backward and one token (gfx950).
//
//   pre_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = pre_t or silu(pre_t)        (per channel)
//   g_t = dy_t (silu'(pre_t) or 1),  dx_t = sum_j w_j g_{t+K-1-j},  dw_j = sum_t x_{t-K+1+j} g_t,  dbias = sum_t g_t
//
// Bound by its bytes.  A thread owns V neighbouring channels (16 bytes) and walks a strip of tokens with the K
// rows of the window in registers, so that a row is read once per strip (K - 1 rows again at its border).
// Rows or pointers that are not 16-byte aligned run with V = 1.
#pragma once
#include "prism_ssm_args.h"
#include "prism_tile.h"

namespace prism {
namespace conv {

template <class T, int V> struct Vec { typedef T type __attribute__((ext_vector_type(V))); };
template <class T> struct Vec<T, 1> { typedef T type; };

template <class T, int V>
__device__ __forceinline__ void load_v(float (&o)[V], const T* p) {
  const auto v = *reinterpret_cast<const typename Vec<T, V>::type*>(p);
  if constexpr (V == 1) o[0] = (float)v;
  else
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = (float)v[k];
}
template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&o)[V]) {
  typename Vec<T, V>::type v;
  if constexpr (V == 1) v = (T)o[0];
  else
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = (T)o[k];
  *reinterpret_cast<typename Vec<T, V>::type*>(p) = v;
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

__device__ __forceinline__ int seq_len(const ConvArgs& a, int b) {
  if (a.lens == nullptr) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

// Row t of the sequence as floats: before 0 from the history (zero without one).
template <class T, int K, int V>
__device__ __forceinline__ void row(float (&o)[V], const ConvArgs& a, int b, int h, int t, int d) {
  if (t >= 0) {
    load_v<T, V>(o, reinterpret_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + (long long)t * a.xs.t + d);
  } else if (a.conv_in != nullptr) {
    load_v<T, V>(o, reinterpret_cast<const T*>(a.conv_in) + ((size_t)(b * a.H + h) * (K - 1) + t + K - 1) * a.D + d);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.f;
  }
}

// Grid (channel blocks, strips, B * H).  The workgroup that holds a sequence's last row also writes conv_out.
template <class T, int K, int V>
__global__ __launch_bounds__(256) void fwd_kernel(ConvArgs a) {
  const int d = (blockIdx.x * 64 + threadIdx.x % 64) * V, strip = blockIdx.y * 4 + threadIdx.x / 64;
  const int bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  if (d >= a.D || strip >= a.nstrip) return;
  const int len = seq_len(a, b), t0 = strip * a.strip, t1 = min(t0 + a.strip, len);
  float w[K][V], bias[V], x[K][V];
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) w[j][k] = a.w[((size_t)h * K + j) * a.D + d + k];
#pragma unroll
  for (int k = 0; k < V; ++k) bias[k] = a.bias != nullptr ? a.bias[(size_t)h * a.D + d + k] : 0.f;
  if (t0 < t1) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row<T, K, V>(x[j + 1], a, b, h, t0 - K + 1 + j, d);
  }
  T* y = reinterpret_cast<T*>(a.y) + b * a.ys.b + h * a.ys.h + d;
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) x[j][k] = x[j + 1][k];
    row<T, K, V>(x[K - 1], a, b, h, t, d);
    float o[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float s = bias[k];
#pragma unroll
      for (int j = 0; j < K; ++j) s += w[j][k] * x[j][k];
      o[k] = a.silu ? s * sigmoid_f(s) : s;
    }
    store_v<T, V>(y + (long long)t * a.ys.t, o);
  }
}

// conv_out: rows len - K + 1 .. len - 1 of [conv_in; x].  Each thread reads its channel's rows before it writes,
// so conv_out may be conv_in.  Grid (channels / 256, B * H).
template <class T, int K>
__global__ __launch_bounds__(256) void tail_kernel(ConvArgs a) {
  const int d = blockIdx.x * 256 + threadIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
  if (d >= a.D) return;
  const int len = seq_len(a, b);
  float v[K - 1][1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) row<T, K, 1>(v[j], a, b, h, len - K + 1 + j, d);
  T* o = reinterpret_cast<T*>(a.conv_out) + (size_t)bh * (K - 1) * a.D + d;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) o[(size_t)j * a.D] = (T)v[j][0];
}

// Grid as fwd_kernel.  A strip's thread forms g for its tokens and the K - 1 after them (their dx reach back), and
// the strip's shares of dw and dbias.
template <class T, int K, int V>
__global__ __launch_bounds__(256) void bwd_kernel(ConvArgs a) {
  const int d = (blockIdx.x * 64 + threadIdx.x % 64) * V, strip = blockIdx.y * 4 + threadIdx.x / 64;
  const int bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  if (d >= a.D || strip >= a.nstrip) return;
  const int t0 = strip * a.strip, t1 = min(t0 + a.strip, a.T);
  float w[K][V], bias[V], x[K][V], g[K][V], dw[K][V], db[V];
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) w[j][k] = a.w[((size_t)h * K + j) * a.D + d + k];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    bias[k] = a.bias != nullptr ? a.bias[(size_t)h * a.D + d + k] : 0.f;
    db[k] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][k] = g[j][k] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j) row<T, K, V>(x[j + 1], a, b, h, t0 - K + 1 + j, d);
  const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dys.b + h * a.dys.h + d;
  T* dx = reinterpret_cast<T*>(a.y) + b * a.ys.b + h * a.ys.h + d;
  for (int t = t0; t < t1 + K - 1; ++t) {
    float gy[V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        x[j][k] = x[j + 1][k];
        g[j][k] = g[j + 1][k];
      }
    if (t < a.T) {
      row<T, K, V>(x[K - 1], a, b, h, t, d);
      load_v<T, V>(gy, dy + (long long)t * a.dys.t);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float s = bias[k];
#pragma unroll
        for (int j = 0; j < K; ++j) s += w[j][k] * x[j][k];
        const float sg = sigmoid_f(s);
        g[K - 1][k] = a.silu ? gy[k] * (sg * (1.f + s * (1.f - sg))) : gy[k];
      }
      if (t < t1) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          db[k] += g[K - 1][k];
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][k] += x[j][k] * g[K - 1][k];
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) g[K - 1][k] = 0.f;
    }
    if (t - K + 1 >= t0) {  // g[j] is g_{t-K+1+j}: dx_{t-K+1} = sum_j w_{K-1-j} g[j]
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        o[k] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) o[k] += w[K - 1 - j][k] * g[j][k];
      }
      store_v<T, V>(dx + (long long)(t - K + 1) * a.ys.t, o);
    }
  }
  float* part = a.part + (((size_t)b * a.nstrip + strip) * a.H + h) * (K + 1) * a.D + d;
#pragma unroll
  for (int j = 0; j < K; ++j) store_v<float, V>(part + (size_t)j * a.D, dw[j]);
  store_v<float, V>(part + (size_t)K * a.D, db);
}

// dw and dbias: the strips' shares summed in a fixed order.  Grid (channels / 64, (K + 1) rows, H); the four waves take a
// quarter of the shares each.
template <int K>
__global__ __launch_bounds__(256) void wsum_kernel(ConvArgs a) {
  const int d = blockIdx.x * 64 + threadIdx.x % 64, j = blockIdx.y, h = blockIdx.z, q = threadIdx.x / 64;
  const int n = a.B * a.nstrip;
  __shared__ double part[4][64];
  double s = 0.0;
  if (d < a.D)
    for (int k = q; k < n; k += 4) s += (double)a.part[(((size_t)k * a.H + h) * (K + 1) + j) * a.D + d];
  part[q][threadIdx.x % 64] = s;
  __syncthreads();
  if (q != 0 || d >= a.D) return;
  s = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
  if (j < K) a.dw[((size_t)h * K + j) * a.D + d] = (float)s;
  else if (a.dbias != nullptr) a.dbias[(size_t)h * a.D + d] = (float)s;
}

// One token per (b, h, channel), the window updated in place.
template <class T, int K>
__global__ __launch_bounds__(256) void step_kernel(ConvArgs a) {
  const size_t n = (size_t)a.B * a.H * a.D, e = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const int d = (int)(e % a.D), bh = (int)(e / a.D), b = bh / a.H, h = bh % a.H;
  T* st = reinterpret_cast<T*>(const_cast<void*>(a.conv_in)) + (size_t)bh * (K - 1) * a.D + d;
  T x[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) x[j] = st[(size_t)j * a.D];
  x[K - 1] = reinterpret_cast<const T*>(a.x)[b * a.xs.b + h * a.xs.h + d];
  float s = a.bias != nullptr ? a.bias[(size_t)h * a.D + d] : 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j) s += a.w[((size_t)h * K + j) * a.D + d] * (float)x[j];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) st[(size_t)j * a.D] = x[j + 1];
  reinterpret_cast<T*>(a.y)[e] = (T)(a.silu ? s * sigmoid_f(s) : s);
}

}  // namespace conv
}  // namespace prism
