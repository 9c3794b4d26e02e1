// prism_conv.h - depthwise causal convolution over the tokens: forward, backward and one token (gfx950).
//
//   pre_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = pre_t or silu(pre_t)        (per channel)
//   g_t = dy_t (silu'(pre_t) or 1),  dx_t = sum_j w_j g_{t+K-1-j},  dw_j = sum_t x_{t-K+1+j} g_t,  dbias = sum_t g_t
//
// Bound by its bytes.  A thread owns V neighbouring channels and walks a strip of tokens with the K rows of the window
// in registers, so that a row is read once per strip (K - 1 rows again at its border).  Rows may start anywhere (the
// accesses need the alignment of an element only); the last thread of a row loads the last V channels and writes those
// its neighbour has not (the history may be written in place, so no value may come from two threads).
//
// Measured on 8 x 2048 x 1792 bfloat16, K = 4, silu: forward (ragged lengths) 13 to 15 us, 3.9 to 4.5 TB/s where a
// copy of 1 GiB makes 5.2; backward 42 us and 4 for the sum of the shares, 3.8 TB/s: it forms silu' again, 24 us of vector
// instructions beside its loads.  One token of 4 x 896: 2.7 us, a launch.
#pragma once
#include <type_traits>

#include "prism_silu.h"
#include "prism_ssm_args.h"
#include "prism_tile.h"

namespace prism {
namespace conv {

template <class T, int V> struct Vec { typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T)))); };
template <class T> struct Vec<T, 1> { typedef T type; };

template <class T, int V>
__device__ __forceinline__ float elem(const typename Vec<T, V>::type& v, int k) {
  if constexpr (V == 1) return (float)v;
  else return (float)v[k];
}
// Values from .. V - 1 of the vector.
template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const typename Vec<T, V>::type& v, int from) {
  if constexpr (V == 1) {
    *p = v;
  } else if (from == 0) {
    *reinterpret_cast<typename Vec<T, V>::type*>(p) = v;
  } else {
#pragma unroll
    for (int k = 1; k < V; ++k)
      if (k >= from) p[k] = v[k];
  }
}
template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&o)[V], int from) {
  typename Vec<T, V>::type v;
  if constexpr (V == 1) v = (T)o[0];
  else
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = (T)o[k];
  store_v<T, V>(p, v, from);
}

// V weights of one channel group in 16-byte loads (any 4-byte alignment).
template <int V>
__device__ __forceinline__ void load_w(float (&o)[V], const float* p) {
  typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
  if constexpr (V == 1) {
    o[0] = *p;
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const f4 v = *reinterpret_cast<const f4*>(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k + e] = v[e];
    }
  }
}
// The filter and bias of channels d .. d + V - 1.
template <int K, int V>
__device__ __forceinline__ void load_filter(float (&w)[K][V], float (&bias)[V], const ConvArgs& a, int h, int d) {
#pragma unroll
  for (int j = 0; j < K; ++j) load_w<V>(w[j], a.w + ((size_t)h * K + j) * a.D + d);
  if (a.bias != nullptr) {
    load_w<V>(bias, a.bias + (size_t)h * a.D + d);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) bias[k] = 0.f;
  }
}

__device__ __forceinline__ int seq_len(const ConvArgs& a, int b) {
  if (a.lens == nullptr) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

// Row t of the sequence: before 0 from the history (zero without one).
template <class T, int K, int V>
__device__ __forceinline__ typename Vec<T, V>::type row(const ConvArgs& a, int b, int h, int t, int d) {
  typedef typename Vec<T, V>::type vec;
  if (t >= 0) return *reinterpret_cast<const vec*>(reinterpret_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + (long long)t * a.xs.t + d);
  if (a.conv_in == nullptr) return vec(0);
  return *reinterpret_cast<const vec*>(reinterpret_cast<const T*>(a.conv_in) + ((size_t)(b * a.H + h) * (K - 1) + t + K - 1) * a.D + d);
}

// Grid (channel blocks of 64 threads, strips / 4, B * H).  Rows are loaded U at a time, so that a thread keeps U 16-byte loads in
// flight.  The first strip's threads also write conv_out: they alone read the history, so it may be the same buffer.
// TAIL: D is not a multiple of V (the check at every store costs 8 x 2048 x 1792 tokens 0.8 of 13 us).
template <class T, int K, int V, int U, bool SILU, bool TAIL>
__global__ __launch_bounds__(256) void fwd_kernel(ConvArgs a) {
  typedef typename Vec<T, V>::type vec;
  const int first = (blockIdx.x * 64 + threadIdx.x % 64) * V, d = TAIL ? min(first, a.D - V) : first, from = TAIL ? first - d : 0;
  const int strip = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);  // one strip per wave
  const int bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  if (first >= a.D || strip >= a.nstrip) return;
  const int len = seq_len(a, b), t0 = strip * a.strip, t1 = t0 + min(a.strip, len - t0);  // the last strip may end past 2^31
  if (t0 < t1) {
    float w[K][V], bias[V], x[K][V];
    load_filter<K, V>(w, bias, a, h, d);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const vec v = row<T, K, V>(a, b, h, t0 - K + 1 + j, d);
#pragma unroll
      for (int k = 0; k < V; ++k) x[j + 1][k] = elem<T, V>(v, k);
    }
    const T* xp = reinterpret_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + d;
    T* y = reinterpret_cast<T*>(a.y) + b * a.ys.b + h * a.ys.h + d;
    for (int t = t0; t < t1; t += U) {
      vec in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) in[u] = *reinterpret_cast<const vec*>(xp + (long long)min(t + u, t1 - 1) * a.xs.t);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t1) break;
        float o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
#pragma unroll
          for (int j = 0; j < K - 1; ++j) x[j][k] = x[j + 1][k];
          x[K - 1][k] = elem<T, V>(in[u], k);
          float s = bias[k];
#pragma unroll
          for (int j = 0; j < K; ++j) s += w[j][k] * x[j][k];
          o[k] = SILU ? s * sigmoid<T>(s) : s;
        }
        store_v<T, V>(y + (long long)(t + u) * a.ys.t, o, from);
      }
    }
  }
  if (strip == 0 && a.conv_out != nullptr) {  // rows len - K + 1 .. len - 1 of [conv_in; x]
    vec tail[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) tail[j] = row<T, K, V>(a, b, h, len - K + 1 + j, d);
    T* o = reinterpret_cast<T*>(a.conv_out) + (size_t)bh * (K - 1) * a.D + d;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_v<T, V>(o + (size_t)j * a.D, tail[j], from);
  }
}

// Grid as fwd_kernel.  A strip's thread forms g for its tokens and the K - 1 after them (their dx reach back), and the
// strip's shares of dw and dbias, which the workgroup's four strips join in LDS.
template <class T, int K, int V, int U, bool SILU, bool TAIL>
__global__ __launch_bounds__(256) void bwd_kernel(ConvArgs a) {
  typedef typename Vec<T, V>::type vec;
  __shared__ float sum[4][V][64];
  const int lane = threadIdx.x % 64, q = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);  // one strip per wave
  const int first = (blockIdx.x * 64 + lane) * V, d = TAIL ? min(first, a.D - V) : first, from = TAIL ? first - d : 0;
  const int strip = blockIdx.y * 4 + q;
  const int bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  float dw[K + 1][V];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[j][k] = 0.f;
  if (first < a.D && strip < a.nstrip) {
    const int t0 = strip * a.strip, t1 = t0 + min(a.strip, a.T - t0);
    float w[K][V], bias[V], x[K][V], g[K][V];
    load_filter<K, V>(w, bias, a, h, d);
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int k = 0; k < V; ++k) g[j][k] = 0.f;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const vec v = row<T, K, V>(a, b, h, t0 - K + 1 + j, d);
#pragma unroll
      for (int k = 0; k < V; ++k) x[j + 1][k] = elem<T, V>(v, k);
    }
    const T* xp = reinterpret_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + d;
    const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dys.b + h * a.dys.h + d;
    T* dx = reinterpret_cast<T*>(a.y) + b * a.ys.b + h * a.ys.h + d;
    // A token of the strip (OWN), or one after it, of which dx only needs g: left out of dw by a product with 0, the rows of the
    // window would carry an infinity into taps that do not read them.
    const auto token = [&](const vec& xin, const vec& gin, int tt, auto is_own) {
      constexpr bool OWN = decltype(is_own)::value;
      const bool real = OWN || tt < a.T;
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          x[j][k] = x[j + 1][k];
          g[j][k] = g[j + 1][k];
        }
        x[K - 1][k] = elem<T, V>(xin, k);
        float gk = real ? elem<T, V>(gin, k) : 0.f;
        if constexpr (SILU) {
          float s = bias[k];
#pragma unroll
          for (int j = 0; j < K; ++j) s += w[j][k] * x[j][k];
          const float sg = sigmoid<T>(s);
          gk = real ? gk * (sg * (1.f + s * (1.f - sg))) : 0.f;
        }
        g[K - 1][k] = gk;
        if constexpr (OWN) {
          dw[K][k] += gk;
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][k] += x[j][k] * gk;
        }
        // g[j] is g_{tt-K+1+j}: dx_{tt-K+1} = sum_j w_{K-1-j} g[j]
        o[k] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) o[k] += w[K - 1 - j][k] * g[j][k];
      }
      if (tt - K + 1 >= t0) store_v<T, V>(dx + (long long)(tt - K + 1) * a.ys.t, o, from);
    };
    for (int t = t0; t < t1; t += U) {
      vec in[U], gy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tt = min(t + u, t1 - 1);
        in[u] = *reinterpret_cast<const vec*>(xp + (long long)tt * a.xs.t);
        gy[u] = *reinterpret_cast<const vec*>(dy + (long long)tt * a.dys.t);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t1) break;
        token(in[u], gy[u], t + u, std::true_type());
      }
    }
    vec in[K - 1], gy[K - 1];
#pragma unroll
    for (int u = 0; u < K - 1; ++u) {
      const int tt = min(t1 + u, a.T - 1);
      in[u] = *reinterpret_cast<const vec*>(xp + (long long)tt * a.xs.t);
      gy[u] = *reinterpret_cast<const vec*>(dy + (long long)tt * a.dys.t);
    }
#pragma unroll
    for (int u = 0; u < K - 1; ++u) token(in[u], gy[u], t1 + u, std::false_type());
  }
  float* part = a.part + (((size_t)b * gridDim.y + blockIdx.y) * a.H + h) * (K + 1) * a.D;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) sum[q][k][lane] = dw[j][k];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * V; i += 256) {
      const int k = i % V, ln = i / V, at = (blockIdx.x * 64 + ln) * V;
      const int col = min(at, a.D - V) + k;
      if (at < a.D && col >= at) part[(size_t)j * a.D + col] = (sum[0][k][ln] + sum[1][k][ln]) + (sum[2][k][ln] + sum[3][k][ln]);
    }
  }
}

// dw and dbias: the workgroups' shares summed in a fixed order.  Grid (channels / 32, (K + 1) rows, H), 32 lanes down the
// shares of a channel.
template <int K>
__global__ __launch_bounds__(1024) void wsum_kernel(ConvArgs a) {
  const int d = blockIdx.x * 32 + threadIdx.x % 32, j = blockIdx.y, h = blockIdx.z, q = threadIdx.x / 32;
  const int n = a.B * ((a.nstrip + 3) / 4);
  __shared__ double part[32][33];
  double s = 0.0;
  if (d < a.D) {
#pragma unroll 4
    for (int k = q; k < n; k += 32) s += (double)a.part[(((size_t)k * a.H + h) * (K + 1) + j) * a.D + d];
  }
  part[q][threadIdx.x % 32] = s;
  __syncthreads();
  if (q != 0 || d >= a.D) return;
  s = 0.0;
#pragma unroll
  for (int k = 0; k < 32; ++k) s += part[k][threadIdx.x];
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
  reinterpret_cast<T*>(a.y)[e] = (T)(a.silu ? s * sigmoid<T>(s) : s);
}

}  // namespace conv
}  // namespace prism
