// prism_rope.h - norm of queries and keys for each head and rotation by position, in one pass, and its gradients (gfx950).
//
//   h = w x / sqrt(mean x^2 + eps) (with weights; else h = x);   for pair i < rot / 2 of channels (a, b):
//   y_a = factor (h_a cos - h_b sin),  y_b = factor (h_b cos + h_a sin),  angle pos freq_i;   the other channels: y = h
//   pairs: channels (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved
//   backward: g = the rotation by -angle of dy;  with u = g w, xhat = x r:  dx = r (u - xhat mean(u xhat)),  dw = sum g xhat
//
// Bound by its bytes: a row is read once, by a group of lanes that holds V pairs (or 2 V of the other channels) each,
// and a lane group takes several heads of one token, whose sines and cosines it forms once, four rows in flight.  The forward runs at 0.72
// of a copy's rate (18 us for 13), the backward, which reads x and dy, at 0.7 without the weights' sum of 4 to 6 us.
#pragma once
#include "prism_attn_args.h"
#include "prism_tile.h"

namespace prism {
namespace rope {

// sin and cos of 2 pi t, t formed and reduced in float64: three roundings, 2^-53 of the angle each (2^-31 at an angle of 2^20).
// What is left is an eighth of a turn on both sides of a quarter; there Taylor's series to x^9 and x^10 end below 2^-28.
__device__ __forceinline__ void turn(double t, float* sn, float* cs) {
  const double q = __builtin_rint(4.0 * t);
  const float x = (float)((4.0 * t - q) * 1.57079632679489661923);
  const float z = x * x;
  const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const int k = (int)(q - 4.0 * __builtin_floor(0.25 * q));           // the quarter, 0 .. 3
  const float a = (k & 1) != 0 ? c : s, b = (k & 1) != 0 ? s : c;
  *sn = (k & 2) != 0 ? -a : a;
  *cs = ((k + 1) & 2) != 0 ? -b : b;
}

// What a lane holds of a row: NU units u = lane, lane + L, ...: pairs V u .. V u + V - 1 (x[0], x[1]: their two
// channels), or behind them 2 V of the other channels.
template <int V, int L, int NU> struct Lane {
  int at[NU][2];       // first channels of a unit's two runs, or of its one run of 2 V
  bool pairs[NU], live[NU];

  __device__ __forceinline__ Lane(const RopeArgs& a, int lane) {
    const int half = a.rot / 2, turned = half / V, units = a.D / (2 * V);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + i * L;
      live[i] = u < units;
      pairs[i] = u < turned;
      at[i][0] = !pairs[i] ? a.rot + (u - turned) * 2 * V : a.interleaved ? 2 * V * u : V * u;
      at[i][1] = pairs[i] && !a.interleaved ? half + V * u : at[i][0] + V;
    }
  }
};

// Channels of a unit in memory order: two runs of V.
template <class T, int V, int NU> struct Row {
  T v[NU][2][V];
  template <class LANE> __device__ __forceinline__ void load(const T* p, const LANE& ln) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (ln.live[i]) __builtin_memcpy(v[i][k], p + ln.at[i][k], sizeof(v[i][k]));
  }
  template <class LANE> __device__ __forceinline__ void store(T* p, const LANE& ln) const {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (ln.live[i]) __builtin_memcpy(p + ln.at[i][k], v[i][k], sizeof(v[i][k]));
  }
};

template <int L> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// The angles of a lane's pairs at a token, times factor.
template <int V, int NU> struct Angles {
  float sn[NU][V], cs[NU][V];
  template <class LANE> __device__ __forceinline__ void set(const RopeArgs& a, const LANE& ln, int lane, int L, int pos) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sn[i][j] = 0.f, cs[i][j] = 1.f;
        if (!ln.pairs[i]) continue;
        turn((double)pos * ((double)a.freq[(lane + i * L) * V + j] * 0.15915494309189533577), &sn[i][j], &cs[i][j]);
        sn[i][j] *= a.factor, cs[i][j] *= a.factor;
      }
  }
};

// The rotation of a unit's V pairs; sign -1: back.  Interleaved pairs are neighbours in memory order.
template <int V>
__device__ __forceinline__ void rotate(float (&x)[2][V], const float (&sn)[V], const float (&cs)[V], bool interleaved, float sign) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float* const pa = interleaved ? &x[2 * j / V][2 * j % V] : &x[0][j];
    float* const pb = interleaved ? &x[(2 * j + 1) / V][(2 * j + 1) % V] : &x[1][j];
    const float p = *pa, q = *pb, s = sign * sn[j];
    *pa = p * cs[j] - q * s;
    *pb = q * cs[j] + p * s;
  }
}

// A lane group's token and heads: unit g of tokens x groups.
struct Work {
  int b, t, first, last;             // heads first .. last - 1 of x[0]'s and then x[1]'s
};
__device__ __forceinline__ Work work_of(const RopeArgs& a, size_t unit) {
  Work w;
  const size_t token = unit / (unsigned)a.groups;
  w.first = (int)(unit - token * a.groups) * a.per;
  w.last = min(w.first + a.per, a.heads[0] + a.heads[1]);
  w.b = (int)(token / (unsigned)a.T);
  w.t = (int)(token - (size_t)w.b * a.T);
  return w;
}
__device__ __forceinline__ long long row_at(const prism_strides& s, const Work& w, int head) { return w.b * s.b + head * s.h + (long long)w.t * s.t; }

// The weights of a lane's channels (ones without).
template <int V, int NU, class LANE>
__device__ __forceinline__ void weights(float (&w)[NU][2][V], const float* p, const LANE& ln) {
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[i][k][j] = ln.live[i] && p == nullptr ? 1.f : 0.f;
      if (ln.live[i] && p != nullptr) __builtin_memcpy(w[i][k], p + ln.at[i][k], sizeof(w[i][k]));
    }
}
template <class T, int V, int NU, class LANE>
__device__ __forceinline__ void widen(float (&x)[NU][2][V], const Row<T, V, NU>& row, const LANE& ln) {
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][k][j] = ln.live[i] ? (float)row.v[i][k][j] : 0.f;
}

constexpr int kAtOnce = 4;           // rows of a lane group in flight

template <class T, int V, int L, int NU, bool INTER>
__global__ __launch_bounds__(256) void fwd_kernel(RopeArgs a) {
  const int lane = threadIdx.x % L;
  const size_t unit = (size_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (unit >= (size_t)a.B * a.T * a.groups) return;
  const Work wk = work_of(a, unit);
  const Lane<V, L, NU> ln(a, lane);
  Angles<V, NU> an;
  an.set(a, ln, lane, L, a.pos != nullptr ? a.pos[(size_t)wk.b * a.T + wk.t] : wk.t);
  const bool norm = a.w[0] != nullptr;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int start = q != 0 ? a.heads[0] : 0, lo = max(wk.first, start) - start, hi = min(wk.last - start, a.heads[q]);
    if (lo >= hi) continue;
    float w[NU][2][V];
    weights<V, NU>(w, a.w[q], ln);
    const T* const src = (const T*)a.x[q] + row_at(a.xs[q], wk, 0);
    T* const dst = (T*)a.y[q] + row_at(a.ys[q], wk, 0);
    for (int head = lo; head < hi; head += kAtOnce) {
      Row<T, V, NU> row[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (head + u < hi) row[u].load(src + (head + u) * a.xs[q].h, ln);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (head + u >= hi) break;
        float x[NU][2][V], ss = 0.f;
        widen<T, V, NU>(x, row[u], ln);
        if (norm) {
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < V; ++j) ss = fmaf(x[i][k][j], x[i][k][j], ss);
          const float r = 1.f / sqrtf(group_sum<L>(ss) / a.D + a.eps);
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < V; ++j) x[i][k][j] *= r * w[i][k][j];
        }
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          if (ln.pairs[i]) rotate<V>(x[i], an.sn[i], an.cs[i], INTER, 1.f);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) row[u].v[i][k][j] = (T)x[i][k][j];
        }
        row[u].store(dst + (head + u) * a.ys[q].h, ln);
      }
    }
  }
}

// Workgroup k takes the lane groups' units k, k + nblk, ... (256 / L at a time); its shares of dw stay in part[k].
template <class T, int V, int L, int NU, bool INTER>
__global__ __launch_bounds__(256) void bwd_kernel(RopeArgs a) {
  constexpr int S = 256 / L, U = 2;
  __shared__ float shares[S][L][NU * 2 * V + 1];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const size_t units = (size_t)a.B * a.T * a.groups;
  const Lane<V, L, NU> ln(a, lane);
  const bool norm = a.w[0] != nullptr;
  float dw[2][NU][2][V], w[2][NU][2][V];
#pragma unroll
  for (int q = 0; q < 2 * NU * 2 * V; ++q) (&dw[0][0][0][0])[q] = 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) weights<V, NU>(w[q], a.w[q], ln);
  for (size_t unit = (size_t)blockIdx.x * S + slot; unit < units; unit += (size_t)a.nblk * S) {
    const Work wk = work_of(a, unit);
    Angles<V, NU> an;
    an.set(a, ln, lane, L, a.pos != nullptr ? a.pos[(size_t)wk.b * a.T + wk.t] : wk.t);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int start = q != 0 ? a.heads[0] : 0, lo = max(wk.first, start) - start, hi = min(wk.last - start, a.heads[q]);
      const T* const src = (const T*)a.dy[q] + row_at(a.dys[q], wk, 0);
      const T* const old = (const T*)a.x[q] + row_at(a.xs[q], wk, 0);
      T* const dst = (T*)a.y[q] + row_at(a.ys[q], wk, 0);
      for (int head = lo; head < hi; head += U) {
        Row<T, V, NU> gr[U], xr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (head + u >= hi) break;
          gr[u].load(src + (head + u) * a.dys[q].h, ln);
          if (norm) xr[u].load(old + (head + u) * a.xs[q].h, ln);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (head + u >= hi) break;
          float g[NU][2][V];
          widen<T, V, NU>(g, gr[u], ln);
#pragma unroll
          for (int i = 0; i < NU; ++i)
            if (ln.pairs[i]) rotate<V>(g[i], an.sn[i], an.cs[i], INTER, -1.f);
          if (norm) {
            float x[NU][2][V], ss = 0.f, ux = 0.f;
            widen<T, V, NU>(x, xr[u], ln);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                  ss = fmaf(x[i][k][j], x[i][k][j], ss);
                  ux = fmaf(g[i][k][j] * w[q][i][k][j], x[i][k][j], ux);
                }
            const float r = 1.f / sqrtf(group_sum<L>(ss) / a.D + a.eps);
            const float mean = group_sum<L>(ux) * r / a.D;             // of u xhat
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                  const float hat = x[i][k][j] * r;
                  dw[q][i][k][j] = fmaf(g[i][k][j], hat, dw[q][i][k][j]);
                  g[i][k][j] = r * (g[i][k][j] * w[q][i][k][j] - hat * mean);
                }
          }
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < V; ++j) gr[u].v[i][k][j] = (T)g[i][k][j];
          gr[u].store(dst + (head + u) * a.ys[q].h, ln);
        }
      }
    }
  }
  if (!norm || a.part == nullptr) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NU * 2 * V; ++c) shares[slot][lane][c] = (&dw[q][0][0][0])[c];
    __syncthreads();
    for (int c = threadIdx.x; c < L * NU * 2 * V; c += 256) {
      const int ln2 = c % L, val = c / L, i = val / (2 * V), k = val / V % 2, j = val % V;
      float sum = 0.f;
      for (int g = 0; g < S; ++g) sum += shares[g][ln2][val];
      const int half = a.rot / 2, turned = half / V, u = ln2 + i * L;
      if (u >= a.D / (2 * V)) continue;
      const bool pair = u < turned;
      const int at0 = !pair ? a.rot + (u - turned) * 2 * V : INTER ? 2 * V * u : V * u;
      const int at1 = pair && !INTER ? half + V * u : at0 + V;
      a.part[((size_t)blockIdx.x * 2 + q) * a.D + (k != 0 ? at1 : at0) + j] = sum;
    }
  }
}

// The sums of the workgroups' shares: 32 columns per workgroup, 32 lanes of shares each.
__global__ __launch_bounds__(1024) void sum_kernel(RopeArgs a) {
  __shared__ float part[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < 2 * a.D)
    for (int k = g; k < a.nblk; k += 32) s += a.part[(size_t)k * 2 * a.D + col];
  part[g][c] = s;
  __syncthreads();
  if (threadIdx.x >= 32 || col >= 2 * a.D) return;
  s = 0.f;
  for (int k = 0; k < 32; ++k) s += part[k][c];
  float* const dw = col < a.D ? a.dw[0] : a.dw[1];
  if (dw != nullptr) dw[col < a.D ? col : col - a.D] = s;
}

}  // namespace rope
}  // namespace prism
