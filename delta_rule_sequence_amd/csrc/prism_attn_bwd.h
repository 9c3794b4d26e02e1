// prism_attn_bwd.h - softmax attention of a prompt's rows (gfx950), backward.
//
//   p_ij = e^(s_ij - lse_i),  dp_ij = <do_i, v_j>,  ds_ij = p_ij (dp_ij - <do_i, o_i>)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij do_i   (i over the group's heads)
//
// Two kernels form the tiles of s and dp once each, so that every sum stays in one wave's registers and has a fixed order
// (seven products where five would do with sums across workgroups): dq by queries, with the forward's transposed tiles;
// dk and dv by keys, with tiles whose columns are keys.
#pragma once
#include "prism_attn.h"

namespace prism {
namespace attn {

// Staged rows of two tensors with one geometry: tiles of BN rows, a thread's pieces on their way to LDS.
template <class T, int D, int BN, int THREADS> struct Stage {
  using R = Rows<T, D>;
  static constexpr int kEach = BN * R::kPieces / THREADS, kStep = THREADS / R::kPieces;
  static_assert(BN * R::kPieces % THREADS == 0, "whole pieces");
  u32x4 x[kEach];
  __device__ __forceinline__ void load(const char* p, int n, int stride, int tid) {
    const auto r = rows_of(p, min(n, BN), stride, R::kBytes);
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = load16(r, (tid / R::kPieces + i * kStep) * stride + tid % R::kPieces * 16);
  }
  __device__ __forceinline__ void store(char* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      *reinterpret_cast<u32x4*>(tile + (tid / R::kPieces + i * kStep) * R::kStride + tid % R::kPieces * 16) = x[i];
  }
};

// One row's piece of an operand held in registers: rows qw + l % 32, steps of 2 pieces.
template <int STEPS>
__device__ __forceinline__ void hold(u32x4 (&f)[STEPS], const char* p, int n, int stride, int l) {
  const auto r = rows_of(p, min(32, n), stride, STEPS * 32);
#pragma unroll
  for (int k = 0; k < STEPS; ++k) f[k] = load16(r, (l & 31) * stride + (2 * k + (l >> 5)) * 16);
}

template <class T>
__device__ __forceinline__ float dot(const u32x4& a, const u32x4& b) {
  constexpr int N = 16 / (int)sizeof(T);
  typedef T vec __attribute__((ext_vector_type(N)));
  const vec x = __builtin_bit_cast(vec, a), y = __builtin_bit_cast(vec, b);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf((float)x[i], (float)y[i], s);
  return s;
}

// Past this, the rounding of lse log2(e) moves p by more than bfloat16's half step.
constexpr float kFarLse = 65536.f;
// log2 of p from a score and an lse beyond it: the score is rounded as lse was, so that equal ones leave 0.
__device__ __forceinline__ float far_exponent(float x, float scale, float lse) {
#pragma clang fp contract(off)
  const float s = x * scale;
  return (s - lse) * kLog2e;
}

template <class T, int D, int NW, int BN> struct BwdTile {
  using R = Rows<T, D>;
  static constexpr int kThreads = 64 * NW, kRows = 32 * NW;
  static constexpr int kTile = BN * R::kStride;
  static constexpr int kLds = 4 * kTile + 2 * 2 * BN * 4;             // two tiles of two tensors; lse and delta of two
};

// dq and delta: a wave owns 32 queries.
template <class T, int D, int NW, int BN>
__global__ __launch_bounds__(64 * NW, D * (int)sizeof(T) > 256 ? 1 : 2) void dq_kernel(AttnArgs a) {
  using F = BwdTile<T, D, NW, BN>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  const int heads = a.H, slot0 = (int)(blockIdx.x / heads), pair = (int)(blockIdx.x - (unsigned)slot0 * heads);
  const int rep = a.H / a.G, head = (pair % a.G) * rep + pair / a.G, group = pair % a.G;
  const Seq s = find_tile(a, slot0, F::kRows, a.causal);
  if (s.id < 0) return;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int q0 = s.tile * F::kRows, qw = q0 + w * 32, i = qw + (l & 31);
  const long long e = sizeof(T);

  u32x4 qf[R::kSteps], gf[R::kSteps];
  const int left = s.n - qw;
  hold(qf, (const char*)a.q + (s.b * a.qs.b + head * a.qs.h + (long long)(s.first + qw) * a.qs.t) * e, left, (int)(a.qs.t * e), l);
  hold(gf, (const char*)a.dout + (s.b * a.dos.b + head * a.dos.h + (long long)(s.first + qw) * a.dos.t) * e, left,
             (int)(a.dos.t * e), l);
  float delta = 0.f;
  {
    u32x4 of[R::kSteps];
    hold(of, (const char*)a.o + (s.b * a.os.b + head * a.os.h + (long long)(s.first + qw) * a.os.t) * e, left,
               (int)(a.os.t * e), l);
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) delta += dot<T>(of[k], gf[k]);
    delta = both_sum(delta);
  }
  const long long at = ((long long)s.b * a.H + head) * a.T + s.first + i;
  const float given = i < s.n ? a.lse[at] : 0.f;
  if (i < s.n && h == 0) a.delta[at] = delta;
  // scores and lse beyond kFarLse are subtracted before they go to powers of 2
  const bool far = __any(fabsf(given) > kFarLse && fabsf(given) < kInf);
  const float c = far ? 1.f : a.scale * kLog2e, lse = far ? 0.f : given * kLog2e;

  const int jend = a.causal ? min(q0 + F::kRows, s.n) : s.n;
  const int jbeg = a.window > 0 ? max(q0 - a.window + 1, 0) : 0;
  const int t0 = jbeg / BN, t1 = (jend + BN - 1) / BN;
  Stage<T, D, BN, F::kThreads> sk, sv;
  const int kst = (int)(a.ks.t * e), vst = (int)(a.vs.t * e);
  const char* kp = (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)s.first * a.ks.t) * e;
  const char* vp = (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)s.first * a.vs.t) * e;
  sk.load(kp + (long long)t0 * BN * kst, s.n - t0 * BN, kst, tid);
  sv.load(vp + (long long)t0 * BN * vst, s.n - t0 * BN, vst, tid);

  f32x16 dq[1][D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dq[0][d] = zero16();
  const int rrow = R::by_rows(l), rcol = R::transposed(l);

  for (int t = t0; t < t1; ++t) {
    char* kt = lds + (t & 1) * F::kTile;
    char* vt = kt + 2 * F::kTile;
    sk.store(kt, tid);
    sv.store(vt, tid);
    __syncthreads();
    const int j0 = t * BN;
    if (t + 1 < t1) {
      sk.load(kp + (long long)(t + 1) * BN * kst, s.n - j0 - BN, kst, tid);
      sv.load(vp + (long long)(t + 1) * BN * vst, s.n - j0 - BN, vst, tid);
    }
    if (a.causal && j0 > qw + 31) continue;
    const bool edge = j0 + BN > s.n || (a.causal && j0 + BN - 1 > qw) || (a.window > 0 && j0 <= qw + 31 - a.window);
    const int last = (a.causal ? min(i, s.n - 1) : s.n - 1) - j0 - 4 * h;
    const int first = (a.window > 0 ? i - a.window + 1 : 0) - j0 - 4 * h;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x16 x = zero16(), g = zero16();
#pragma unroll
      for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(kt + rrow + n * 32 * R::kStride + k * 32), qf[k], T());
#pragma unroll
      for (int k = 0; k < R::kSteps; ++k) mma(g, lds16(vt + rrow + n * 32 * R::kStride + k * 32), gf[k], T());
      if (far) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = far_exponent(x[r], a.scale, given);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float p = __builtin_amdgcn_exp2f(fmaf(x[r], c, -lse)) * (g[r] - delta);
        if (edge) {
          const int j = 32 * n + 8 * (r >> 2) + (r & 3);
          p = j <= last && j >= first ? p : 0.f;
        }
        x[r] = p;
      }
      Operand<T, 1> ds[1];
      ds[0].set(x);
      mul_transposed<D, 1, 1>(dq, kt + rcol + n * 32 * R::kStride, ds);
    }
  }
  if (i < s.n)
    store_columns<T, D>((char*)a.dq + (s.b * a.dqs.b + head * a.dqs.h + (long long)(s.first + i) * a.dqs.t) * e, dq[0], a.scale, h);
}

// dk and dv: a wave owns 32 keys and takes the queries of the group's heads in turn.
template <class T, int D, int NW, int BN>
__global__ __launch_bounds__(64 * NW, D * (int)sizeof(T) > 128 ? 1 : 2) void dkv_kernel(AttnArgs a) {
  using F = BwdTile<T, D, NW, BN>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  const int slot0 = (int)(blockIdx.x / (unsigned)a.G), group = (int)(blockIdx.x - (unsigned)slot0 * a.G);
  const int rep = a.H / a.G;
  const Seq s = find_tile(a, slot0, F::kRows, false);
  if (s.id < 0) return;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int j0 = s.tile * F::kRows, jw = j0 + w * 32, j = jw + (l & 31);
  const long long e = sizeof(T);

  u32x4 kf[R::kSteps], vf[R::kSteps];
  hold(kf, (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)(s.first + jw) * a.ks.t) * e, s.n - jw, (int)(a.ks.t * e), l);
  hold(vf, (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)(s.first + jw) * a.vs.t) * e, s.n - jw, (int)(a.vs.t * e), l);

  // queries ibeg .. iend - 1 of each head, in tiles t0 .. t1 - 1
  const int iend = a.window > 0 ? (int)min((long long)s.n, (long long)min(j0 + F::kRows, s.n) - 1 + a.window) : s.n;
  const int t0 = (a.causal ? j0 : 0) / BN, t1 = (iend + BN - 1) / BN, per = t1 - t0, steps = per * rep;
  float* const rows = reinterpret_cast<float*>(lds + 4 * F::kTile);   // [2][lse, delta][BN]
  Stage<T, D, BN, F::kThreads> sq, sg;
  float row = 0.f;
  const int qst = (int)(a.qs.t * e), gst = (int)(a.dos.t * e);
  const char* qp = (const char*)a.q + (s.b * a.qs.b + (long long)group * rep * a.qs.h + (long long)s.first * a.qs.t) * e;
  const char* gp = (const char*)a.dout + (s.b * a.dos.b + (long long)group * rep * a.dos.h + (long long)s.first * a.dos.t) * e;
  const auto load = [&](int head, int t) {
    const int i0 = t * BN;
    sq.load(qp + (head * a.qs.h * e + (long long)i0 * qst), s.n - i0, qst, tid);
    sg.load(gp + (head * a.dos.h * e + (long long)i0 * gst), s.n - i0, gst, tid);
    if (tid < 2 * BN) {
      const int i = i0 + (tid & (BN - 1));
      const long long at = ((long long)s.b * a.H + group * rep + head) * a.T + s.first + i;
      // past the last query p is 0
      row = i >= s.n ? (tid < BN ? kInf : 0.f) : tid < BN ? a.lse[at] : a.delta[at];
    }
  };
  load(0, t0);

  f32x16 dk[1][D / 32], dv[1][D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dk[0][d] = zero16(), dv[0][d] = zero16();
  const float c = a.scale * kLog2e;
  const int rrow = R::by_rows(l), rcol = R::transposed(l);

  int t = t0, head = 0;
  for (int step = 0; step < steps; ++step) {
    char* qt = lds + (step & 1) * F::kTile;
    char* gt = qt + 2 * F::kTile;
    float* rt = rows + (step & 1) * 2 * BN;
    sq.store(qt, tid);
    sg.store(gt, tid);
    if (tid < 2 * BN) rt[tid] = row;
    __syncthreads();
    const int i0 = t * BN;
    if (++t == t1) t = t0, ++head;
    if (step + 1 < steps) load(head, t);
    if (a.causal && i0 + BN - 1 < jw) continue;
    if (a.window > 0 && i0 > jw + 31 + (long long)a.window - 1) continue;
    const bool edge = (a.causal && i0 < jw + 31) || (a.window > 0 && i0 + BN - 1 >= jw + (long long)a.window);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x16 x = zero16(), g = zero16();
#pragma unroll
      for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(qt + rrow + n * 32 * R::kStride + k * 32), kf[k], T());
#pragma unroll
      for (int k = 0; k < R::kSteps; ++k) mma(g, lds16(gt + rrow + n * 32 * R::kStride + k * 32), vf[k], T());
      const int first = (a.causal ? j : 0) - i0 - 4 * h;
      const int last = (a.window > 0 ? (int)min((long long)j + a.window - 1, (long long)INT_MAX) : INT_MAX) - i0 - 4 * h;
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 lse = *reinterpret_cast<const f32x4*>(rt + 32 * n + 8 * r4 + 4 * h);
        // scores and lse beyond kFarLse are subtracted before they go to powers of 2
        float by = c;
        bool far = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) far |= fabsf(lse[u]) > kFarLse && fabsf(lse[u]) < kInf;
        if (__any(far)) {
#pragma unroll
          for (int u = 0; u < 4; ++u) x[4 * r4 + u] = far_exponent(x[4 * r4 + u], a.scale, lse[u]), lse[u] = 0.f;
          by = 1.f;
        } else {
          lse *= kLog2e;
        }
        const f32x4 delta = *reinterpret_cast<const f32x4*>(rt + BN + 32 * n + 8 * r4 + 4 * h);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = 4 * r4 + u;
          float p = __builtin_amdgcn_exp2f(fmaf(x[r], by, -lse[u]));
          float ds = p * (g[r] - delta[u]);
          if (edge) {
            const int i = 32 * n + 8 * r4 + u;
            const bool in = i >= first && i <= last;
            p = in ? p : 0.f;
            ds = in ? ds : 0.f;
          }
          x[r] = p;
          g[r] = ds;
        }
      }
      Operand<T, 1> p[1], ds[1];
      p[0].set(x);
      mul_transposed<D, 1, 1>(dv, gt + rcol + n * 32 * R::kStride, p);
      ds[0].set(g);
      mul_transposed<D, 1, 1>(dk, qt + rcol + n * 32 * R::kStride, ds);
    }
  }
  if (j < s.n) {
    store_columns<T, D>((char*)a.dk + (s.b * a.dks.b + group * a.dks.h + (long long)(s.first + j) * a.dks.t) * e, dk[0], a.scale, h);
    store_columns<T, D>((char*)a.dv + (s.b * a.dvs.b + group * a.dvs.h + (long long)(s.first + j) * a.dvs.t) * e, dv[0], 1.f, h);
  }
}

}  // namespace attn
}  // namespace prism
