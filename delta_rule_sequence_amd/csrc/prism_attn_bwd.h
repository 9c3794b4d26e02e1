// prism_attn_bwd.h - softmax attention of a prompt's rows (gfx950), backward.
//
//   p_ij = e^(s_ij - lse_i),  dp_ij = <do_i, v_j>,  ds_ij = p_ij (dp_ij - <do_i, o_i>)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij do_i   (i over the group's heads)
//
// Two kernels form the tiles of s and dp once each, so that every sum stays in one wave's registers and has a fixed order
// (seven products where five would do with sums across workgroups): dq by queries, with the forward's transposed tiles;
// dk and dv by keys, with tiles whose columns are keys.
//
// Rounding: p and ds pass as one bfloat16 part each, as in the forward: gradients are off by 0.0024 of their size where float32
// products would leave 0.0018.  The tiles' scores and their lse come from the same products as the forward's.
//
// Bounds, bfloat16: 8 x 12 x 2048 of 64, causal, 234 us (dq 95, dk and dv 135): the matrix cores are busy for 0.31 of the cycles at
// 2.4 GHz, the vector instructions of the exponentials, of ds and of the two roundings for about as many, and the two overlap in part only;
// reads from LDS are not what bounds it (a spacing without conflicts for dq's values: equal).  4 x 16 x 4096 of 128: 1077 us, 638 TFLOP/s
// of the five products that are needed, 890 of the seven formed.  dk and dv in two kernels: 1195 to 1545 us there; the next
// tile's products ahead in dkv of 128: 1137.
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
__device__ __forceinline__ bool is_far(float lse) { return fabsf(lse) > kFarLse && fabsf(lse) < kInf; }
// log2 of p from a score and an lse beyond it: the score is rounded as lse was, so that equal ones leave 0.
__device__ __forceinline__ float far_exponent(float x, float scale, float lse) {
#pragma clang fp contract(off)
  const float s = x * scale;
  return (s - lse) * kLog2e;
}

template <class T, int D, int NW, int BN, bool AHEAD> struct BwdTile {
  using R = Rows<T, D>;
  static constexpr int kThreads = 64 * NW, kRows = 32 * NW;
  static constexpr int kTile = BN * R::kStride;
  // AHEAD: the next rows' two products are formed beside these rows' exponentials, so a tile is in LDS one step ahead.
  static constexpr bool kAhead = AHEAD;
  static constexpr int kTiles = kAhead ? 3 : 2;
  static constexpr int kRowsAt = 2 * kTiles * kTile;                  // of two tensors; then lse log2(e), delta and lse; zeros
  static constexpr int kLds = kRowsAt + (kTiles * 3 + 1) * BN * 4;
};
// OW x SW waves: OW own 32 rows each, SW take a tile's rows by turns.
template <class T, int D, int OW, int SW, int BN, bool AHEAD> struct Pass : BwdTile<T, D, OW * SW, BN, AHEAD> {
  static constexpr int kOwn = 32 * OW;
  static_assert(BN % (32 * SW) == 0, "every wave has rows of a tile");
  static_assert((SW - 1) * OW * 32 * (D + 4) * 4 <= Pass::kLds, "a join fits");
};

// The sums of the waves that own the same rows, in their order, in the first one's registers.
template <int D, int OW, int SW>
__device__ __forceinline__ void join_waves(f32x16 (&acc)[D / 32], char* lds, int ow, int sw) {
  const int l = lane_id(), h = l >> 5;
  __syncthreads();
  float* const rows = reinterpret_cast<float*>(lds) + (l & 31) * (D + 4);
  if (sw > 0) store_columns<float, D>(reinterpret_cast<char*>(rows + ((sw - 1) * OW + ow) * 32 * (D + 4)), acc, 1.f, h);
  __syncthreads();
  if (sw > 0) return;
  for (int o = 0; o < SW - 1; ++o)
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(rows + (o * OW + ow) * 32 * (D + 4) + 32 * d + 8 * r + 4 * h);
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[d][4 * r + u] += y[u];
      }
}

// dq and delta: OW waves of 32 queries, SW that take a tile's keys by turns.
template <class T, int D, int OW, int SW, int BN, bool AHEAD>
__global__ __launch_bounds__(64 * OW * SW, SW > 1 || D * (int)sizeof(T) > 256 ? 1 : 2) void dq_kernel(AttnArgs a) {
  using F = Pass<T, D, OW, SW, BN, AHEAD>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  const int rep = a.H / a.G;
  const Seq s = find_tile(a, blockIdx.x, F::kOwn, rep, a.causal);
  if (s.id < 0) return;
  const int group = s.group, head = group * rep + s.head;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id()), ow = w % OW, sw = w / OW;
  const int q0 = s.tile * F::kOwn, qw = q0 + ow * 32, i = qw + (l & 31);
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
  if (i < s.n && h == 0 && sw == 0) a.delta[at] = delta;
  const bool far = __any(is_far(given));                              // then the exponents are formed by themselves
  const float scale = a.scale * kLog2e, c = far ? 1.f : scale, lse = far ? 0.f : given * kLog2e;

  const int jend = a.causal ? min(q0 + F::kOwn, s.n) : s.n;
  const int jbeg = a.window > 0 ? max(q0 - a.window + 1, 0) : 0;
  const int t0 = jbeg / BN, t1 = (jend + BN - 1) / BN;
  Stage<T, D, BN, F::kThreads> sk, sv;
  const int kst = (int)(a.ks.t * e), vst = (int)(a.vs.t * e);
  const char* kp = (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)s.first * a.ks.t) * e;
  const char* vp = (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)s.first * a.vs.t) * e;
  const auto load = [&](int t) {
    sk.load(kp + (long long)t * BN * kst, s.n - t * BN, kst, tid);
    sv.load(vp + (long long)t * BN * vst, s.n - t * BN, vst, tid);
  };
  constexpr int M = NT / SW;                                          // a tile's parts of a wave
  static_assert(!F::kAhead || M % 2 == 0, "two halves by turns");
  char* const v_tiles = lds + F::kTiles * F::kTile;
  const auto store = [&](int place) {
    sk.store(lds + place * F::kTile, tid);
    sv.store(v_tiles + place * F::kTile, tid);
  };

  f32x16 dq[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dq[d] = zero16();
  const int rrow = R::by_rows(l), rcol = R::transposed(l);
  const int last = a.causal ? min(i, s.n - 1) : s.n - 1, first = a.window > 0 ? i - a.window + 1 : 0;
  const int wlast = a.causal ? min(qw + 31, s.n - 1) : s.n - 1;
  f32x16 xs[F::kAhead ? 2 : 1], gs[F::kAhead ? 2 : 1];                // s and dp of these 32 keys, and of the next
  const auto products = [&](f32x16& x, f32x16& g, int at) {
    x = zero16(), g = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(lds + at + rrow + k * 32), qf[k], T());
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(g, lds16(v_tiles + at + rrow + k * 32), gf[k], T());
  };

  load(t0);
  int place = 0;                                                      // tile t's in LDS
  if constexpr (F::kAhead) {
    store(0);
    if (t0 + 1 < t1) {
      load(t0 + 1);
      store(1);
    }
    if (t0 + 2 < t1) load(t0 + 2);
    __syncthreads();
    products(xs[0], gs[0], sw * 32 * R::kStride);
  }
  const auto stage = [&](int t, int next) {
    if (t > t0) __syncthreads();
    if (t + 2 < t1) store(next + 1 == F::kTiles ? 0 : next + 1);
    if (t + 3 < t1) load(t + 3);
  };
  int t = t0;
  if constexpr (F::kAhead) {
    // Tiles in front of all of the wave's windows stay out of its sums: a key that is not finite, times a p of 0, would enter
    // rows of the workgroup's last waves, up to 318 tokens behind the last one that sees it.
    const int own = a.window > 0 ? min(max(qw - a.window + 1, 0) / BN, t1) : t0;
    for (; t < own; ++t) {
      const int next = place + 1 == F::kTiles ? 0 : place + 1;
      stage(t, next);
      place = next;
      if (t + 1 == own && own < t1) products(xs[0], gs[0], place * F::kTile + sw * 32 * R::kStride);
    }
  }
  for (; t < t1; ++t) {
    int next = place + 1 == F::kTiles ? 0 : place + 1;
    if constexpr (F::kAhead) {
      stage(t, next);
    } else {
      store(place);
      __syncthreads();
      if (t + 1 < t1) load(t + 1);
    }
    const int at = place * F::kTile, after = next * F::kTile;
    place = next;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int n = m * SW + sw, j0 = t * BN + 32 * n, here = at + n * 32 * R::kStride;
      if (j0 > wlast) break;                                          // nothing for this wave's queries
      f32x16 &x = xs[F::kAhead ? m & 1 : 0], &g = gs[F::kAhead ? m & 1 : 0];
      if constexpr (!F::kAhead) products(x, g, here);
      const bool edge = j0 + 31 > (a.causal ? min(qw, s.n - 1) : s.n - 1) || (a.window > 0 && j0 <= qw + 31 - a.window);
      if (edge || far) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = 8 * (r >> 2) + (r & 3) + j0 + 4 * h;
          const bool in = j <= last && j >= first;
          if (far) x[r] = is_far(given) ? far_exponent(x[r], a.scale, given) : fmaf(x[r], scale, -given * kLog2e);
          x[r] = in ? x[r] : -kInf;
          g[r] = in ? g[r] : 0.f;
        }
      }
      if constexpr (F::kAhead)
        products(xs[(m + 1) & 1], gs[(m + 1) & 1], m + 1 < M ? here + SW * 32 * R::kStride : after + sw * 32 * R::kStride);
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], c, -lse)) * (g[r] - delta);
      Operand<T, 1> ds;
      ds.set(x);
      mul_transposed<D, 1>(dq, lds + here + rcol, ds);
    }
  }
  if constexpr (SW > 1) join_waves<D, OW, SW>(dq, lds, ow, sw);
  if (i < s.n && sw == 0)
    store_columns<T, D>((char*)a.dq + (s.b * a.dqs.b + head * a.dqs.h + (long long)(s.first + i) * a.dqs.t) * e, dq, a.scale, h);
}

// dk and dv: KW waves of 32 keys, QW that take a tile's queries by turns; the heads of the group one after the other.
template <class T, int D, int KW, int QW, int BN, bool AHEAD>
__global__ __launch_bounds__(64 * KW * QW, D * (int)sizeof(T) > 128 ? 1 : 2) void dkv_kernel(AttnArgs a) {
  using F = Pass<T, D, KW, QW, BN, AHEAD>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  // the heads of a group go to a.splits workgroups
  const unsigned unit = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - unit * a.splits;
  const int rep = a.H / a.G, each = (rep + a.splits - 1) / a.splits, h0 = min((int)split * each, rep), h1 = min(h0 + each, rep);
  const Seq s = find_tile(a, unit, F::kOwn, 1, false);
  if (s.id < 0) return;
  const int group = s.group;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id()), kw = w % KW, qw = w / KW;
  const int j0 = s.tile * F::kOwn, jw = j0 + kw * 32, j = jw + (l & 31);
  const long long e = sizeof(T);

  u32x4 kf[R::kSteps], vf[R::kSteps];
  hold(kf, (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)(s.first + jw) * a.ks.t) * e, s.n - jw, (int)(a.ks.t * e), l);
  hold(vf, (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)(s.first + jw) * a.vs.t) * e, s.n - jw, (int)(a.vs.t * e), l);

  // queries ibeg .. iend - 1 of each head, in tiles t0 .. t1 - 1
  const int iend = a.window > 0 ? (int)min((long long)s.n, (long long)min(j0 + F::kOwn, s.n) - 1 + a.window) : s.n;
  const int t0 = (a.causal ? j0 : 0) / BN, t1 = (iend + BN - 1) / BN, steps = (t1 - t0) * (h1 - h0);
  float* const rows = reinterpret_cast<float*>(lds + F::kRowsAt);     // [kTiles][lse log2(e), delta, lse][BN], zeros [BN]
  float* const zeros = rows + F::kTiles * 3 * BN;
  if (tid < BN) zeros[tid] = 0.f;
  Stage<T, D, BN, F::kThreads> sq, sg;
  float row = 0.f;
  const int qst = (int)(a.qs.t * e), gst = (int)(a.dos.t * e);
  const char* qp = (const char*)a.q + (s.b * a.qs.b + (long long)group * rep * a.qs.h + (long long)s.first * a.qs.t) * e;
  const char* gp = (const char*)a.dout + (s.b * a.dos.b + (long long)group * rep * a.dos.h + (long long)s.first * a.dos.t) * e;
  int lt = t0, lh = h0;                                               // the tile that is loaded next, and its head
  const auto load = [&]() {
    const int i0 = lt * BN;
    sq.load(qp + (lh * a.qs.h * e + (long long)i0 * qst), s.n - i0, qst, tid);
    sg.load(gp + (lh * a.dos.h * e + (long long)i0 * gst), s.n - i0, gst, tid);
    if (tid < 2 * BN) {
      const int i = i0 + (tid & (BN - 1));
      const long long at = ((long long)s.b * a.H + group * rep + lh) * a.T + s.first + i;
      // past the last query p is 0
      row = i >= s.n ? (tid < BN ? kInf : 0.f) : tid < BN ? a.lse[at] : a.delta[at];
    }
    if (++lt == t1) lt = t0, ++lh;
  };
  char* const g_tiles = lds + F::kTiles * F::kTile;
  const auto store = [&](int place) {
    sq.store(lds + place * F::kTile, tid);
    sg.store(g_tiles + place * F::kTile, tid);
    float* const rt = rows + place * 3 * BN;
    if (tid < 2 * BN) rt[tid] = tid < BN ? row * kLog2e : row;
    if (tid < BN) rt[2 * BN + tid] = row;
  };

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dk[d] = zero16(), dv[d] = zero16();
  const float scale = a.scale * kLog2e;
  const int rrow = R::by_rows(l), rcol = R::transposed(l);
  f32x16 xs[F::kAhead ? 2 : 1], gs[F::kAhead ? 2 : 1];                // s and dp of these 32 queries, and of the next
  const auto products = [&](f32x16& x, f32x16& g, int at) {
    x = zero16(), g = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(lds + at + rrow + k * 32), kf[k], T());
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(g, lds16(g_tiles + at + rrow + k * 32), vf[k], T());
  };

  constexpr int M = NT / QW;                                          // a tile's parts of a wave
  static_assert(!F::kAhead || M % 2 == 0, "two halves by turns");
  int place = 0;                                                      // this step's tile in LDS
  if (steps > 0) load();
  if constexpr (F::kAhead) {
    if (steps > 0) store(0);
    if (steps > 1) {
      load();
      store(1);
    }
    if (steps > 2) load();
    __syncthreads();
    products(xs[0], gs[0], qw * 32 * R::kStride);
  }
  int t = t0;
  for (int step = 0; step < steps; ++step) {
    const int next = place + 1 == F::kTiles ? 0 : place + 1;
    if constexpr (F::kAhead) {
      if (step > 0) __syncthreads();
      if (step + 2 < steps) store(next + 1 == F::kTiles ? 0 : next + 1);
      if (step + 3 < steps) load();
    } else {
      store(place);
      __syncthreads();
      if (step + 1 < steps) load();
    }
    const int i0 = t * BN, tile = place * F::kTile, after = next * F::kTile;
    const float* const rt = rows + place * 3 * BN;
    place = next;
    if (++t == t1) t = t0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int n = m * QW + qw, i1 = i0 + 32 * n, at = tile + n * 32 * R::kStride;
      const int at1 = m + 1 < M ? at + QW * 32 * R::kStride : after + qw * 32 * R::kStride;
      f32x16 &x = xs[F::kAhead ? m & 1 : 0], &g = gs[F::kAhead ? m & 1 : 0];
      if constexpr (!F::kAhead)
        if ((a.causal && i1 + 31 < jw) || (a.window > 0 && i1 > jw + 31 + (long long)a.window - 1)) continue;
      if constexpr (!F::kAhead) products(x, g, at);
      const bool edge = (a.causal && i1 < jw + 31) || (a.window > 0 && i1 + 31 >= jw + (long long)a.window);
      const bool far = __any(is_far(rt[2 * BN + 32 * n + (l & 31)]));  // then the exponents are formed by themselves
      const float c = far ? 1.f : scale;
      const float* const lse2 = far ? zeros : rt;
      if (edge || far) {
        const int first = (a.causal ? j : 0) - i1 - 4 * h;
        const int last = (a.window > 0 ? (int)min((long long)j + a.window - 1, (long long)INT_MAX) : INT_MAX) - i1 - 4 * h;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int i = 8 * (r >> 2) + (r & 3);
          const bool in = i >= first && i <= last;
          if (far) {
            const float lse = rt[2 * BN + 32 * n + i + 4 * h];
            x[r] = is_far(lse) ? far_exponent(x[r], a.scale, lse) : fmaf(x[r], scale, -rt[32 * n + i + 4 * h]);
          }
          x[r] = in ? x[r] : -kInf;
          g[r] = in ? g[r] : 0.f;
        }
      }
      if constexpr (F::kAhead) products(xs[(m + 1) & 1], gs[(m + 1) & 1], at1);
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const f32x4 lse = *reinterpret_cast<const f32x4*>(lse2 + 32 * n + 8 * r4 + 4 * h);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(rt + BN + 32 * n + 8 * r4 + 4 * h);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = 4 * r4 + u;
          x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], c, -lse[u]));
          g[r] = x[r] * (g[r] - delta[u]);
        }
      }
      Operand<T, 1> p;
      p.set(x);
      mul_transposed<D, 1>(dv, g_tiles + at + rcol, p);
      p.set(g);
      mul_transposed<D, 1>(dk, lds + at + rcol, p);
    }
  }
  if constexpr (QW > 1) {
    join_waves<D, KW, QW>(dk, lds, kw, qw);
    join_waves<D, KW, QW>(dv, lds, kw, qw);
  }
  if (j >= s.n || qw > 0) return;
  if (a.splits > 1) {                                                 // [splits][dk, dv][B G T][D], added up by sum_kernel
    const size_t all = (size_t)a.B * a.G * a.T, at = ((size_t)s.b * a.G + group) * a.T + s.first + j;
    store_columns<float, D>((char*)(a.part + ((2 * split) * all + at) * D), dk, a.scale, h);
    store_columns<float, D>((char*)(a.part + ((2 * split + 1) * all + at) * D), dv, 1.f, h);
    return;
  }
  store_columns<T, D>((char*)a.dk + (s.b * a.dks.b + group * a.dks.h + (long long)(s.first + j) * a.dks.t) * e, dk, a.scale, h);
  store_columns<T, D>((char*)a.dv + (s.b * a.dvs.b + group * a.dvs.h + (long long)(s.first + j) * a.dvs.t) * e, dv, 1.f, h);
}

// dk and dv from the shares of the heads: D / 4 lanes per row of one of them, tokens of the sequences only.
template <class T, int D>
__global__ __launch_bounds__(256) void sum_kernel(AttnArgs a) {
  constexpr int L = D / 4;
  const size_t all = (size_t)a.B * a.G * a.T, row = (size_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= 2 * all) return;
  const bool of_v = row >= all;
  const size_t r = of_v ? row - all : row, bg = r / a.T;
  const int at = threadIdx.x % L * 4, t = (int)(r - bg * a.T), b = (int)(bg / a.G), g = (int)(bg - (size_t)b * a.G);
  if (a.starts != nullptr) {
    if (t < a.starts[0] || t >= a.starts[a.S]) return;
  } else if (a.lens != nullptr && t >= a.lens[b]) {
    return;
  }
  f32x4 y = zero4();
  for (int k = 0; k < a.splits; ++k) y += *reinterpret_cast<const f32x4*>(a.part + ((2 * k + of_v) * all + r) * D + at);
  T z[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) z[u] = (T)y[u];
  const prism_strides st = of_v ? a.dvs : a.dks;
  __builtin_memcpy((char*)(of_v ? a.dv : a.dk) + (b * st.b + g * st.h + (long long)t * st.t + at) * (long long)sizeof(T), z, sizeof(z));
}

}  // namespace attn
}  // namespace prism
