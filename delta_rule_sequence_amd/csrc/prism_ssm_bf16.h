// prism_ssm_bf16.h - the selective state space scan of bfloat16 tensors on the bf16 matrix instructions (gfx950).
//
// The chunked form and the passes of prism_ssm.h with 16x16x32 bf16 MFMA tiles and float32 sums.  Which operands are
// rounded:
//   * x, B, C, dy are bfloat16 already: C B^T and dy x^T have exact operands;
//   * what enters a state (decay-weighted x or dy) is split into three bfloat16 parts that together hold its 24 bits,
//     so states keep float32 accuracy over any length (three MFMAs in place of one);
//   * the score matrix M, the state as it is read out into y, the summed score gradients and R in dx are rounded to
//     bfloat16 once: each is one rounding of 2^-9 on average in a result that is itself rounded to bfloat16;
//   * ddt and dA are float32 results: H and R enter the products behind them as two parts (16 bits).
//
// Waves own 16 columns p of the state in MFMA accumulators from chunk to chunk; an accumulator tile is the operand of
// the readout without passing LDS (rows of a tile pair are the k values of one MFMA, in the order of Mma::koff).
// Tiles lie in LDS without padding, their 16-byte pieces permuted inside a row (Tile::at) so that row reads and
// transposing reads both touch all banks evenly.
#pragma once
#include "prism_ssm.h"

namespace prism {
namespace ssm {
namespace mx {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// A bfloat16 matrix in LDS, W columns.  Piece c (8 values) of row r lies at position c ^ swz(r): the 16 rows of a row
// read (one piece each) and the 8 rows of a transposing read (two pieces each) then fall on different banks.
template <int W>
struct Tile {
  static constexpr int C = W / 8, LW = W == 128 ? 0 : W == 64 ? 1 : W == 32 ? 2 : 3;
  static __device__ __forceinline__ int swz(int r) { return (((r >> LW) & (C / 2 - 1)) << 1) | ((r >> 3) & 1); }
  static __device__ __forceinline__ int at(int r, int c) { return r * W + (((c >> 3) ^ swz(r)) << 3) + (c & 7); }
};

// k blocks of a product over W values: 32 each, the only one of W = 16 half empty
template <int W> constexpr int kblocks() { return W < 32 ? 1 : W / 32; }

// Operand fragments.  frag_n: index = row, k natural (8 g + j; W >= 32).  frag_o: index = row, k in koff order.
// frag_t: index = column, k = row, koff order (gfx950 transposing LDS reads).
template <int W>
__device__ __forceinline__ bf16x8 frag_n(const bf16_t* t, int row0, int k0) {
  const int l = lane_id();
  return *reinterpret_cast<const bf16x8*>(t + Tile<W>::at(row0 + (l & 15), k0 + 8 * (l >> 4)));
}
template <int W>
__device__ __forceinline__ bf16x8 frag_o(const bf16_t* t, int row0, int k0) {
  const int l = lane_id(), r = row0 + (l & 15), k = k0 + 4 * (l >> 4);
  const bf16x4 lo = *reinterpret_cast<const bf16x4*>(t + Tile<W>::at(r, k));
  bf16x4 hi = {0, 0, 0, 0};
  if constexpr (W >= 32) hi = *reinterpret_cast<const bf16x4*>(t + Tile<W>::at(r, k + 16));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int W>
__device__ __forceinline__ bf16x8 frag_row(const bf16_t* t, int row0, int k0) {  // any k order, the same on both sides
  if constexpr (W >= 32) return frag_n<W>(t, row0, k0);
  else return frag_o<W>(t, row0, k0);
}
template <int W>
__device__ __forceinline__ bf16x8 frag_t(const bf16_t* t, int k0, int col0) {
  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
  const int l = lane_id(), i = l & 15, r = k0 + 4 * (l >> 4) + (i >> 2), c = col0 + 4 * (i & 3);
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(const_cast<bf16_t*>(t + Tile<W>::at(r, c))));
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(const_cast<bf16_t*>(t + Tile<W>::at(r + 16, c))));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ unsigned bits(float v) { return __builtin_bit_cast(unsigned, v); }
__device__ __forceinline__ float val(unsigned v) { return __builtin_bit_cast(float, v); }
// the upper halves of two floats as two bfloat16 (truncation)
__device__ __forceinline__ unsigned pack_hi(float a, float b) { return __builtin_amdgcn_perm(bits(b), bits(a), 0x07060302u); }

// v = p[0] + p[1] + p[2] exactly for finite v that do not underflow: each part takes the next 8 bits.
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8 (&p)[3]) {
  u32x4 q[3];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a = v[2 * k], b = v[2 * k + 1];
    q[0][k] = pack_hi(a, b);
    a -= val(bits(a) & 0xffff0000u), b -= val(bits(b) & 0xffff0000u);
    q[1][k] = pack_hi(a, b);
    a -= val(bits(a) & 0xffff0000u), b -= val(bits(b) & 0xffff0000u);
    q[2][k] = pack_hi(a, b);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) p[k] = __builtin_bit_cast(bf16x8, q[k]);
}

// Two state tiles (k values of one block) as an operand, rounded to nearest; the second is absent for W = 16.
__device__ __forceinline__ bf16x8 round8(const f32x4& a, const f32x4& b) {
  bf16x8 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    o[r] = (bf16_t)a[r];
    o[4 + r] = (bf16_t)b[r];
  }
  return o;
}

// Rows t0 .. t0 + 63 of a strided [T, W] tensor on the way from memory to an LDS tile: loaded into registers early, stored
// when the tile is free.  Rows at or past len are 0.
template <int W, int NTH>
struct Stage {
  static constexpr int NV = Q * W / 8, PER = (NV + NTH - 1) / NTH;
  bf16x8 v[PER];
  __device__ __forceinline__ void load(const bf16_t* p, long long st, int t0, int len) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = threadIdx.x + k * NTH, t = t0 + i / (W / 8);
      v[k] = bf16x8(0);
      if ((NV % NTH == 0 || i < NV) && t < len) v[k] = *reinterpret_cast<const bf16x8*>(p + (long long)t * st + i % (W / 8) * 8);
    }
  }
  __device__ __forceinline__ void store(bf16_t* tile) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = threadIdx.x + k * NTH;
      if (NV % NTH == 0 || i < NV) *reinterpret_cast<bf16x8*>(tile + Tile<W>::at(i / (W / 8), i % (W / 8) * 8)) = v[k];
    }
  }
};

__device__ __forceinline__ float decay(const Scal& s, int t, int r) {  // e^{c_t - c_r}
  return __builtin_amdgcn_exp2f((s.ch[t] - s.ch[r]) + (s.cl[t] - s.cl[r]));
}

// The decay-weighted rows of V (index = column p0 .., k = token) in three parts: weight wa[k] (times wb[k]).
template <int W>
__device__ __forceinline__ void weighted(bf16x8 (&p)[3], const bf16_t* tile, int k0, int p0, const float* wa, const float* wb) {
  const int g4 = 4 * (lane_id() >> 4);
  const bf16x8 f = frag_t<W>(tile, k0, p0);
  float v[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float a = wa[k0 + g4 + r], b = wa[k0 + 16 + g4 + r];
    if (wb != nullptr) a *= wb[k0 + g4 + r], b *= wb[k0 + 16 + g4 + r];
    v[r] = (float)f[r] * a;
    v[4 + r] = (float)f[4 + r] * b;
  }
  split3(v, p);
}

// Piece of a saved state: H^T tile (pt, nt) is half of the 8 k = p values of lane (g, n) in block pt / 2, for the products
// that contract over p.  Two planes (parts) of N * PW bfloat16 each.
template <int N, int PW>
__device__ __forceinline__ size_t plane_at(int pt, int nt) {
  if constexpr (PW == 16) return ((size_t)nt * 64 + lane_id()) * 4;
  else return (((size_t)nt * (PW / 32) + (pt >> 1)) * 64 + lane_id()) * 8 + (pt & 1) * 4;
}

// States of a segment, as ssm::state_kernel.  SAVE = false (H: rows n, columns p, as the sweep keeps it; or, for the
// backward, transposed): from zero, the end state to seg.  SAVE = true: from the entering state, saving the state in
// front of every chunk in two planes.
template <int N, int PW, bool TRANS, bool SAVE>
__global__ __launch_bounds__(PW * 4) void state_kernel(SsmArgs a) {
  constexpr int NTH = PW * 4, NW = PW / 16, NT = N / 16;
  __shared__ __attribute__((aligned(16))) bf16_t sA[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sV[Q * PW];
  __shared__ Scal scal[NW];
  const int seg = blockIdx.x, bh = blockIdx.y, rev = blockIdx.z;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW, grp = h / (a.H / a.G);
  const int len = seq_len(a, b), pt = wave_id(), tid = threadIdx.x;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nch);
  const size_t slot = ((size_t)rev * gridDim.y + bh) * a.nseg + seg;
  const bf16_t *pa, *pv;
  long long ta, tv;
  if (rev) {
    pa = (const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h, ta = a.cs.t;
    pv = (const bf16_t*)a.dy + b * a.dys.b + h * a.dys.h + p0, tv = a.dys.t;
  } else {
    pa = (const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h, ta = a.bs.t;
    pv = (const bf16_t*)a.x + b * a.xs.b + h * a.xs.h + p0, tv = a.xs.t;
  }
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    acc[n] = SAVE ? *reinterpret_cast<const f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(pt, n)) : zero4();
  // chunks that hold tokens, in walking order
  const int live = min(c1, (len + Q - 1) / Q) - c0, steps = SAVE ? c1 - c0 : max(live, 0);
  Stage<N, NTH> la;
  Stage<PW, NTH> lv;
  if (steps > 0) {
    const int t0 = (rev ? c1 - 1 : c0) * Q;
    la.load(pa, ta, t0, len);
    lv.load(pv, tv, t0, len);
  }
  double log_dec = 0.0;
  for (int k = 0; k < steps; ++k) {
    const int ch = rev ? c1 - 1 - k : c0 + k;
    __syncthreads();
    la.store(sA);
    lv.store(sV);
    if (k % NW == 0) {  // the next NW chunks' scalars, one wave each
      const int kk = k + wave_id();
      if (kk < steps) log_dec += chunk_scalars(a, b, h, (rev ? c1 - 1 - kk : c0 + kk) * Q, len, scal[wave_id()]);
    }
    if (k + 1 < steps) {
      const int t0 = (rev ? ch - 1 : ch + 1) * Q;
      la.load(pa, ta, t0, len);
      lv.load(pv, tv, t0, len);
    }
    if constexpr (SAVE) {
      bf16_t* st = reinterpret_cast<bf16_t*>(a.st) + (((size_t)rev * gridDim.y + bh) * a.nch + ch) * (2 * N * PW);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        bf16x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          hi[r] = (bf16_t)acc[n][r];
          lo[r] = (bf16_t)(acc[n][r] - (float)hi[r]);
        }
        *reinterpret_cast<bf16x4*>(st + plane_at<N, PW>(pt, n)) = hi;
        *reinterpret_cast<bf16x4*>(st + N * PW + plane_at<N, PW>(pt, n)) = lo;
      }
    }
    __syncthreads();
    const Scal& sc = scal[k % NW];
    const float dec = sc.dec;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] *= dec;
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 32) {
      bf16x8 f[3];
      weighted<PW>(f, sV, k0, 16 * pt, rev ? sc.eo : sc.w, rev ? nullptr : sc.d);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bf16x8 fa = frag_t<N>(sA, k0, 16 * n);
#pragma unroll
        for (int q = 2; q >= 0; --q) acc[n] = TRANS ? mfma(f[q], fa, acc[n]) : mfma(fa, f[q], acc[n]);
      }
    }
  }
  if constexpr (!SAVE) {
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(pt, n)) = acc[n];
    // the waves' shares of the segment's log decay
    __shared__ double part[NW];
    if (lane_id() == 0) part[wave_id()] = log_dec;
    __syncthreads();
    if (rev == 0 && tid == 0) {
      double s = part[0];
#pragma unroll
      for (int k = 1; k < NW; ++k) s += part[k];
      a.seg_dec[(size_t)bh * a.nseg + seg] = exp2f((float)s);
    }
  }
}

// The scan over segments (see ssm::seg_scan_kernel); TRANS: which way the tiles lie.
template <int N, int PW, bool TRANS>
__global__ __launch_bounds__(256) void seg_scan_kernel(SsmArgs a, int has_end) {
  const int e = blockIdx.x * 256 + threadIdx.x, bh = blockIdx.y, rev = blockIdx.z;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW;
  const int tile = e >> 8, row = ((e >> 6) & 3) * 4 + (e & 3), col = (e >> 2) & 15;  // position inside a 16 x 16 tile
  const int p = tile / (N / 16) * 16 + (TRANS ? row : col), n = tile % (N / 16) * 16 + (TRANS ? col : row);
  const float* init = rev ? a.dS : a.S0;
  float v = init != nullptr ? init[((size_t)(b * a.H + h) * N + n) * a.P + p0 + p] : 0.f;
  float* q = a.seg + ((size_t)rev * gridDim.y + bh) * a.nseg * (N * PW) + e;
  for (int k = 0; k < a.nseg; ++k) {
    const int s = rev ? a.nseg - 1 - k : k;
    const float own = has_end ? q[(size_t)s * (N * PW)] : 0.f;
    q[(size_t)s * (N * PW)] = v;
    if (has_end) v = a.seg_dec[(size_t)bh * a.nseg + s] * v + own;
  }
}

// Outputs of a segment from its entering state, as ssm::sweep_kernel.  y tiles are formed transposed (rows p, columns t), so
// that a lane stores 4 neighbouring columns.
template <int N, int PW>
__global__ __launch_bounds__(PW * 4) void sweep_kernel(SsmArgs a) {
  constexpr int NTH = PW * 4, NW = PW / 16, NT = N / 16, KN = kblocks<N>();
  __shared__ __attribute__((aligned(16))) bf16_t sB[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sC[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sX[Q * PW];
  __shared__ __attribute__((aligned(16))) bf16_t sM[Q * Q];
  __shared__ Scal scal[NW];
  const int seg = blockIdx.x, bh = blockIdx.y;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW, grp = h / (a.H / a.G);
  const int len = seq_len(a, b), pt = wave_id(), l = lane_id(), g = l >> 4, i = l & 15;
  const int c0 = seg * a.seg_chunks, steps = min(min(c0 + a.seg_chunks, a.nch), (len + Q - 1) / Q) - c0;
  const float Dh = a.D != nullptr ? a.D[h] : 0.f;
  const size_t gstate = ((size_t)(b * a.H + h) * N) * a.P + p0 + 16 * pt;
  const bf16_t* pb = (const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h;
  const bf16_t* pc = (const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h;
  const bf16_t* px = (const bf16_t*)a.x + b * a.xs.b + h * a.xs.h + p0;
  bf16_t* py = (bf16_t*)a.y + b * a.ys.b + h * a.ys.h + p0 + 16 * pt + 4 * g;
  Stage<N, NTH> lb, lc;
  Stage<PW, NTH> lx;
  if (steps > 0) {
    lb.load(pb, a.bs.t, c0 * Q, len);
    lc.load(pc, a.cs.t, c0 * Q, len);
    lx.load(px, a.xs.t, c0 * Q, len);
  }
  // state tiles: rows n = 16 nt + 4 g + r, column p = 16 pt + i
  f32x4 hs[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (a.nseg > 1) {
      hs[n] = *reinterpret_cast<const f32x4*>(a.seg + ((size_t)bh * a.nseg + seg) * (N * PW) + tile_at<N>(pt, n));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        hs[n][r] = a.S0 != nullptr ? a.S0[gstate + (size_t)(16 * n + 4 * g + r) * a.P + i] : 0.f;
    }
  }
  // score tiles above the diagonal that share a k block with one on it
  for (int k = threadIdx.x; k < 2 * 16 * 16; k += NTH) {
    const int blk = k >> 8, r = (k >> 4) & 15, c = k & 15;
    sM[Tile<Q>::at(32 * blk + r, 32 * blk + 16 + c)] = (bf16_t)0.f;
  }
  for (int k = 0; k < steps; ++k) {
    const int t0 = (c0 + k) * Q;
    __syncthreads();
    lb.store(sB);
    lc.store(sC);
    lx.store(sX);
    if (k % NW == 0 && k + wave_id() < steps) chunk_scalars(a, b, h, (c0 + k + wave_id()) * Q, len, scal[wave_id()]);
    if (k + 1 < steps) {
      lb.load(pb, a.bs.t, t0 + Q, len);
      lc.load(pc, a.cs.t, t0 + Q, len);
      lx.load(px, a.xs.t, t0 + Q, len);
    }
    __syncthreads();
    const Scal& sc = scal[k % NW];
    // M, tile (ts, tt): rows s, columns t
    for (int idx = wave_id(); idx < 10; idx += NW) {
      int tt = 0, ts = idx;
      while (ts > tt) ts -= ++tt;
      f32x4 acc = zero4();
#pragma unroll
      for (int n = 0; n < KN; ++n) acc = mfma(frag_row<N>(sB, 16 * ts, 32 * n), frag_row<N>(sC, 16 * tt, 32 * n), acc);
      const int t = 16 * tt + i;
      bf16x4 m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int s = 16 * ts + 4 * g + r;
        m[r] = (bf16_t)(s <= t ? acc[r] * (decay(sc, t, s) * sc.d[s]) : 0.f);
      }
      *reinterpret_cast<bf16x4*>(sM + Tile<Q>::at(t, 16 * ts + 4 * g)) = m;
    }
    bf16x8 hf[KN];
#pragma unroll
    for (int n = 0; n < KN; ++n) hf[n] = round8(hs[2 * n < NT ? 2 * n : 0], 2 * n + 1 < NT ? hs[2 * n + 1 < NT ? 2 * n + 1 : 0] : zero4());
    __syncthreads();
#pragma unroll
    for (int tt = 0; tt < Q / 16; ++tt) {
      const int t = 16 * tt + i;
      f32x4 acc = zero4();
#pragma unroll
      for (int n = 0; n < KN; ++n) acc = mfma(hf[n], frag_o<N>(sC, 16 * tt, 32 * n), acc);
      acc *= sc.eo[t];
#pragma unroll
      for (int kb = 0; kb <= tt / 2; ++kb) acc = mfma(frag_t<PW>(sX, 32 * kb, 16 * pt), frag_o<Q>(sM, 16 * tt, 32 * kb), acc);
      const bf16x4 xv = *reinterpret_cast<const bf16x4*>(sX + Tile<PW>::at(t, 16 * pt + 4 * g));
      bf16x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = (bf16_t)(acc[r] + Dh * (float)xv[r]);
      if (t0 + t < len) *reinterpret_cast<bf16x4*>(py + (long long)(t0 + t) * a.ys.t) = o;
    }
    const float dec = sc.dec;
#pragma unroll
    for (int n = 0; n < NT; ++n) hs[n] *= dec;
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 32) {
      bf16x8 f[3];
      weighted<PW>(f, sX, k0, 16 * pt, sc.w, sc.d);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bf16x8 fb = frag_t<N>(sB, k0, 16 * n);
#pragma unroll
        for (int q = 2; q >= 0; --q) hs[n] = mfma(fb, f[q], hs[n]);
      }
    }
  }
  if (seg == a.nseg - 1) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) a.S_final[gstate + (size_t)(16 * n + 4 * g + r) * a.P + i] = hs[n][r];
  }
}

// Gradients of one chunk for one group, as ssm::grad_kernel (the same grid, formulas and sums).  The four waves share
//   * the ten score tiles, three or two each, kept for every head;
//   * the products with the states by columns n (each wave loads its own part of H and R, from memory to registers);
//   * dx by columns p, with R's leading part passed on through LDS.
template <int N, int PW>
__global__ __launch_bounds__(256) void grad_kernel(SsmArgs a) {
  constexpr int NT = N / 16, PT = PW / 16, KN = kblocks<N>(), KP = kblocks<PW>();
  constexpr int NTW = NT >= 4 ? NT / 4 : 1, SL = NT / NTW, TTW = NT / NTW < 4 ? NT / NTW : 4;  // n tiles per wave, slices, token tiles
  __shared__ __attribute__((aligned(16))) bf16_t sB[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sC[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sX[Q * PW];
  __shared__ __attribute__((aligned(16))) bf16_t sY[Q * PW];  // dy
  __shared__ __attribute__((aligned(16))) bf16_t sM[Q * Q];   // [t][s]
  __shared__ __attribute__((aligned(16))) bf16_t sR[N < 32 ? 32 * PW : N * PW];  // [n][p]
  __shared__ Scal scal[4];
  __shared__ float sRow[10][16], sCol[10][16], sDiag[Q], sI[SL][Q], sJ[SL][Q], sK[4], sDD[4];
  const int ch = blockIdx.x, bg = blockIdx.z, b = bg / a.G, grp = bg % a.G, t0 = ch * Q;
  const int w = wave_id(), tid = threadIdx.x, l = lane_id(), g = l >> 4, i = l & 15;
  const int HV = a.H * a.nsl, per_group = HV / a.G;
  const int v0 = blockIdx.y * a.per_split, v1 = min(v0 + a.per_split, per_group);
  const int slice = w % SL, n0 = slice * NTW, tt0 = w / SL * TTW;  // this wave's part of the products with the states
  const int pw = w % PT, st0 = w / PT * PT;                        // its part of dx: column tile, token tiles st0 .. st0 + PT - 1
  {
    Stage<N, 256> lb, lc;
    lb.load((const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h, a.bs.t, t0, a.T);
    lc.load((const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h, a.cs.t, t0, a.T);
    lb.store(sB);
    lc.store(sC);
  }
  for (int k = tid; k < 2 * 16 * 16; k += 256) {  // score tiles above the diagonal inside a k block
    const int blk = k >> 8, r = (k >> 4) & 15, c = k & 15;
    sM[Tile<Q>::at(32 * blk + r, 32 * blk + 16 + c)] = (bf16_t)0.f;
  }
  if constexpr (N < 32)
    for (int k = tid; k < 16 * PW; k += 256) sR[16 * PW + k] = (bf16_t)0.f;  // the empty half of the only k block
  Stage<PW, 256> lx, ly;
  const auto load_head = [&](int v) {
    const int hv = grp * per_group + v, h = hv / a.nsl, p0 = hv % a.nsl * PW;
    lx.load((const bf16_t*)a.x + b * a.xs.b + h * a.xs.h + p0, a.xs.t, t0, a.T);
    ly.load((const bf16_t*)a.dy + b * a.dys.b + h * a.dys.h + p0, a.dys.t, t0, a.T);
  };
  load_head(v0);
  __syncthreads();
  int stt[3], sts[3];  // this wave's score tiles w, w + 4, w + 8
  f32x4 gm[3], dg[3], dc[NTW][TTW], db[NTW][TTW];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int tt = 0, ts = w + 4 * k;
    while (ts > tt) ts -= ++tt;
    stt[k] = tt, sts[k] = ts;
    gm[k] = dg[k] = zero4();
    if (w + 4 * k < 10)
#pragma unroll
      for (int n = 0; n < KN; ++n) gm[k] = mfma(frag_row<N>(sB, 16 * ts, 32 * n), frag_row<N>(sC, 16 * tt, 32 * n), gm[k]);
  }
#pragma unroll
  for (int n = 0; n < NTW; ++n)
#pragma unroll
    for (int t = 0; t < TTW; ++t) dc[n][t] = db[n][t] = zero4();
  for (int v = v0; v < v1; ++v) {
    const int hv = grp * per_group + v, h = hv / a.nsl, sl = hv % a.nsl, p0 = sl * PW;
    const size_t bh = (size_t)b * HV + hv;
    const bf16_t* H = reinterpret_cast<const bf16_t*>(a.st) + (bh * a.nch + ch) * (2 * N * PW);
    const bf16_t* R = reinterpret_cast<const bf16_t*>(a.st) + (((size_t)a.B * HV + bh) * a.nch + ch) * (2 * N * PW);
    const Scal& sc = scal[(v - v0) & 3];
    __syncthreads();
    lx.store(sX);
    ly.store(sY);
    if (((v - v0) & 3) == 0 && v + w < v1) chunk_scalars(a, b, (grp * per_group + v + w) / a.nsl, t0, a.T, scal[w]);
    // this wave's parts of the states: index n, k = p
    bf16x8 fh[2][NTW][KP], fr[2][NTW][KP];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int p = 0; p < KP; ++p) {
          const size_t at = q * (N * PW) + plane_at<N, PW>(2 * p, n0 + n);
          if constexpr (PW == 16) {
            const bf16x4 zero = {0, 0, 0, 0};
            fh[q][n][p] = __builtin_shufflevector(*reinterpret_cast<const bf16x4*>(H + at), zero, 0, 1, 2, 3, 4, 5, 6, 7);
            fr[q][n][p] = __builtin_shufflevector(*reinterpret_cast<const bf16x4*>(R + at), zero, 0, 1, 2, 3, 4, 5, 6, 7);
          } else {
            fh[q][n][p] = *reinterpret_cast<const bf16x8*>(H + at);
            fr[q][n][p] = *reinterpret_cast<const bf16x8*>(R + at);
          }
        }
    if (v + 1 < v1) load_head(v + 1);
    __syncthreads();
    // scores: rows s, columns t
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (w + 4 * k >= 10) break;
      const int tt = stt[k], ts = sts[k], t = 16 * tt + i;
      f32x4 dm = zero4(), col = zero4();
#pragma unroll
      for (int p = 0; p < KP; ++p) dm = mfma(frag_row<PW>(sX, 16 * ts, 32 * p), frag_row<PW>(sY, 16 * tt, 32 * p), dm);
      float row = 0.f;
      bf16x4 m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int s = 16 * ts + 4 * g + r;
        const bool in = s <= t;
        const float e = in ? decay(sc, t, s) : 0.f, d = sc.d[s];
        const float ge = in ? gm[k][r] * e : 0.f, q = in ? ge * dm[r] : 0.f;
        m[r] = (bf16_t)(in ? ge * d : 0.f);
        dg[k][r] += in ? dm[r] * (e * d) : 0.f;
        if (s < t) {
          row += q * d;
          col[r] = q;
        }
        if (s == t) sDiag[s] = q;
      }
      *reinterpret_cast<bf16x4*>(sM + Tile<Q>::at(t, 16 * ts + 4 * g)) = m;
      row = sum_groups(row);
      if (g == 0) sRow[w + 4 * k][i] = row;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float c = sum_lanes16(col[r]);
        if (i == 0) sCol[w + 4 * k][4 * g + r] = c;
      }
    }
    // products with the states: rows n, columns token
    float K = 0.f;
#pragma unroll
    for (int n = 0; n < NTW; ++n)
#pragma unroll
      for (int p = 0; p < KP; ++p) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (tt0 == 0) K += ((float)fh[0][n][p][e] + (float)fh[1][n][p][e]) * ((float)fr[0][n][p][e] + (float)fr[1][n][p][e]);
        // R's leading part as rows n for dx
        if (tt0 == 0) {
          const bf16x8 f = fr[0][n][p];
          const int row = 16 * (n0 + n) + i;
          *reinterpret_cast<bf16x4*>(sR + Tile<PW>::at(row, 32 * p + 4 * g)) = __builtin_shufflevector(f, f, 0, 1, 2, 3);
          if constexpr (PW >= 32)
            *reinterpret_cast<bf16x4*>(sR + Tile<PW>::at(row, 32 * p + 16 + 4 * g)) = __builtin_shufflevector(f, f, 4, 5, 6, 7);
        }
      }
#pragma unroll
    for (int tk = 0; tk < TTW; ++tk) {
      const int tt = tt0 + tk, t = 16 * tt + i;
      const float eo = sc.eo[t], ww = sc.w[t], dd = sc.d[t];
      float I = 0.f, J = 0.f;
      bf16x8 by[KP], bx[KP];
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        by[p] = frag_o<PW>(sY, 16 * tt, 32 * p);
        bx[p] = frag_o<PW>(sX, 16 * tt, 32 * p);
      }
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        f32x4 uc = zero4(), ub = zero4();
#pragma unroll
        for (int q = 1; q >= 0; --q)
#pragma unroll
          for (int p = 0; p < KP; ++p) {
            uc = mfma(fh[q][n][p], by[p], uc);
            ub = mfma(fr[q][n][p], bx[p], ub);
          }
        const bf16x4 fc = *reinterpret_cast<const bf16x4*>(sC + Tile<N>::at(t, 16 * (n0 + n) + 4 * g));
        const bf16x4 fb = *reinterpret_cast<const bf16x4*>(sB + Tile<N>::at(t, 16 * (n0 + n) + 4 * g));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uc[r] *= eo;
          ub[r] *= ww;
          I += (float)fc[r] * uc[r];
          J += (float)fb[r] * ub[r];
          dc[n][tk][r] += uc[r];
          db[n][tk][r] += dd * ub[r];
        }
      }
      I = sum_groups(I);
      J = sum_groups(J);
      if (g == 0) {
        sI[slice][t] = I;
        sJ[slice][t] = J;
      }
    }
    K = sum_groups(sum_lanes16(K));
    if (l == 0) sK[w] = K;
    __syncthreads();
    // dx: rows p, columns s
    const float Dh = a.D != nullptr ? a.D[h] : 0.f;
    float xd = 0.f;
#pragma unroll
    for (int sk = 0; sk < PT; ++sk) {
      const int st = st0 + sk, s = 16 * st + i;
      f32x4 acc = zero4();
#pragma unroll
      for (int n = 0; n < KN; ++n) acc = mfma(frag_t<PW>(sR, 32 * n, 16 * pw), frag_o<N>(sB, 16 * st, 32 * n), acc);
      acc *= sc.w[s] * sc.d[s];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        if (kb >= st / 2) acc = mfma(frag_t<PW>(sY, 32 * kb, 16 * pw), frag_t<Q>(sM, 32 * kb, 16 * st), acc);
      const bf16x4 yv = *reinterpret_cast<const bf16x4*>(sY + Tile<PW>::at(s, 16 * pw + 4 * g));
      const bf16x4 xv = *reinterpret_cast<const bf16x4*>(sX + Tile<PW>::at(s, 16 * pw + 4 * g));
      bf16x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        o[r] = (bf16_t)(acc[r] + Dh * (float)yv[r]);
        xd += (float)xv[r] * (float)yv[r];
      }
      if (t0 + s < a.T)
        *reinterpret_cast<bf16x4*>((bf16_t*)a.dx + b * a.dxs.b + h * a.dxs.h + (long long)(t0 + s) * a.dxs.t + p0 + 16 * pw + 4 * g) = o;
    }
    xd = sum_groups(sum_lanes16(xd));
    if (l == 0) sDD[w] = xd;
    __syncthreads();
    if (w == ((v - v0) & 3)) {  // the head's scalars, the waves in turn
      const int t = l, tt = t >> 4;
      float row = 0.f, qoff = 0.f, I = 0.f, J0 = 0.f, kk = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k <= tt) row += sRow[tt * (tt + 1) / 2 + k][t & 15];
        if (k >= tt) qoff += sCol[k * (k + 1) / 2 + tt][t & 15];
        kk += sK[k];
      }
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        I += sI[k][t];
        J0 += sJ[k][t];
      }
      const float d = sc.d[t], Ah = a.A[h];
      const double jd = (double)d * J0;
      const double f = (double)row - (double)d * qoff + I;
      const double fs = wave_scan(f, t), ftot = __shfl(fs, 63, 64);  // suffix sum from t: ftot - fs + f
      const double js = wave_scan(jd, t);                            // prefix sum before t: js - jd
      const float dl = (float)((ftot - fs + f) + (js - jd) + (double)(sc.dec * kk));
      const float ddt = (qoff + sDiag[t] + J0 + Ah * dl) * sc.sig[t];
      const bool in = t0 + t < a.T;
      if (in) {
        const size_t at = ((size_t)b * a.H + h) * a.T + t0 + t;
        if (a.nsl == 1) a.ddt[at] = ddt;
        else a.part_ddt[(size_t)sl * a.B * a.H * a.T + at] = ddt;
      }
      double sa = in ? (double)dl * d : 0.0, sb = in ? (double)ddt : 0.0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        sa += __shfl_xor(sa, o, 64);
        sb += __shfl_xor(sb, o, 64);
      }
      if (t == 0) {
        const size_t at = bh * a.nch + ch, n = (size_t)a.B * HV * a.nch;
        a.part_sum[at] = (float)sa;
        a.part_sum[n + at] = (sDD[0] + sDD[1]) + (sDD[2] + sDD[3]);
        a.part_sum[2 * n + at] = (float)sb;
      }
    }
  }
  // the summed score gradients times B and C
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (w + 4 * k >= 10) break;
    bf16x4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (bf16_t)dg[k][r];
    *reinterpret_cast<bf16x4*>(sM + Tile<Q>::at(16 * stt[k] + i, 16 * sts[k] + 4 * g)) = o;
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NTW; ++n) {
#pragma unroll
    for (int tk = 0; tk < TTW; ++tk) {
      const int tt = tt0 + tk, t = 16 * tt + i, c = 16 * (n0 + n) + 4 * g;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb <= tt / 2) dc[n][tk] = mfma(frag_t<N>(sB, 32 * kb, 16 * (n0 + n)), frag_o<Q>(sM, 16 * tt, 32 * kb), dc[n][tk]);
        if (kb >= tt / 2) db[n][tk] = mfma(frag_t<N>(sC, 32 * kb, 16 * (n0 + n)), frag_t<Q>(sM, 32 * kb, 16 * tt), db[n][tk]);
      }
      if (t0 + t >= a.T) continue;
      if (a.nsplit == 1) {
        bf16x4 ob, oc;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          ob[r] = (bf16_t)db[n][tk][r];
          oc[r] = (bf16_t)dc[n][tk][r];
        }
        *reinterpret_cast<bf16x4*>((bf16_t*)a.dbm + b * a.dbs.b + grp * a.dbs.h + (long long)(t0 + t) * a.dbs.t + c) = ob;
        *reinterpret_cast<bf16x4*>((bf16_t*)a.dcm + b * a.dcs.b + grp * a.dcs.h + (long long)(t0 + t) * a.dcs.t + c) = oc;
      } else {
        const size_t at = (((size_t)blockIdx.y * a.B * a.G + bg) * a.T + t0 + t) * N + c;
        *reinterpret_cast<f32x4*>(a.part_b + at) = db[n][tk];
        *reinterpret_cast<f32x4*>(a.part_c + at) = dc[n][tk];
      }
    }
  }
}

}  // namespace mx
}  // namespace ssm
}  // namespace prism
