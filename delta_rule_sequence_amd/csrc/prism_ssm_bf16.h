// prism_ssm_bf16.h - the selective state space scan of bfloat16 tensors on the bf16 matrix instructions (gfx950).
//
// The chunked form and the passes of prism_ssm.h with 16x16x32 bf16 MFMA tiles and float32 sums.  Which operands are
// rounded:
//   * x, B, C, dy are bfloat16 already: C B^T and dy x^T have exact operands;
//   * what enters a state (decay-weighted x or dy) is split into three bfloat16 parts that together hold its 24 bits,
//     so states keep float32 accuracy over any length (three MFMAs in place of one);
//   * the score matrix M and the state as it is read out into y pass as two bfloat16 parts, off by 2^-16 at most, and y is
//     rounded to bfloat16 once (one part each: y was off by 0.0023 of its size for the 0.0017 of that one rounding; the second
//     parts cost 8 of 61 us in the sweep of 8 x 24 x 2048 tokens);
//   * so do M, the summed score gradients and R on their way into dx, dB and dC (2 us of 190 for the backward of 8 x 12 x 2048);
//   * ddt and dA are float32 results: H and R enter the products behind them as three parts, and <H, R> in float32 (two parts:
//     5 us less there, but ddt off by 1e-6 for 1e-7); the sums of score terms that cancel in dA run in float64 (3 us there,
//     for dA off by 4e-6 at most over 40 draws of two heads where float32 sums leave 3e-5).
//
// Waves own 16 columns p of the state in MFMA accumulators from chunk to chunk; an accumulator tile is the operand of
// the readout without passing LDS (rows of a tile pair are the k values of one MFMA, in the order of Mma::koff).
// Tiles lie in LDS without padding, their 16-byte pieces permuted inside a row (Tile::at) so that row reads and
// transposing reads both touch all banks evenly.
//
// Measured, N = 128, P = 64: forward of 8 x 24 x 2048 ragged tokens 30 us for the segments' ends and 60 for the sweep;
// backward of 8 x 12 x 2048: 35 us for the ends, 52 saving states, 110 to 113 for the gradients.  N = P = 64, 2 x 4 x 16384: 13
// and 20 us, and 8 for the scan over 128 segments.  Two waves per SIMD at most (state tiles, operands and scores take
// all 256 registers for N = 128, 194 for N = 64), so a sweep waits for latencies: over all SIMDs its matrix unit is busy 11 %
// of the time, vector instructions 25 %, LDS 16 %; in a ragged batch the XCD with the longest sequence (see Place) works 1.8
// times the mean.
// Saving writes 201 MB at 3.9 TB/s, and the gradients read them again; these issue vector instructions 41 % of the time (the
// splits into parts, float64 sums, LDS places), with the matrix unit busy 11 %, LDS 25 %, and the waves waiting for 48 %.
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
__device__ __forceinline__ bf16x8 frag_n(const bf16_t* t, int row0, int k0, int l = lane_id()) {
  return *reinterpret_cast<const bf16x8*>(t + Tile<W>::at(row0 + (l & 15), k0 + 8 * (l >> 4)));
}
template <int W>
__device__ __forceinline__ bf16x8 frag_o(const bf16_t* t, int row0, int k0, int l = lane_id()) {
  const int r = row0 + (l & 15), k = k0 + 4 * (l >> 4);
  const bf16x4 lo = *reinterpret_cast<const bf16x4*>(t + Tile<W>::at(r, k));
  bf16x4 hi = {0, 0, 0, 0};
  if constexpr (W >= 32) hi = *reinterpret_cast<const bf16x4*>(t + Tile<W>::at(r, k + 16));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int W>
__device__ __forceinline__ bf16x8 frag_row(const bf16_t* t, int row0, int k0, int l = lane_id()) {  // any k order, the same on both sides
  if constexpr (W >= 32) return frag_n<W>(t, row0, k0, l);
  else return frag_o<W>(t, row0, k0, l);
}
template <int W>
__device__ __forceinline__ bf16x8 frag_t(const bf16_t* t, int k0, int col0, int l = lane_id()) {
  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
  const int i = l & 15, r = k0 + 4 * (l >> 4) + (i >> 2), c = col0 + 4 * (i & 3);
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

// The leading part of 8 values, rounded to nearest and taken off them: two parts hold 16 bits (off by 2^-16 at most), three
// the values' float32 digits.
__device__ __forceinline__ bf16x8 take(f32x4& a, f32x4& b) {
  const bf16x8 o = round8(a, b);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    a[r] -= (float)o[r];
    b[r] -= (float)o[4 + r];
  }
  return o;
}

// Loads 64 rows of a strided [T, W] tensor into an LDS tile without passing registers, 16 bytes per lane (buffer loads to
// LDS): a wave's 64 pieces fill 1 KB of the tile in a row, so the permutation of Tile::at is applied to the source
// pieces.  Rows past the sequence's end lie outside the buffer descriptor and arrive as zeros.  Complete after
// loads_done() and a barrier.
template <int W, int NW>
struct Rows {
  static constexpr int RPI = 512 / W, STEP = RPI > 16 ? RPI : 16, PERIOD = STEP / RPI;  // rows per load, rows per permutation period
  static constexpr int NI = Q / RPI, PER = (NI + NW - 1) / NW;                          // loads of a tile, per wave
  static constexpr int OWN = PER < PERIOD ? PER : PERIOD;                               // a wave's places in a period
  int off[OWN];
  int stride;  // bytes
  __device__ __forceinline__ void init(long long st) {
    stride = (int)st * 2;
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int r = (wave_id() * PER + k) % PERIOD * RPI + lane_id() / (W / 8), c = (lane_id() % (W / 8)) ^ Tile<W>::swz(r);
      off[k] = r * stride + c * 16;
    }
  }
  // p: row 0 of the tile (wave-uniform); rows: how many exist
  __device__ __forceinline__ void load(bf16_t* tile, const bf16_t* p, int rows) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know the builtins
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int bytes = rows <= 0 ? 0 : (min(rows, Q) - 1) * stride + W * 2;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t*>(p), 0, bytes, 0x00027000);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int j = w * PER + k;  // wave-uniform
      if (NI % NW != 0 && j >= NI) break;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(tile + j * 512), 16,
                                               off[k % OWN], (j / PERIOD) * STEP * stride, 0, 0);
    }
#endif
  }
};
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// v, of unknown origin: the compiler then forms the LDS places of a phase when it comes to it, rather than once for all heads
// in registers that the other phases lack.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// v, or 0 where !on, whatever v is (as bits: the compiler would branch around what leads to v otherwise).
__device__ __forceinline__ float keep(float v, bool on) { return val(bits(v) & (on ? 0xffffffffu : 0u)); }

// The decay-weighted rows of V (index = column p0 .., k = token k0 ..) in three parts, times wt[k].
__device__ __forceinline__ void weighted(bf16x8 (&p)[3], const bf16x8& f, int k0, const float* wt) {
  const int g4 = 4 * (lane_id() >> 4);
  const f32x4 a = *reinterpret_cast<const f32x4*>(wt + k0 + g4), b = *reinterpret_cast<const f32x4*>(wt + k0 + 16 + g4);
  float v[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] = (float)f[r] * a[r];
    v[4 + r] = (float)f[4 + r] * b[r];
  }
  split3(v, p);
}

// Piece of a saved state: tile (pt, nt) of H^T, 4 values p = 16 pt + 4 g + r of column n = 16 nt + i per lane, for the
// products that contract over p.
template <int N, int PW>
__device__ __forceinline__ size_t saved_at(int pt, int nt) {
  return ((size_t)nt * (PW / 16) + pt) * 256 + lane_id() * 4;
}

// The place of a workgroup of the passes over segments: HP virtual heads of one group from hv0 on, one segment.  Grid
// (B * HV / HP * segments, directions).  The workgroups of one (batch, group, segment) read the same rows of B and C, so
// they take neighbouring numbers; the hardware deals workgroups out to the eight XCDs in turn, so each XCD is given a
// range of numbers of its own, and reads those rows into its L2 once.  (Dealing single units out to the XCDs instead:
// the state pass of 8 x 12 x 2048 tokens 70 us, this way 61; a batch's segments on several XCDs, for the balance of ragged
// batches: 69, since a segment reads the ends of those before it.)  A batch of eight thus lies one sequence to an XCD: ragged,
// the call lasts as long as its longest sequence, 1.8 times the mean for lengths uniform in 0 .. T.
struct Place {
  int b, hv0, seg;
};
template <int HP>
__device__ __forceinline__ Place place(const SsmArgs& a, int segs) {
  const int HV = a.H * a.nsl, pg = HV / a.G / HP;  // workgroups per (batch, group, segment)
  const int q = gridDim.x / 8, r = gridDim.x % 8, x = blockIdx.x % 8;
  int id = x * q + min(x, r) + blockIdx.x / 8;
  const int u = id % pg;
  id /= pg;
  const int seg = id % segs;
  id /= segs;
  return {id / a.G, (id % a.G) * (HV / a.G) + u * HP, seg};
}

// The given first state of virtual head hv of batch b (rev: the adjoint of its last), tiles pt0 .. of 16 columns.
template <int N, int PTW, bool TRANS>
__device__ __forceinline__ void first_state(f32x4 (&acc)[PTW][N / 16], const SsmArgs& a, int rev, int b, int hv, int p0) {
  const int l = lane_id(), g = l >> 4, i = l & 15;
  const float* init = rev ? a.dS : a.S0;
  const size_t at = (size_t)(b * a.H + hv / a.nsl) * N * a.P + p0;
#pragma unroll
  for (int p = 0; p < PTW; ++p)
#pragma unroll
    for (int n = 0; n < N / 16; ++n) {
      acc[p][n] = zero4();
      if (init != nullptr) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = TRANS ? 16 * n + i : 16 * n + 4 * g + r, col = 16 * p + (TRANS ? 4 * g + r : i);
          acc[p][n][r] = init[at + (size_t)row * a.P + col];
        }
      }
    }
}
// The state that enters segment seg (rev: the adjoint that arrives at its end) from the ends of the segments before it: what
// seg_scan_kernel forms, for few segments.  The end that nobody needs gives its place to the first state, which the sweep
// thus does not read from S0 (S_final may be the same buffer).
template <int N, int PW, int PTW, bool TRANS>
__device__ __forceinline__ void entering(f32x4 (&acc)[PTW][N / 16], const SsmArgs& a, int rev, int b, int bh, int hv, int seg, int pt0) {
  if (a.nseg == 1) return first_state<N, PTW, TRANS>(acc, a, rev, b, hv, hv % a.nsl * PW + 16 * pt0);
  const size_t slot = ((size_t)rev * a.B * a.H * a.nsl + bh) * a.nseg;
  const int spare = rev ? 0 : a.nseg - 1;
#pragma unroll
  for (int p = 0; p < PTW; ++p)
#pragma unroll
    for (int n = 0; n < N / 16; ++n) acc[p][n] = *reinterpret_cast<const f32x4*>(a.seg + (slot + spare) * (N * PW) + tile_at<N>(pt0 + p, n));
  const int count = rev ? a.nseg - 1 - seg : seg;
  for (int k = 0; k < count; k += 2) {  // two states in flight; past the last one, the last again, unused
    const int s0 = rev ? a.nseg - 1 - k : k, k1 = min(k + 1, count - 1), s1 = rev ? a.nseg - 1 - k1 : k1;
    const bool two = k + 1 < count;
    const float d0 = a.seg_dec[slot + s0], d1 = two ? a.seg_dec[slot + s1] : 1.f;
    f32x4 u[PTW][N / 16], v[PTW][N / 16];
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < N / 16; ++n) {
        u[p][n] = *reinterpret_cast<const f32x4*>(a.seg + (slot + s0) * (N * PW) + tile_at<N>(pt0 + p, n));
        v[p][n] = *reinterpret_cast<const f32x4*>(a.seg + (slot + s1) * (N * PW) + tile_at<N>(pt0 + p, n));
      }
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < N / 16; ++n) {
        acc[p][n] = acc[p][n] * d0 + u[p][n];
        if (two) acc[p][n] = acc[p][n] * d1 + v[p][n];
      }
  }
}

// PTW: column tiles (16 columns) per wave.  With two, an operand of B or C read from LDS serves two products; with one,
// a head has twice the waves.
template <int PW, int PTW> constexpr int waves_per_head() { return PW / 16 / PTW; }

// States of a segment, as ssm::state_kernel, for HP virtual heads of a group at once (they share the rows of B or C).
// A wave owns PTW tiles of 16 columns of one head.  SAVE = false: from zero, the end state to seg (H: rows n, columns p, as
// the sweep keeps it; or, for the backward, transposed); the segment whose end nobody reads is left out.  SAVE = true:
// from the entering state, saving the state in front of every chunk.  The next chunk's rows arrive in the
// second half of the tiles meanwhile.
template <int N, int PW, int PTW, int HP, bool TRANS, bool SAVE>
__global__ __launch_bounds__((waves_per_head<PW, PTW>() * HP * 64), 2) void state_kernel(SsmArgs a) {
  constexpr int NW = waves_per_head<PW, PTW>(), NWG = NW * HP, NT = N / 16, NB = 4;  // chunks per batch of weights
  __shared__ __attribute__((aligned(16))) bf16_t sA[2][Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sV[2][HP][Q * PW];
  __shared__ __attribute__((aligned(16))) float sWt[2][HP][NB][Q];
  __shared__ float sDec[2][HP][NB];
  const int rev = blockIdx.y, HV = a.H * a.nsl;
  const Place pl = place<HP>(a, SAVE ? a.nseg : a.nseg - 1);
  const int seg = SAVE ? pl.seg : pl.seg + rev, b = pl.b, grp = pl.hv0 / (HV / a.G);
  const int wv = __builtin_amdgcn_readfirstlane(wave_id()), sub = wv / NW, wh = wv % NW, hv = pl.hv0 + sub, h = hv / a.nsl;
  const int bh = b * HV + hv, len = seq_len(a, b);
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nch);
  const size_t slot = ((size_t)rev * a.B * HV + bh) * a.nseg + seg;
  const bf16_t *pa, *pv[HP];
  long long ta, tv;
  if (rev) {
    pa = (const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h, ta = a.cs.t, tv = a.dys.t;
  } else {
    pa = (const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h, ta = a.bs.t, tv = a.xs.t;
  }
#pragma unroll
  for (int q = 0; q < HP; ++q) {
    const int v = pl.hv0 + q, off = v % a.nsl * PW;
    pv[q] = rev ? (const bf16_t*)a.dy + b * a.dys.b + v / a.nsl * a.dys.h + off : (const bf16_t*)a.x + b * a.xs.b + v / a.nsl * a.xs.h + off;
  }
  f32x4 acc[PTW][NT];
  if (!SAVE && a.fold && seg == (rev ? a.nseg - 1 : 0)) {  // see entering()
    first_state<N, PTW, TRANS>(acc, a, rev, b, hv, hv % a.nsl * PW + 16 * wh * PTW);
    float* spare = a.seg + (((size_t)rev * a.B * HV + bh) * a.nseg + (rev ? 0 : a.nseg - 1)) * (N * PW);
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(spare + tile_at<N>(wh * PTW + p, n)) = acc[p][n];
  }
  if (SAVE && a.fold) {
    entering<N, PW, PTW, TRANS>(acc, a, rev, b, bh, hv, seg, wh * PTW);
  } else {
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[p][n] = SAVE ? *reinterpret_cast<const f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(wh * PTW + p, n)) : zero4();
  }
  // chunks that hold tokens, in walking order
  const int live = min(c1, (len + Q - 1) / Q) - c0, steps = SAVE ? c1 - c0 : max(live, 0), last = SAVE ? c1 - 1 : c0 + steps - 1;
  Rows<N, NWG> la;
  Rows<PW, NWG> lv;
  la.init(ta);
  lv.init(tv);
  const auto load = [&](int k) {
    const int t0 = (rev ? last - k : c0 + k) * Q;
    la.load(sA[k & 1], pa + (long long)t0 * ta, len - t0);
#pragma unroll
    for (int q = 0; q < HP; ++q) lv.load(sV[k & 1][q], pv[q] + (long long)t0 * tv, len - t0);
  };
  // saving, the last chunk only has its state saved
  const int rows = SAVE ? steps - 1 : steps;
  if (rows > 0) load(0);
  double log_dec = 0.0;
  for (int k = 0; k < steps; ++k) {
    const int ch = rev ? last - k : c0 + k, par = (k / NB) & 1;
    if (k % NB == 0) {  // the next NB chunks' weights, the head's waves in turn; the other half may still be read
#pragma unroll
      for (int q = 0; q < NB; q += NW) {
        const int kk = k + q + wh;
        if (kk < rows) {
          const Token tk = chunk_token(a, b, h, (rev ? last - kk : c0 + kk) * Q, len);
          log_dec += tk.tot;
          sWt[par][sub][q + wh][lane_id()] = rev ? tk.from_start() : tk.to_end() * tk.d;
          if (lane_id() == 0) sDec[par][sub][q + wh] = tk.all();
        }
      }
    }
    loads_done();
    __syncthreads();  // this chunk's rows are there, the other half's reads are over
    if constexpr (SAVE) {
      float* st = a.st + (((size_t)rev * a.B * HV + bh) * a.nch + ch) * (N * PW);
#pragma unroll
      for (int p = 0; p < PTW; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(st + saved_at<N, PW>(wh * PTW + p, n)) = acc[p][n];
    }
    if (SAVE && k == rows) break;
    if (k + 1 < rows) load(k + 1);
    const float dec = sDec[par][sub][k % NB];
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[p][n] *= dec;
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 32) {
      bf16x8 f[PTW][3];
#pragma unroll
      for (int p = 0; p < PTW; ++p) weighted(f[p], frag_t<PW>(sV[k & 1][sub], k0, 16 * (wh * PTW + p)), k0, sWt[par][sub][k % NB]);
      bf16x8 fa[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) fa[n] = frag_t<N>(sA[k & 1], k0, 16 * n);
      // parts outermost: neighbouring products go to different accumulators
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int p = 0; p < PTW; ++p) acc[p][n] = TRANS ? mfma(f[p][q], fa[n], acc[p][n]) : mfma(fa[n], f[p][q], acc[p][n]);
    }
  }
  if constexpr (!SAVE) {
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(wh * PTW + p, n)) = acc[p][n];
    // the waves' shares of the segment's log decay
    __shared__ double part[HP][NW];
    if (lane_id() == 0) part[sub][wh] = log_dec;
    __syncthreads();
    if (lane_id() == 0 && wh == 0) {
      double s = part[sub][0];
#pragma unroll
      for (int k = 1; k < NW; ++k) s += part[sub][k];
      a.seg_dec[((size_t)rev * a.B * HV + bh) * a.nseg + seg] = exp2f((float)s);
    }
  }
}

// y of row tile tt, rounded: the columns that a lane stores.  One column tile: its own 4.  Two: lanes g, g ^ 1 exchange, and
// a lane holds 8 neighbouring columns, from 16 (g & 1) + 8 (g >> 1) on.
template <int TT>
__device__ __forceinline__ bf16x4 row_piece(const f32x4 (&yt)[1][TT], int tt) {
  bf16x4 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = (bf16_t)yt[0][tt][r];
  return o;
}
template <int TT>
__device__ __forceinline__ bf16x8 row_piece(const f32x4 (&yt)[2][TT], int tt) {
  unsigned v[4] = {};
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    typedef bf16_t pair __attribute__((ext_vector_type(2)));
    const pair p = {(bf16_t)yt[0][tt][2 * k], (bf16_t)yt[0][tt][2 * k + 1]}, q = {(bf16_t)yt[1][tt][2 * k], (bf16_t)yt[1][tt][2 * k + 1]};
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, p), __builtin_bit_cast(unsigned, q), false, false);
    v[k] = s[0], v[2 + k] = s[1];
  }
#endif
  return __builtin_bit_cast(bf16x8, v);
}

// Outputs of a segment from its entering state, as ssm::sweep_kernel, for HP virtual heads of a group at once.  The heads
// share B, C and their products: a wave forms C B^T tiles and the scores of all HP heads from them.  y tiles are formed
// transposed (rows p, columns t), so that a lane stores 8 neighbouring columns (55 -> 53 us at 8 x 24 x 2048 against 4);
// they are stored one chunk later, so that no wave waits for its stores before the next rows.
template <int N, int PW, int PTW, int HP>
__global__ __launch_bounds__((waves_per_head<PW, PTW>() * HP * 64), 2) void sweep_kernel(SsmArgs a) {
  constexpr int NW = waves_per_head<PW, PTW>(), NWG = NW * HP, NT = N / 16, KN = kblocks<N>(), TT = Q / 16;
  constexpr int NB = 2;  // chunks per batch of scalars
  __shared__ __attribute__((aligned(16))) bf16_t sB[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sC[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sX[HP][Q * PW];
  __shared__ __attribute__((aligned(16))) bf16_t sM[HP][2][10 * 256];  // two parts of the tiles on and below the diagonal
  __shared__ Scal scal[HP][NB];
  const int HV = a.H * a.nsl;
  const Place pl = place<HP>(a, a.nseg);
  const int seg = pl.seg, b = pl.b, grp = pl.hv0 / (HV / a.G);
  const int wv = __builtin_amdgcn_readfirstlane(wave_id()), sub = wv / NW, wh = wv % NW, pt0 = wh * PTW;
  const int hv = pl.hv0 + sub, h = hv / a.nsl, p0 = hv % a.nsl * PW;
  const int bh = b * HV + hv, len = seq_len(a, b), l = lane_id(), g = l >> 4, i = l & 15;
  const int c0 = seg * a.seg_chunks, steps = min(min(c0 + a.seg_chunks, a.nch), (len + Q - 1) / Q) - c0;
  float Dh[HP];
#pragma unroll
  for (int q = 0; q < HP; ++q) Dh[q] = a.D != nullptr ? a.D[(pl.hv0 + q) / a.nsl] : 0.f;
  const size_t gstate = ((size_t)(b * a.H + h) * N) * a.P + p0 + 16 * pt0;
  const bf16_t* pb = (const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h;
  const bf16_t* pc = (const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h;
  bf16_t* py = (bf16_t*)a.y + b * a.ys.b + h * a.ys.h + p0 + 16 * pt0 + (PTW == 2 ? 16 * (g & 1) + 8 * (g >> 1) : 4 * g);
  Rows<N, NWG> lb, lc;
  Rows<PW, NWG> lx;
  lb.init(a.bs.t);
  lc.init(a.cs.t);
  lx.init(a.xs.t);
  // state tiles: rows n = 16 nt + 4 g + r, column 16 (pt0 + p) + i
  f32x4 hs[PTW][NT];
  if (a.fold) {
    entering<N, PW, PTW, false>(hs, a, 0, b, bh, hv, seg, pt0);
  } else {
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        hs[p][n] = *reinterpret_cast<const f32x4*>(a.seg + ((size_t)bh * a.nseg + seg) * (N * PW) + tile_at<N>(pt0 + p, n));
  }
  typedef bf16_t ypiece __attribute__((ext_vector_type(4 * PTW)));
  ypiece out[TT];
  const auto store = [&](int k) {
    const int t0 = (c0 + k) * Q;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int t = t0 + 16 * tt + i;
      if (t < len) *reinterpret_cast<ypiece*>(py + (long long)t * a.ys.t) = out[tt];
    }
  };
  for (int k = 0; k < steps; ++k) {
    const int t0 = (c0 + k) * Q;
    __syncthreads();  // the last chunk's reads are over
    lb.load(sB, pb + (long long)t0 * a.bs.t, len - t0);
    lc.load(sC, pc + (long long)t0 * a.cs.t, len - t0);
#pragma unroll
    for (int q = 0; q < HP; ++q) {
      const int v = pl.hv0 + q;
      lx.load(sX[q], (const bf16_t*)a.x + b * a.xs.b + v / a.nsl * a.xs.h + v % a.nsl * PW + (long long)t0 * a.xs.t, len - t0);
    }
    if (k % NB == 0) {  // the next NB chunks' scalars, the head's waves in turn
#pragma unroll
      for (int q = 0; q < NB; q += NW)
        if (q + wh < NB && k + q + wh < steps) put_scalars<true>(chunk_token(a, b, h, t0 + (q + wh) * Q, len), scal[sub][q + wh]);
    }
    loads_done();
    __syncthreads();
    if (k > 0) store(k - 1);
    // scores: ten tiles (rows s, columns t) over the waves; a wave without one forms the last tile again.  Here and below
    // the k block is the outer loop, so that neighbouring products go to different accumulators.
    constexpr int SL = (10 + NWG - 1) / NWG;
    int stt[SL], sts[SL];
    f32x4 sacc[SL];
#pragma unroll
    for (int q = 0; q < SL; ++q) {
      const int idx = min(wv + NWG * q, 9);
      stt[q] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
      sts[q] = idx - stt[q] * (stt[q] + 1) / 2;
      sacc[q] = zero4();
    }
#pragma unroll
    for (int n = 0; n < KN; ++n)
#pragma unroll
      for (int q = 0; q < SL; ++q) sacc[q] = mfma(frag_row<N>(sB, 16 * sts[q], 32 * n), frag_row<N>(sC, 16 * stt[q], 32 * n), sacc[q]);
#pragma unroll
    for (int q = 0; q < SL; ++q) {
      const int t = 16 * stt[q] + i, s0 = 16 * sts[q] + 4 * g;
#pragma unroll
      for (int u = 0; u < HP; ++u) {
        const Scal& sc = scal[u][k % NB];
        const float cht = sc.ch[t], clt = sc.cl[t];
        const f32x4 chs = *reinterpret_cast<const f32x4*>(sc.ch + s0), cls = *reinterpret_cast<const f32x4*>(sc.cl + s0);
        const f32x4 ds = *reinterpret_cast<const f32x4*>(sc.d + s0);
        bf16x4 m[2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f((cht - chs[r]) + (clt - cls[r]));
          float v = keep(sacc[q][r] * (e * ds[r]), s0 + r <= t);
          if (stt[q] == sts[q]) v += s0 + r == t ? Dh[u] : 0.f;  // the skip term: D x_t = D x_s for s = t
          m[0][r] = (bf16_t)v;
          m[1][r] = (bf16_t)(v - (float)m[0][r]);
        }
        // in the order in which the readout's lanes take them: lane (g, i) has row t = i, columns 4 g .. 4 g + 3 of a tile
        const int tile = stt[q] * (stt[q] + 1) / 2 + sts[q];
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) *reinterpret_cast<bf16x4*>(&sM[u][h2][tile * 256 + 4 * l]) = m[h2];
      }
    }
    __syncthreads();
    const Scal& sc = scal[sub][k % NB];
    const bf16_t* tX = sX[sub];
    f32x4 yt[PTW][TT];
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) yt[p][tt] = zero4();
#pragma unroll
    for (int n = 0; n < KN; ++n) {
      bf16x8 hf[PTW][2], fc[TT];
#pragma unroll
      for (int p = 0; p < PTW; ++p) {
        f32x4 h0 = hs[p][2 * n], h1 = 2 * n + 1 < NT ? hs[p][2 * n + 1 < NT ? 2 * n + 1 : 0] : zero4();
        hf[p][0] = take(h0, h1);
        hf[p][1] = round8(h0, h1);
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) fc[tt] = frag_o<N>(sC, 16 * tt, 32 * n);
#pragma unroll
      for (int q = 1; q >= 0; --q)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
          for (int p = 0; p < PTW; ++p) yt[p][tt] = mfma(hf[p][q], fc[tt], yt[p][tt]);
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const float eo = sc.eo[16 * tt + i];
#pragma unroll
      for (int p = 0; p < PTW; ++p) yt[p][tt] *= eo;
    }
    // nobody reads the state behind a segment but the last
    const bool go_on = k + 1 < steps || seg == a.nseg - 1;
    if (go_on) {
      const float dec = sc.dec;
#pragma unroll
      for (int p = 0; p < PTW; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n) hs[p][n] *= dec;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      bf16x8 fx[PTW], f[PTW][3];
#pragma unroll
      for (int p = 0; p < PTW; ++p) fx[p] = frag_t<PW>(tX, 32 * kb, 16 * (pt0 + p));
#pragma unroll
      for (int q = 1; q >= 0; --q)
#pragma unroll
        for (int tt = 2 * kb; tt < TT; ++tt) {
          const bf16_t* m = &sM[sub][q][(tt * (tt + 1) / 2 + 2 * kb) * 256 + 4 * l];
          const bf16x4 lo = *reinterpret_cast<const bf16x4*>(m);
          bf16x4 hi = {0, 0, 0, 0};
          if (tt > 2 * kb) hi = *reinterpret_cast<const bf16x4*>(m + 256);
          const bf16x8 fm = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int p = 0; p < PTW; ++p) yt[p][tt] = mfma(fx[p], fm, yt[p][tt]);
        }
      if (!go_on) continue;
#pragma unroll
      for (int p = 0; p < PTW; ++p) weighted(f[p], fx[p], 32 * kb, sc.w);
      bf16x8 fb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) fb[n] = frag_t<N>(sB, 32 * kb, 16 * n);
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int p = 0; p < PTW; ++p) hs[p][n] = mfma(fb[n], f[p][q], hs[p][n]);
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) out[tt] = row_piece(yt, tt);
  }
  if (steps > 0) store(steps - 1);
  if (seg == a.nseg - 1) {
#pragma unroll
    for (int p = 0; p < PTW; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.S_final[gstate + (size_t)(16 * n + 4 * g + r) * a.P + 16 * p + i] = hs[p][n][r];
  }
}

// Gradients of one chunk for one group, as ssm::grad_kernel (the same grid, formulas and sums).  The eight waves share
//   * the ten score tiles, two or one each, kept for every head;
//   * the products with the states by columns n (each wave loads its own part of H and R, from memory to registers);
//   * dx by columns p, with R's first two parts passed on through LDS.
// Eight waves rather than four: a wave's accumulators and operands then fit its registers (245 of 256 for N = 128, P = 64),
// since the scores' and dx's places in LDS are formed anew for every head (fresh): kept from head to head they leave 30
// registers to scratch (8 x 12 x 2048 tokens: the backward 239 us for 190).
// The skip term sits on the scores' diagonal (D dy_s = D dy_t for t = s), and dD is the sum of the diagonal of dy x^T.
template <int N, int PW>
__global__ __launch_bounds__(512, 2) void grad_kernel(SsmArgs a) {
  constexpr int NT = N / 16, PT = PW / 16, KN = kblocks<N>(), KP = kblocks<PW>(), WV = 8;
  constexpr int NB = 2;                            // heads per batch of scalars
  constexpr int SLOTS = 2;                         // score tiles per wave
  constexpr int TTW = NT * 4 > WV ? NT * 4 / WV : 1;  // token tiles of a wave's column tile n; N = 16 leaves half the waves without
  constexpr int STW = PT * 4 > WV ? PT * 4 / WV : 1;  // token tiles of a wave's column tile p in dx; P = 16 likewise
  __shared__ __attribute__((aligned(16))) bf16_t sB[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sC[Q * N];
  __shared__ __attribute__((aligned(16))) bf16_t sXs[2][Q * PW];
  __shared__ __attribute__((aligned(16))) bf16_t sYs[2][Q * PW];  // dy
  __shared__ __attribute__((aligned(16))) bf16_t sM[2][Q * Q];   // [t][s], two parts
  __shared__ __attribute__((aligned(16))) bf16_t sR[2][N < 32 ? 32 * PW : N * PW];  // [n][p], the first two of three parts
  __shared__ Scal scals[2][NB];
  __shared__ double sRow[10][16], sColZ[10][16];  // sums of q_ts d_s, s < t, over s and over t
  __shared__ float sSig[2][NB][Q], sCol[10][16], sDiag[Q], sXY[Q], sI[NT][Q], sJ[NT][Q], sK[WV];
  const int ch = blockIdx.x, bg = blockIdx.z, b = bg / a.G, grp = bg % a.G, t0 = ch * Q;
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), tid = threadIdx.x, l = lane_id(), g = l >> 4, i = l & 15;
  const int HV = a.H * a.nsl, per_group = HV / a.G;
  const int v0 = blockIdx.y * a.per_split, v1 = min(v0 + a.per_split, per_group);
  const int nt = w % NT, tt0 = w / NT * TTW;   // this wave's part of the products with the states
  const int pw = w % PT, st0 = w / PT * STW;   // its part of dx
  const bool has_n = tt0 < 4, has_p = st0 < 4;
  {
    Rows<N, WV> lb, lc;
    lb.init(a.bs.t);
    lc.init(a.cs.t);
    lb.load(sB, (const bf16_t*)a.bm + b * a.bs.b + grp * a.bs.h + (long long)t0 * a.bs.t, a.T - t0);
    lc.load(sC, (const bf16_t*)a.cm + b * a.cs.b + grp * a.cs.h + (long long)t0 * a.cs.t, a.T - t0);
  }
  for (int k = tid; k < 2 * 16 * 16; k += 512) {  // score tiles above the diagonal inside a k block
    const int blk = k >> 8, r = (k >> 4) & 15, c = k & 15;
    sM[0][Tile<Q>::at(32 * blk + r, 32 * blk + 16 + c)] = sM[1][Tile<Q>::at(32 * blk + r, 32 * blk + 16 + c)] = (bf16_t)0.f;
  }
  if constexpr (N < 32)
    for (int k = tid; k < 16 * PW; k += 512) sR[0][16 * PW + k] = sR[1][16 * PW + k] = (bf16_t)0.f;  // the empty half of the only k block
  Rows<PW, WV> lx, ly;
  lx.init(a.xs.t);
  ly.init(a.dys.t);
  const auto load = [&](int v) {
    const int hv = grp * per_group + v, h = hv / a.nsl, p0 = hv % a.nsl * PW, buf = (v - v0) & 1;
    lx.load(sXs[buf], (const bf16_t*)a.x + b * a.xs.b + h * a.xs.h + p0 + (long long)t0 * a.xs.t, a.T - t0);
    ly.load(sYs[buf], (const bf16_t*)a.dy + b * a.dys.b + h * a.dys.h + p0 + (long long)t0 * a.dys.t, a.T - t0);
  };
  load(v0);
  // this wave's parts of the states: index n, k = p (zeros in the empty half of P = 16).  Loaded a head ahead: in flight over
  // dx and the next head's scores.
  f32x4 hv4[2 * KP], rv4[2 * KP];
  const auto load_states = [&](int v) {
    const size_t bh = (size_t)b * HV + grp * per_group + v;
    const float* H = a.st + (bh * a.nch + ch) * (N * PW);
    const float* R = a.st + (((size_t)a.B * HV + bh) * a.nch + ch) * (N * PW);
#pragma unroll
    for (int p = 0; p < 2 * KP; ++p) {
      hv4[p] = p < PT ? *reinterpret_cast<const f32x4*>(H + saved_at<N, PW>(p < PT ? p : 0, nt)) : zero4();
      rv4[p] = p < PT ? *reinterpret_cast<const f32x4*>(R + saved_at<N, PW>(p < PT ? p : 0, nt)) : zero4();
    }
  };
  loads_done();
  load_states(v0);
  __syncthreads();
  int stt[SLOTS], sts[SLOTS];  // this wave's score tiles w, w + 8
  f32x4 gm[SLOTS], dg[SLOTS], dc[TTW], db[TTW];
#pragma unroll
  for (int k = 0; k < SLOTS; ++k) {
    const int idx = min(w + WV * k, 9);
    stt[k] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
    sts[k] = idx - stt[k] * (stt[k] + 1) / 2;
    gm[k] = dg[k] = zero4();
    if (w + WV * k < 10)
#pragma unroll
      for (int n = 0; n < KN; ++n) gm[k] = mfma(frag_row<N>(sB, 16 * sts[k], 32 * n), frag_row<N>(sC, 16 * stt[k], 32 * n), gm[k]);
  }
#pragma unroll
  for (int t = 0; t < TTW; ++t) dc[t] = db[t] = zero4();
  // the scalars of NB heads from v on, by the last NB waves
  const auto scalars = [&](int v) {
    const int k = w - (WV - NB), par = ((v - v0) / NB) & 1;
    if (k < 0 || v + k >= v1) return;
    const Token tk = chunk_token(a, b, (grp * per_group + v + k) / a.nsl, t0, a.T);
    put_scalars<false>(tk, scals[par][k]);
    sSig[par][k][l] = tk.dz;
  };
  scalars(v0);
  for (int v = v0; v < v1; ++v) {
    const int hv = grp * per_group + v, h = hv / a.nsl, sl = hv % a.nsl, p0 = sl * PW, hb = (v - v0) % NB;
    const size_t bh = (size_t)b * HV + hv;
    const int par = ((v - v0) / NB) & 1;
    const Scal& sc = scals[par][hb];
    const bf16_t *sX = sXs[(v - v0) & 1], *sY = sYs[(v - v0) & 1];
    const float Dh = a.D != nullptr ? a.D[h] : 0.f;
    __syncthreads();  // every wave has its rows of this head (waited for below), the last head's reads are over
    if (v + 1 < v1) load(v + 1);
    // scores: rows s, columns t
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      if (w + WV * k >= 10) break;
      const int lf = fresh(l), g = lf >> 4, i = lf & 15;
      const int tt = stt[k], ts = sts[k], t = 16 * tt + i, s0 = 16 * ts + 4 * g;
      f32x4 dm = zero4(), col;
#pragma unroll
      for (int p = 0; p < KP; ++p) dm = mfma(frag_row<PW>(sX, 16 * ts, 32 * p, lf), frag_row<PW>(sY, 16 * tt, 32 * p, lf), dm);
      const float cht = sc.ch[t], clt = sc.cl[t];
      const f32x4 chs = *reinterpret_cast<const f32x4*>(sc.ch + s0), cls = *reinterpret_cast<const f32x4*>(sc.cl + s0);
      const f32x4 ds = *reinterpret_cast<const f32x4*>(sc.d + s0);
      double row = 0.0;
      f32x4 colf;
      bf16x4 m[2];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f((cht - chs[r]) + (clt - cls[r])), ed = e * ds[r];
        const float q = gm[k][r] * e * dm[r];
        float mm = gm[k][r] * ed, dd = dm[r] * ed, off = q;
        if (tt == ts) {
          mm = keep(mm, s0 + r <= t) + (s0 + r == t ? Dh : 0.f);
          dd = keep(dd, s0 + r <= t);
          off = keep(q, s0 + r < t);
          if (s0 + r == t) {
            sDiag[t] = q;
            sXY[t] = dm[r];
          }
        }
        m[0][r] = (bf16_t)mm;
        m[1][r] = (bf16_t)(mm - (float)m[0][r]);
        dg[k][r] += dd;
        const float z = off * ds[r];
        row += (double)z;
        colf[r] = z;
        col[r] = off;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) *reinterpret_cast<bf16x4*>(sM[q] + Tile<Q>::at(t, s0)) = m[q];
      row = sum_groups(row);
      if (g == 0) sRow[w + WV * k][i] = row;
#pragma unroll
      for (int r = 0; r < 4; ++r) col[r] = sum_lanes16(col[r]);
      if (i == 0) *reinterpret_cast<f32x4*>(&sCol[w + WV * k][4 * g]) = col;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float cz = colf[r];
        const double z = sum_lanes16((double)cz);
        if (i == 0) sColZ[w + WV * k][4 * g + r] = z;
      }
    }
    // products with the states: rows n, columns token
    float K = 0.f;
    if (has_n) {
      f32x4 uc[TTW], ub[TTW];
#pragma unroll
      for (int k = 0; k < TTW; ++k) uc[k] = ub[k] = zero4();
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        f32x4 &h0 = hv4[2 * p], &h1 = hv4[2 * p + 1], &r0 = rv4[2 * p], &r1 = rv4[2 * p + 1];
        if (tt0 == 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r) K += h0[r] * r0[r] + h1[r] * r1[r];
        }
        bf16x8 by[TTW], bx[TTW];
#pragma unroll
        for (int k = 0; k < TTW; ++k) by[k] = frag_o<PW>(sY, 16 * (tt0 + k), 32 * p), bx[k] = frag_o<PW>(sX, 16 * (tt0 + k), 32 * p);
        // part by part, each taken off the values in place
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const bf16x8 fh = take(h0, h1), fr = take(r0, r1);
          if (q < 2 && tt0 == 0) {  // R as rows n for dx
            *reinterpret_cast<bf16x4*>(sR[q] + Tile<PW>::at(16 * nt + i, 32 * p + 4 * g)) = __builtin_shufflevector(fr, fr, 0, 1, 2, 3);
            if constexpr (PW >= 32)
              *reinterpret_cast<bf16x4*>(sR[q] + Tile<PW>::at(16 * nt + i, 32 * p + 16 + 4 * g)) = __builtin_shufflevector(fr, fr, 4, 5, 6, 7);
          }
#pragma unroll
          for (int k = 0; k < TTW; ++k) {
            uc[k] = mfma(fh, by[k], uc[k]);
            ub[k] = mfma(fr, bx[k], ub[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < TTW; ++k) {
        const int t = 16 * (tt0 + k) + i;
        const float eo = sc.eo[t], ww = sc.w[t], wd = ww * sc.d[t];
        const bf16x4 fc = *reinterpret_cast<const bf16x4*>(sC + Tile<N>::at(t, 16 * nt + 4 * g));
        const bf16x4 fb = *reinterpret_cast<const bf16x4*>(sB + Tile<N>::at(t, 16 * nt + 4 * g));
        float I = 0.f, J = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          I += (float)fc[r] * uc[k][r];
          J += (float)fb[r] * ub[k][r];
          dc[k][r] += eo * uc[k][r];
          db[k][r] += wd * ub[k][r];
        }
        I = sum_groups(I);
        J = sum_groups(J);
        if (g == 0) {
          sI[nt][t] = I * eo;
          sJ[nt][t] = J * ww;
        }
      }
      K = sum_groups(sum_lanes16(K));
    }
    if (l == 0) sK[w] = K;
    loads_done();  // the next head's rows
    // unconditional (the last head's again): behind a branch the compiler would wait for them at the barrier
    load_states(min(v + 1, v1 - 1));
    __syncthreads();
    // dx: rows p, columns s
    if (has_p) {
      const int lf = fresh(l), g = lf >> 4, i = lf & 15;
      f32x4 ax[STW];
#pragma unroll
      for (int k = 0; k < STW; ++k) ax[k] = zero4();
#pragma unroll
      for (int n = 0; n < KN; ++n) {
        bf16x8 f[2], fb[STW];
#pragma unroll
        for (int q = 0; q < 2; ++q) f[q] = frag_t<PW>(sR[q], 32 * n, 16 * pw, lf);
#pragma unroll
        for (int k = 0; k < STW; ++k) fb[k] = frag_o<N>(sB, 16 * (st0 + k), 32 * n, lf);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int k = 0; k < STW; ++k) ax[k] = mfma(f[q], fb[k], ax[k]);
      }
#pragma unroll
      for (int k = 0; k < STW; ++k) {
        const int s = 16 * (st0 + k) + i;
        ax[k] *= sc.w[s] * sc.d[s];
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 f = frag_t<PW>(sY, 32 * kb, 16 * pw, lf);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int k = 0; k < STW; ++k)
            if (kb >= (st0 + k) / 2) ax[k] = mfma(f, frag_t<Q>(sM[q], 32 * kb, 16 * (st0 + k), lf), ax[k]);
      }
#pragma unroll
      for (int k = 0; k < STW; ++k) {
        const int s = 16 * (st0 + k) + i;
        bf16x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = (bf16_t)ax[k][r];
        if (t0 + s < a.T)
          *reinterpret_cast<bf16x4*>((bf16_t*)a.dx + b * a.dxs.b + h * a.dxs.h + (long long)(t0 + s) * a.dxs.t + p0 + 16 * pw + 4 * g) = o;
      }
    }
    // The later waves have less to do for dx: they form what is left of this head, and the next heads' scalars in the half
    // that the last heads' reads have left (in front of the first barrier, by the first waves: 4 us more).
    if (hb == NB - 1) scalars(v + 1);
    if (w == WV / 2 + hb) {
      const int t = l, tt = t >> 4;
      float qoff = 0.f, I = 0.f, J0 = 0.f;
      double row = 0.0, zoff = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k <= tt) row += sRow[tt * (tt + 1) / 2 + k][t & 15];
        if (k >= tt) qoff += sCol[k * (k + 1) / 2 + tt][t & 15], zoff += sColZ[k * (k + 1) / 2 + tt][t & 15];
      }
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        I += sI[k][t];
        J0 += sJ[k][t];
      }
      float kk = 0.f;
#pragma unroll
      for (int k = 0; k < WV; ++k) kk += sK[k];
      const float d = sc.d[t], Ah = a.A[h];
      const double jd = (double)d * J0;
      // rows and columns of the same terms in float64: those between two tokens after t cancel in the suffix sum
      const double f = row - zoff + I;
      const double fs = wave_scan(f), ftot = last_lane(fs);  // suffix sum from t: ftot - fs + f
      const double js = wave_scan(jd);                       // prefix sum before t: js - jd
      const float dl = closed(d * Ah) ? 0.f : (float)((ftot - fs + f) + (js - jd) + (double)(sc.dec * kk));
      const float ddt = (qoff + sDiag[t] + J0 + Ah * dl) * sSig[par][hb][t];
      const bool in = t0 + t < a.T;
      if (in) {
        const size_t at = ((size_t)b * a.H + h) * a.T + t0 + t;
        if (a.nsl == 1) a.ddt[at] = ddt;
        else a.part_ddt[(size_t)sl * a.B * a.H * a.T + at] = ddt;
      }
      const double sa = last_lane(wave_scan(in ? (double)dl * d : 0.0)), sb = last_lane(wave_scan(in ? (double)ddt : 0.0));
      const double sd = last_lane(wave_scan((double)sXY[t]));
      if (t == 0) {
        const size_t at = bh * a.nch + ch, n = (size_t)a.B * HV * a.nch;
        a.part_sum[at] = (float)sa;
        a.part_sum[n + at] = (float)sd;
        a.part_sum[2 * n + at] = (float)sb;
      }
    }
  }
  // the summed score gradients times B and C
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SLOTS; ++k) {
    if (w + WV * k >= 10) break;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      bf16x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = (bf16_t)dg[k][r], dg[k][r] -= (float)o[r];
      *reinterpret_cast<bf16x4*>(sM[q] + Tile<Q>::at(16 * stt[k] + i, 16 * sts[k] + 4 * g)) = o;
    }
  }
  __syncthreads();
  if (!has_n) return;
#pragma unroll
  for (int k = 0; k < TTW; ++k) {
    const int tt = tt0 + k, t = 16 * tt + i, c = 16 * nt + 4 * g;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (kb <= tt / 2) dc[k] = mfma(frag_t<N>(sB, 32 * kb, 16 * nt), frag_o<Q>(sM[q], 16 * tt, 32 * kb), dc[k]);
        if (kb >= tt / 2) db[k] = mfma(frag_t<N>(sC, 32 * kb, 16 * nt), frag_t<Q>(sM[q], 32 * kb, 16 * tt), db[k]);
      }
    }
    if (t0 + t >= a.T) continue;
    if (a.nsplit == 1) {
      bf16x4 ob, oc;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ob[r] = (bf16_t)db[k][r];
        oc[r] = (bf16_t)dc[k][r];
      }
      *reinterpret_cast<bf16x4*>((bf16_t*)a.dbm + b * a.dbs.b + grp * a.dbs.h + (long long)(t0 + t) * a.dbs.t + c) = ob;
      *reinterpret_cast<bf16x4*>((bf16_t*)a.dcm + b * a.dcs.b + grp * a.dcs.h + (long long)(t0 + t) * a.dcs.t + c) = oc;
    } else {
      const size_t at = (((size_t)blockIdx.y * a.B * a.G + bg) * a.T + t0 + t) * N + c;
      *reinterpret_cast<f32x4*>(a.part_b + at) = db[k];
      *reinterpret_cast<f32x4*>(a.part_c + at) = dc[k];
    }
  }
}

}  // namespace mx
}  // namespace ssm
}  // namespace prism
