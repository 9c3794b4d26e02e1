// prism_ssm.h - the selective state space scan in float32 arithmetic (gfx950): forward and backward of float32
// tensors, and for both types the single-token step, the scan over segments and the sums of the gradients' shares.
//
//   d_t = softplus(dt_t + bias),  l_t = d_t A,  S_t = e^{l_t} S_{t-1} + d_t B_t x_t^T,  y_t = S_t^T C_t + D x_t
//
// Chunked form, 64 tokens per chunk, with c_t the running sum of l inside the chunk and H the state entering it:
//   y_t  = e^{c_t} H^T C_t + sum_{s<=t} M_ts x_s + D x_t,    M_ts = (C_t . B_s) e^{c_t - c_s} d_s
//   H'   = e^{c_63} H + sum_s e^{c_63 - c_s} d_s B_s x_s^T
// A sequence is cut into segments of chunks that run side by side: a first pass forms each
// segment's end state from zero, a scan over the segments gives the states that enter them.
// c is summed in float64 and held as base-2 exponents in two floats, so that e^{c_t - c_s} keeps
// float32 accuracy after long decays.
//
// Products run on the float32 matrix instructions (153 TFLOP/s in a library product of 8192^3).  Measured: forward of
// 3 x 6 x 509 tokens, N = P = 32: passes of 7, 3 and 11 us; backward of 2 x 6 x 333: 7, 3, 3, 19 and 4 us: launches and one
// chunk's chain of products bound small calls.  8 x 12 x 2048, N = 128, P = 64: forward 283 us, backward 720, where their products
// take 42 and 105 at that rate: the sweep's 104 KB of LDS leave a CU one workgroup of 4 waves, whose rows pass registers
// between two barriers with nothing else in flight, and every head reads B and C again.
#pragma once
#include "prism_ssm_args.h"
#include "prism_tile.h"

namespace prism {
namespace ssm {

constexpr int Q = 64;  // tokens per chunk

// Per-token scalars of one chunk in LDS.
struct Scal {
  float ch[Q], cl[Q];  // running log2 decay, high and low part
  float d[Q];          // step
  float eo[Q];         // decay from the chunk's start through token t
  float w[Q];          // decay from token t to the chunk's end (or that times the step)
  float dec;           // decay over the chunk
};

__device__ __forceinline__ int seq_len(const SsmArgs& a, int b) {
  if (a.lens == nullptr) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

// Lane exchanges inside the VALU (DPP and half swaps), without the LDS round trip of a shuffle.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {  // v plus its neighbour's value, 0 where there is none
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xf, false);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// Inclusive prefix sum over the wave: inside rows of 16 lanes, then row ends into the rows after them.
__device__ __forceinline__ double wave_scan(double v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // row_bcast 15
  return dpp_add<0x143, 0xc>(v);  // row_bcast 31
}
__device__ __forceinline__ double last_lane(double v) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)u, 63), hi = __builtin_amdgcn_readlane((int)(unsigned)(u >> 32), 63);
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
template <int CTRL>
__device__ __forceinline__ float ror_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum_lanes16(float v) {  // over the 16 lanes of a group
  return ror_add<0x121>(ror_add<0x122>(ror_add<0x124>(ror_add<0x128>(v))));
}
__device__ __forceinline__ float sum_groups(float v) {  // over the four 16-lane groups
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know the builtins
  unsigned u = __builtin_bit_cast(unsigned, v);
  const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned h0 = h[0], h1 = h[1];
  v = __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
  u = __builtin_bit_cast(unsigned, v);
  const auto q = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned q0 = q[0], q1 = q[1];
  v = __builtin_bit_cast(float, q0) + __builtin_bit_cast(float, q1);
#endif
  return v;
}

// The same sums in float64, for terms whose row and column sums cancel each other.
template <int CTRL>
__device__ __forceinline__ double ror_add(double v) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, 0xf, 0xf, false);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, 0xf, 0xf, false);
  return v + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double sum_lanes16(double v) {
  return ror_add<0x121>(ror_add<0x122>(ror_add<0x124>(ror_add<0x128>(v))));
}
__device__ __forceinline__ double sum_groups(double v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Whether a token of log decay l lets nothing of the state through: its gradient e^l <S, R> is 0 in float32, where the
// sums that cancel to it would leave their roundings (times a large step, in dA).
__device__ __forceinline__ bool closed(float l) { return l < -105.f; }

__device__ __forceinline__ float softplus_f(float z) { return z > 20.f ? z : log1pf(expf(z)); }

constexpr double kLog2e = 1.4426950408889634;
// A token that decays the state by more than 2^-kGone leaves 0 of it in float32; the decay counts as this much, so that a
// chunk's running sum keeps its digits for the tokens after it.
constexpr double kGone = 160.0;

// Lane t's share of a chunk's scalars: running and total log2 decay, step, and the step's derivative with respect to
// dt.  Tokens at or past len have a step of 0 (decay 1, nothing written).
struct Token {
  double c, tot;
  float d, dz;
  __device__ __forceinline__ float from_start() const { return exp2f((float)c); }
  __device__ __forceinline__ float to_end() const { return exp2f((float)(tot - c)); }
  __device__ __forceinline__ float all() const { return exp2f((float)tot); }
};
__device__ __forceinline__ Token chunk_token(const SsmArgs& a, int b, int h, int t0, int len) {
  const int lane = lane_id(), t = t0 + lane;
  Token k;
  k.d = k.dz = 0.f;
  double l2 = 0.0;
  if (t < len) {
    const float z = a.dt[b * a.ts.b + h * a.ts.h + t * a.ts.t] + (a.dt_bias != nullptr ? a.dt_bias[h] : 0.f);
    k.d = a.softplus ? softplus_f(z) : z;
    k.dz = a.softplus ? 1.f / (1.f + expf(-z)) : 1.f;
    l2 = (double)k.d * (double)a.A[h] * kLog2e;
    if (l2 < -kGone) l2 = -kGone;
  }
  k.c = wave_scan(l2);
  k.tot = last_lane(k.c);
  return k;
}
// One wave: all of a chunk's scalars (w: to the chunk's end, or with WD that times the step).
template <bool WD>
__device__ __forceinline__ void put_scalars(const Token& k, Scal& s) {
  const int lane = lane_id();
  const float hi = (float)k.c;
  s.ch[lane] = hi;
  s.cl[lane] = (float)(k.c - (double)hi);
  s.d[lane] = k.d;
  s.eo[lane] = k.from_start();
  s.w[lane] = WD ? k.to_end() * k.d : k.to_end();
  if (lane == 0) s.dec = k.all();
}

// Rows t0 .. t0 + 63 of a strided [T, W] tensor in LDS (row stride LD); rows at or past len are 0.
template <int W, int LD>
__device__ __forceinline__ void load_rows(float* dst, const void* base, long long off, long long st, int t0, int len,
                                          int nthreads) {
  const float* p = reinterpret_cast<const float*>(base) + off;
  for (int i = threadIdx.x; i < Q * W / 4; i += nthreads) {
    const int r = i / (W / 4), c = i % (W / 4) * 4;
    f32x4 v = zero4();
    if (t0 + r < len) v = *reinterpret_cast<const f32x4*>(p + (long long)(t0 + r) * st + c);
    *reinterpret_cast<f32x4*>(dst + r * LD + c) = v;
  }
}

// Operand fragments of the 16x16x4 float32 MFMA over 16 k values: element r of lane (g, i) is k = 4 g + r.
__device__ __forceinline__ f32x4 frag_k(const float* p, int ld, int row0, int k0) {  // index = row, k contiguous
  const int l = lane_id();
  return *reinterpret_cast<const f32x4*>(p + (row0 + (l & 15)) * ld + k0 + 4 * (l >> 4));
}
__device__ __forceinline__ f32x4 frag_t(const float* p, int ld, int k0, int col0) {  // k = row, index = column
  const int l = lane_id();
  const float* q = p + (k0 + 4 * (l >> 4)) * ld + col0 + (l & 15);
  f32x4 f;
#pragma unroll
  for (int r = 0; r < 4; ++r) f[r] = q[r * ld];
  return f;
}
__device__ __forceinline__ f32x4 scale4(const f32x4& f, const float* s, int k0) {  // times s[k]
  const int g = lane_id() >> 4;
  f32x4 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = f[r] * s[k0 + 4 * g + r];
  return o;
}
// acc[k][row = index of a[k]][col = index of b[k]] += sum over 16 values, for K tiles at once: the values are the outer loop,
// so that neighbouring products go to different accumulators (a product waits about eight times its issue for the one
// before it on the same accumulator).
template <int K>
__device__ __forceinline__ void mm4k(f32x4 (&acc)[K], const f32x4 (&a)[K], const f32x4 (&b)[K]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] = mfma(a[k][r], b[k][r], acc[k]);
}

// A state tile in the workspace: tile (pt, nt) of a transposed state H^T [PW][N] as 64 lanes x 4 floats, lane (g, i)
// holding rows p = 16 pt + 4 g + r, column n = 16 nt + i.
template <int N>
__device__ __forceinline__ size_t tile_at(int pt, int nt) {
  return ((size_t)pt * (N / 16) + nt) * 256 + 4 * lane_id();
}
// Offset of element (n, p) in that layout.
template <int N>
__device__ __forceinline__ size_t elem_at(int n, int p) {
  return ((size_t)(p >> 4) * (N / 16) + (n >> 4)) * 256 + ((p >> 2) & 3) * 64 + (n & 15) * 4 + (p & 3);
}

// States of a segment from zero (or, with SAVE, from the entering state, storing the state at every chunk border).
// Grid (nseg, B * HV, directions); NW = PW / 16 waves, each owning 16 columns.
//   direction 0: H' = dec H + (w d B)^T x over the chunks in order;   saved: the state entering each chunk
//   direction 1: R' = dec R + (eo C)^T dy in reverse order;           saved: the adjoint leaving each chunk
template <int N, int PW, bool SAVE>
__global__ __launch_bounds__(PW * 4) void state_kernel(SsmArgs a) {
  constexpr int NTH = PW * 4, LDN = N + 4, LDP = PW + 4, NT = N / 16;
  __shared__ float sA[Q * LDN];
  __shared__ float sV[Q * LDP];
  __shared__ float sWt[Q], sDec;
  const int seg = blockIdx.x, bh = blockIdx.y, rev = blockIdx.z;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW, grp = h / (a.H / a.G);
  const int len = seq_len(a, b), pt = wave_id(), tid = threadIdx.x;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nch);
  const size_t slot = ((size_t)rev * gridDim.y + bh) * a.nseg + seg;
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    acc[n] = SAVE ? *reinterpret_cast<const f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(pt, n)) : zero4();
  double log_dec = 0.0;
  for (int k = 0; k < c1 - c0; ++k) {
    const int ch = rev ? c1 - 1 - k : c0 + k, t0 = ch * Q;
    if constexpr (SAVE) {
      float* st = a.st + (((size_t)rev * gridDim.y + bh) * a.nch + ch) * (N * PW);
#pragma unroll
      for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(st + tile_at<N>(pt, n)) = acc[n];
      if (k + 1 == c1 - c0) break;  // nobody reads the state behind the segment
    }
    if (t0 >= len) continue;
    __syncthreads();
    if (rev) {
      load_rows<N, LDN>(sA, a.cm, b * a.cs.b + grp * a.cs.h, a.cs.t, t0, len, NTH);
      load_rows<PW, LDP>(sV, a.dy, b * a.dys.b + h * a.dys.h + p0, a.dys.t, t0, len, NTH);
    } else {
      load_rows<N, LDN>(sA, a.bm, b * a.bs.b + grp * a.bs.h, a.bs.t, t0, len, NTH);
      load_rows<PW, LDP>(sV, a.x, b * a.xs.b + h * a.xs.h + p0, a.xs.t, t0, len, NTH);
    }
    if (tid < 64) {
      const Token tk = chunk_token(a, b, h, t0, len);
      log_dec += tk.tot;
      sWt[tid] = rev ? tk.from_start() : tk.to_end() * tk.d;
      if (tid == 0) sDec = tk.all();
    }
    __syncthreads();
    const float dec = sDec;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] *= dec;
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 16) {
      const f32x4 fv = scale4(frag_t(sV, LDP, k0, 16 * pt), sWt, k0);
      f32x4 fvs[NT], fa[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        fvs[n] = fv;
        fa[n] = frag_t(sA, LDN, k0, 16 * n);
      }
      mm4k<NT>(acc, fvs, fa);
    }
  }
  if constexpr (!SAVE) {
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(a.seg + slot * (N * PW) + tile_at<N>(pt, n)) = acc[n];
    if (tid == 0) a.seg_dec[slot] = exp2f((float)log_dec);
  }
}

// The states entering each segment, in place of the segments' own end states: forward from S0, and (direction 1) the
// adjoints arriving at each segment's end, backward from dS_final.  Grid (N * PW / (256 / groups), B * HV, directions): a
// thread holds up to 16 segments of one state element, `groups` (a power of two) threads share an element and pass on
// their products of decays and local sums in LDS, so that the loads of all segments are in flight at once.  TRANS: the
// tiles hold rows p and columns n (else rows n, columns p).
template <int N, int PW, bool TRANS>
__global__ __launch_bounds__(256) void seg_scan_kernel(SsmArgs a, int groups) {
  constexpr int U = 16;
  __shared__ float sP[256], sV[256];
  const int el = 256 / groups, grp = threadIdx.x / el, e = blockIdx.x * el + threadIdx.x % el, bh = blockIdx.y, rev = blockIdx.z;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW;
  const int tile = e >> 8, row = ((e >> 6) & 3) * 4 + (e & 3), col = (e >> 2) & 15;  // position inside a 16 x 16 tile
  const int p = tile / (N / 16) * 16 + (TRANS ? row : col), n = tile % (N / 16) * 16 + (TRANS ? col : row);
  const float* init = rev ? a.dS : a.S0;
  const size_t slot = ((size_t)rev * gridDim.y + bh) * a.nseg;
  float* q = a.seg + slot * (N * PW) + e;
  float own[U], d[U], prod = 1.f, sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = grp * U + u, s = rev ? a.nseg - 1 - k : k;
    own[u] = 0.f, d[u] = 1.f;
    if (k < a.nseg - 1) {  // nothing enters from the last segment's end
      own[u] = q[(size_t)s * (N * PW)];
      d[u] = a.seg_dec[slot + s];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    sum = d[u] * sum + own[u];
    prod *= d[u];
  }
  sP[threadIdx.x] = prod;
  sV[threadIdx.x] = sum;
  float v = init != nullptr ? init[((size_t)(b * a.H + h) * N + n) * a.P + p0 + p] : 0.f;
  __syncthreads();
  for (int k = 0; k < grp; ++k) v = sP[k * el + threadIdx.x % el] * v + sV[k * el + threadIdx.x % el];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = grp * U + u, s = rev ? a.nseg - 1 - k : k;
    if (k >= a.nseg) break;
    q[(size_t)s * (N * PW)] = v;
    v = d[u] * v + own[u];
  }
}

// The scan of a segment from its entering state (seg when nseg > 1, else S0): outputs, and the final state
// from the last segment.  Grid (nseg, B * HV).
template <int N, int PW>
__global__ __launch_bounds__(PW * 4) void sweep_kernel(SsmArgs a) {
  constexpr int NTH = PW * 4, NW = PW / 16, LDN = N + 4, LDP = PW + 4, LDQ = Q + 4, NT = N / 16;
  __shared__ float sB[Q * LDN];
  __shared__ float sC[Q * LDN];
  __shared__ float sX[Q * LDP];
  __shared__ float sM[Q * LDQ];
  __shared__ Scal sc;
  const int seg = blockIdx.x, bh = blockIdx.y;
  const int HV = a.H * a.nsl, b = bh / HV, hv = bh % HV, h = hv / a.nsl, p0 = hv % a.nsl * PW, grp = h / (a.H / a.G);
  const int len = seq_len(a, b), pt = wave_id(), tid = threadIdx.x, l = lane_id(), g = l >> 4, i = l & 15;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nch);
  const float Dh = a.D != nullptr ? a.D[h] : 0.f;
  const size_t gstate = ((size_t)(b * a.H + h) * N) * a.P + p0 + 16 * pt;
  // state tiles: rows n = 16 nt + 4 g + r, column p = 16 pt + i
  f32x4 hs[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * n + 4 * g + r;
      if (a.nseg > 1) hs[n][r] = a.seg[((size_t)bh * a.nseg + seg) * (N * PW) + elem_at<N>(row, 16 * pt + i)];
      else hs[n][r] = a.S0 != nullptr ? a.S0[gstate + (size_t)row * a.P + i] : 0.f;
    }
  for (int ch = c0; ch < c1; ++ch) {
    const int t0 = ch * Q;
    if (t0 >= len) break;
    __syncthreads();
    load_rows<N, LDN>(sB, a.bm, b * a.bs.b + grp * a.bs.h, a.bs.t, t0, len, NTH);
    load_rows<N, LDN>(sC, a.cm, b * a.cs.b + grp * a.cs.h, a.cs.t, t0, len, NTH);
    load_rows<PW, LDP>(sX, a.x, b * a.xs.b + h * a.xs.h + p0, a.xs.t, t0, len, NTH);
    if (tid < 64) put_scalars<false>(chunk_token(a, b, h, t0, len), sc);
    __syncthreads();
    // M: ten tiles (rows s, columns t) over the waves, TG of a wave's at a time; a wave without one forms the last again
    constexpr int SL = (10 + NW - 1) / NW, TG = SL > 5 ? 5 : SL;
#pragma unroll
    for (int q0 = 0; q0 < SL; q0 += TG) {
      f32x4 acc[TG];
      int stt[TG], sts[TG];
#pragma unroll
      for (int q = 0; q < TG; ++q) {
        const int idx = min(pt + NW * (q0 + q), 9);
        stt[q] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
        sts[q] = idx - stt[q] * (stt[q] + 1) / 2;
        acc[q] = zero4();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 fb[TG], fc[TG];
#pragma unroll
        for (int q = 0; q < TG; ++q) {
          fb[q] = frag_k(sB, LDN, 16 * sts[q], 16 * n);
          fc[q] = frag_k(sC, LDN, 16 * stt[q], 16 * n);
        }
        mm4k<TG>(acc, fb, fc);
      }
#pragma unroll
      for (int q = 0; q < TG; ++q) {
        const int t = 16 * stt[q] + i;
        f32x4 m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = 16 * sts[q] + 4 * g + r;
          m[r] = s <= t ? acc[q][r] * exp2f((sc.ch[t] - sc.ch[s]) + (sc.cl[t] - sc.cl[s])) * sc.d[s] : 0.f;
        }
        *reinterpret_cast<f32x4*>(sM + t * LDQ + 16 * sts[q] + 4 * g) = m;
      }
    }
    __syncthreads();
    f32x4 yt[Q / 16];
#pragma unroll
    for (int tt = 0; tt < Q / 16; ++tt) yt[tt] = zero4();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 fh[Q / 16], fc[Q / 16];
#pragma unroll
      for (int tt = 0; tt < Q / 16; ++tt) {
        fh[tt] = hs[n];
        fc[tt] = frag_k(sC, LDN, 16 * tt, 16 * n);
      }
      mm4k<Q / 16>(yt, fh, fc);
    }
#pragma unroll
    for (int tt = 0; tt < Q / 16; ++tt) yt[tt] *= sc.eo[16 * tt + i];
#pragma unroll
    for (int ts = 0; ts < Q / 16; ++ts) {
      const f32x4 fx = frag_t(sX, LDP, 16 * ts, 16 * pt);
      f32x4 fm[Q / 16];
#pragma unroll
      for (int tt = ts; tt < Q / 16; ++tt) fm[tt] = frag_k(sM, LDQ, 16 * tt, 16 * ts);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int tt = ts; tt < Q / 16; ++tt) yt[tt] = mfma(fx[r], fm[tt][r], yt[tt]);
    }
#pragma unroll
    for (int tt = 0; tt < Q / 16; ++tt) {
      const int t = 16 * tt + i;
      const f32x4 xv = *reinterpret_cast<const f32x4*>(sX + t * LDP + 16 * pt + 4 * g);
      if (t0 + t < len) {
        f32x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = yt[tt][r] + Dh * xv[r];
        float* y = reinterpret_cast<float*>(a.y) + b * a.ys.b + h * a.ys.h + (long long)(t0 + t) * a.ys.t + p0 + 16 * pt + 4 * g;
        *reinterpret_cast<f32x4*>(y) = o;
      }
    }
    if ((ch + 1 == c1 || t0 + Q >= len) && seg != a.nseg - 1) break;  // nobody reads the state behind the segment
    const float dec = sc.dec;
#pragma unroll
    for (int n = 0; n < NT; ++n) hs[n] *= dec;
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 16) {
      const f32x4 fx = scale4(scale4(frag_t(sX, LDP, k0, 16 * pt), sc.w, k0), sc.d, k0);
      f32x4 fxs[NT], fb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        fxs[n] = fx;
        fb[n] = frag_t(sB, LDN, k0, 16 * n);
      }
      mm4k<NT>(hs, fb, fxs);
    }
  }
  if (seg == a.nseg - 1) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) a.S_final[gstate + (size_t)(16 * n + 4 * g + r) * a.P + i] = hs[n][r];
  }
}

// Gradients of one chunk for one group (grid (nch, nsplit, B * G)): the workgroup walks its share of the group's
// virtual heads, so that dB and dC are summed over heads in registers.  With H the state entering the chunk and R the
// adjoint of the state leaving it (state_kernel), dM = dy x^T, E_ts = e^{c_t - c_s}:
//   dx_s = sum_t M_ts dy_t + w_s d_s R^T B_s + D dy_s
//   dC_t = sum_s (dM E)_ts d_s B_s + eo_t H dy_t,       dB_s = d_s (sum_t (dM E)_ts C_t + w_s R x_s)
//   dd_s = sum_t q_ts + J_s + A dl_s,   q = (C B^T) E dM,   J_s = w_s B_s . (R x_s)
//   dl_t = sum_{s<t<=t'} q_t's d_s + sum_{t'>=t} I_t' + sum_{s<t} d_s J_s + e^{c_63} <H, R>,   I_t = eo_t C_t . (H dy_t)
// Four waves, wave w owning tokens 16 w .. 16 w + 15 as columns t of the score tiles and as rows of dx, dB and dC.
template <int N, int PW>
__global__ __launch_bounds__(256) void grad_kernel(SsmArgs a) {
  constexpr int LDN = N + 4, LDP = PW + 4, LDQ = Q + 4, NT = N / 16, PT = PW / 16;
  __shared__ float sB[Q * LDN];
  __shared__ float sC[Q * LDN];
  __shared__ float sX[Q * LDP];
  __shared__ float sY[Q * LDP];  // dy
  __shared__ float sM[Q * LDQ];  // M[t][s]
  __shared__ Scal sc;
  __shared__ float sSig[Q], sI[Q], sJ[Q], sDiag[Q], sCol[4][Q], sK[4], sDD[4];
  __shared__ double sRow[Q], sColZ[4][Q];  // sums of q_ts d_s, s < t, over s and over t
  const int ch = blockIdx.x, bg = blockIdx.z, b = bg / a.G, grp = bg % a.G, t0 = ch * Q;
  const int w = wave_id(), tid = threadIdx.x, l = lane_id(), g = l >> 4, i = l & 15;
  const int HV = a.H * a.nsl, per_group = HV / a.G;
  const int v0 = blockIdx.y * a.per_split, v1 = min(v0 + a.per_split, per_group);
  load_rows<N, LDN>(sB, a.bm, b * a.bs.b + grp * a.bs.h, a.bs.t, t0, a.T, 256);
  load_rows<N, LDN>(sC, a.cm, b * a.cs.b + grp * a.cs.h, a.cs.t, t0, a.T, 256);
  __syncthreads();
  const int tok = 16 * w + i;  // this lane's token
  f32x4 gm[4], dg[4], dc[NT], db[NT];
#pragma unroll
  for (int ts = 0; ts < 4; ++ts) gm[ts] = dg[ts] = zero4();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    f32x4 fb[4], fc[4];
#pragma unroll
    for (int ts = 0; ts < 4; ++ts) {
      fb[ts] = frag_k(sB, LDN, 16 * ts, 16 * n);
      fc[ts] = frag_k(sC, LDN, 16 * w, 16 * n);
    }
    mm4k<4>(gm, fb, fc);  // the tiles after the diagonal are formed too, and not used
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) dc[n] = db[n] = zero4();
  for (int v = v0; v < v1; ++v) {
    const int hv = grp * per_group + v, h = hv / a.nsl, slice = hv % a.nsl, p0 = slice * PW;
    const size_t bh = (size_t)b * HV + hv;
    const float* H = a.st + (bh * a.nch + ch) * (N * PW);
    const float* R = a.st + (((size_t)a.B * HV + bh) * a.nch + ch) * (N * PW);
    __syncthreads();
    load_rows<PW, LDP>(sX, a.x, b * a.xs.b + h * a.xs.h + p0, a.xs.t, t0, a.T, 256);
    load_rows<PW, LDP>(sY, a.dy, b * a.dys.b + h * a.dys.h + p0, a.dys.t, t0, a.T, 256);
    if (tid < 64) {
      const Token tk = chunk_token(a, b, h, t0, a.T);
      put_scalars<false>(tk, sc);
      sSig[tid] = tk.dz;
    }
    __syncthreads();
    double row = 0.0;
    f32x4 dms[4];
#pragma unroll
    for (int ts = 0; ts < 4; ++ts) dms[ts] = zero4();
#pragma unroll
    for (int p = 0; p < PT; ++p) {
      f32x4 fx[4], fy[4];
#pragma unroll
      for (int ts = 0; ts < 4; ++ts) {
        fx[ts] = frag_k(sX, LDP, 16 * ts, 16 * p);
        fy[ts] = frag_k(sY, LDP, 16 * w, 16 * p);
      }
      mm4k<4>(dms, fx, fy);
    }
#pragma unroll
    for (int ts = 0; ts < 4; ++ts) {
      f32x4 col = zero4(), colz = zero4();
      if (ts <= w) {
        f32x4 m;
        const f32x4 dm = dms[ts];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = 16 * ts + 4 * g + r;
          const float e = s <= tok ? exp2f((sc.ch[tok] - sc.ch[s]) + (sc.cl[tok] - sc.cl[s])) : 0.f;
          m[r] = s <= tok ? gm[ts][r] * e * sc.d[s] : 0.f;
          dg[ts][r] += s <= tok ? dm[r] * e * sc.d[s] : 0.f;
          const float q = s <= tok ? gm[ts][r] * e * dm[r] : 0.f;
          if (s < tok) {
            col[r] = q;
            colz[r] = q * sc.d[s];
            row += (double)colz[r];
          }
          if (s == tok) sDiag[s] = q;
        }
        *reinterpret_cast<f32x4*>(sM + tok * LDQ + 16 * ts + 4 * g) = m;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float cz = colz[r], c = sum_lanes16(col[r]);
        const double z = sum_lanes16((double)cz);
        if (i == 0) {
          sCol[w][16 * ts + 4 * g + r] = c;
          sColZ[w][16 * ts + 4 * g + r] = z;
        }
      }
    }
    row = sum_groups(row);
    if (g == 0) sRow[tok] = row;
    // products with the states: rows n, columns token
    float I = 0.f, J = 0.f, K = 0.f;
    const float eo = sc.eo[tok], ww = sc.w[tok], dd = sc.d[tok];
    constexpr int NG = NT >= 2 ? 2 : 1;  // columns tiles at a time: four independent chains of products
#pragma unroll
    for (int n1 = 0; n1 < NT; n1 += NG) {
      f32x4 u[2 * NG];
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k) u[k] = zero4();
#pragma unroll
      for (int p = 0; p < PT; ++p) {
        f32x4 f[2 * NG], v2[2 * NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          f[2 * k] = *reinterpret_cast<const f32x4*>(H + tile_at<N>(p, n1 + k));
          f[2 * k + 1] = *reinterpret_cast<const f32x4*>(R + tile_at<N>(p, n1 + k));
          v2[2 * k] = frag_k(sY, LDP, 16 * w, 16 * p);
          v2[2 * k + 1] = frag_k(sX, LDP, 16 * w, 16 * p);
          if ((p * NT + n1 + k) % 4 == w)
#pragma unroll
            for (int r = 0; r < 4; ++r) K += f[2 * k][r] * f[2 * k + 1][r];
        }
        mm4k<2 * NG>(u, f, v2);
      }
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const int n = n1 + k;
        const f32x4 fc = *reinterpret_cast<const f32x4*>(sC + tok * LDN + 16 * n + 4 * g);
        const f32x4 fb = *reinterpret_cast<const f32x4*>(sB + tok * LDN + 16 * n + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float uc = u[2 * k][r] * eo, ub = u[2 * k + 1][r] * ww;
          I += fc[r] * uc;
          J += fb[r] * ub;
          dc[n][r] += uc;
          db[n][r] += dd * ub;
        }
      }
    }
    I = sum_groups(I);
    J = sum_groups(J);
    K = sum_groups(sum_lanes16(K));
    if (g == 0) {
      sI[tok] = I;
      sJ[tok] = J;
    }
    if (l == 0) sK[w] = K;
    __syncthreads();
    // dx: rows p, columns s (this lane's token)
    const float Dh = a.D != nullptr ? a.D[h] : 0.f;
    float xd = 0.f;
    f32x4 ax[PT];
#pragma unroll
    for (int p = 0; p < PT; ++p) ax[p] = zero4();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const f32x4 fb = frag_k(sB, LDN, 16 * w, 16 * n);
      f32x4 fr[PT], fbs[PT];
#pragma unroll
      for (int p = 0; p < PT; ++p) {  // index p, k = n
        fbs[p] = fb;
#pragma unroll
        for (int r = 0; r < 4; ++r) fr[p][r] = R[elem_at<N>(16 * n + 4 * g + r, 16 * p + i)];
      }
      mm4k<PT>(ax, fr, fbs);
    }
#pragma unroll
    for (int p = 0; p < PT; ++p) ax[p] *= ww * dd;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      if (tt < w) continue;
      const f32x4 fm = frag_t(sM, LDQ, 16 * tt, 16 * w);
      f32x4 fy[PT], fms[PT];
#pragma unroll
      for (int p = 0; p < PT; ++p) {
        fms[p] = fm;
        fy[p] = frag_t(sY, LDP, 16 * tt, 16 * p);
      }
      mm4k<PT>(ax, fy, fms);
    }
#pragma unroll
    for (int p = 0; p < PT; ++p) {
      const f32x4 yv = *reinterpret_cast<const f32x4*>(sY + tok * LDP + 16 * p + 4 * g);
      const f32x4 xv = *reinterpret_cast<const f32x4*>(sX + tok * LDP + 16 * p + 4 * g);
      f32x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        o[r] = ax[p][r] + Dh * yv[r];
        xd += xv[r] * yv[r];
      }
      if (t0 + tok < a.T) {
        float* q = reinterpret_cast<float*>(a.dx) + b * a.dxs.b + h * a.dxs.h + (long long)(t0 + tok) * a.dxs.t + p0 + 16 * p + 4 * g;
        *reinterpret_cast<f32x4*>(q) = o;
      }
    }
    xd = sum_groups(sum_lanes16(xd));
    if (l == 0) sDD[w] = xd;
    __syncthreads();
    if (tid < 64) {
      const int t = tid;
      float qoff = 0.f;
      double zoff = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        qoff += (t >> 4) <= k ? sCol[k][t] : 0.f;
        zoff += (t >> 4) <= k ? sColZ[k][t] : 0.0;
      }
      const float d = sc.d[t], J0 = sJ[t], Ah = a.A[h];
      const double jd = (double)d * J0;
      // rows and columns of the same terms in float64: those between two tokens after t cancel in the suffix sum
      const double f = sRow[t] - zoff + sI[t];
      const double fs = wave_scan(f), ftot = last_lane(fs);  // suffix sum from t: ftot - fs + f
      const double js = wave_scan(jd);                       // prefix sum before t: js - jd
      const float kk = sc.dec * ((sK[0] + sK[1]) + (sK[2] + sK[3]));
      const float dl = closed(d * Ah) ? 0.f : (float)((ftot - fs + f) + (js - jd) + kk);
      const float ddt = (qoff + sDiag[t] + J0 + Ah * dl) * sSig[t];
      const bool in = t0 + t < a.T;
      if (in) {
        const size_t at = ((size_t)b * a.H + h) * a.T + t0 + t;
        if (a.nsl == 1) a.ddt[at] = ddt;
        else a.part_ddt[(size_t)slice * a.B * a.H * a.T + at] = ddt;
      }
      const double sa = last_lane(wave_scan(in ? (double)dl * d : 0.0)), sb = last_lane(wave_scan(in ? (double)ddt : 0.0));
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
  for (int ts = 0; ts < 4; ++ts)
    if (ts <= w) *reinterpret_cast<f32x4*>(sM + tok * LDQ + 16 * ts + 4 * g) = dg[ts];
  __syncthreads();
#pragma unroll
  for (int ts = 0; ts < 4; ++ts) {
    f32x4 f[NT], v2[NT];
    if (ts <= w) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f[n] = frag_t(sB, LDN, 16 * ts, 16 * n);
        v2[n] = dg[ts];
      }
      mm4k<NT>(dc, f, v2);
    }
    if (ts >= w) {
      const f32x4 fm = frag_t(sM, LDQ, 16 * ts, 16 * w);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f[n] = frag_t(sC, LDN, 16 * ts, 16 * n);
        v2[n] = fm;
      }
      mm4k<NT>(db, f, v2);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (t0 + tok < a.T) {
      const int c = 16 * n + 4 * g;
      if (a.nsplit == 1) {
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.dbm) + b * a.dbs.b + grp * a.dbs.h + (long long)(t0 + tok) * a.dbs.t + c) = db[n];
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.dcm) + b * a.dcs.b + grp * a.dcs.h + (long long)(t0 + tok) * a.dcs.t + c) = dc[n];
      } else {
        const size_t at = (((size_t)blockIdx.y * a.B * a.G + bg) * a.T + t0 + tok) * N + c;
        *reinterpret_cast<f32x4*>(a.part_b + at) = db[n];
        *reinterpret_cast<f32x4*>(a.part_c + at) = dc[n];
      }
    }
  }
}

// What is left of the gradients once every chunk has its shares, in one launch: workgroups 0 .. 3 H - 1 form dA, dD, ddt_bias of
// a head from the chunks' shares (in float64 and a fixed order); the next n_ddt ddt from the slices' shares (nsl > 1); the rest
// dB, dC from the splits' shares in split order (nsplit > 1), a group of 4 values per thread.
template <class T, int N>
__global__ __launch_bounds__(256) void finish_kernel(SsmArgs a, unsigned n_ddt) {
  __shared__ double part[256];
  unsigned blk = blockIdx.x;
  if (blk < 3u * a.H) {
    const int h = blk / 3, which = blk % 3, HV = a.H * a.nsl;
    float* out = which == 0 ? a.dA : which == 1 ? a.dD : a.ddt_bias;
    if (out == nullptr) return;
    const size_t per = (size_t)a.nsl * a.nch, n = (size_t)a.B * HV * a.nch;
    double s = 0.0;
    for (size_t k = threadIdx.x; k < a.B * per; k += 256)
      s += (double)a.part_sum[which * n + (k / per * HV + (size_t)h * a.nsl) * a.nch + k % per];
    part[threadIdx.x] = s;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
      if ((int)threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
      __syncthreads();
    }
    if (threadIdx.x == 0) out[h] = (float)part[0];
    return;
  }
  blk -= 3u * a.H;
  if (blk < n_ddt) {
    const size_t n = (size_t)a.B * a.H * a.T, i = (size_t)blk * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int k = 0; k < a.nsl; ++k) s += a.part_ddt[k * n + i];
    a.ddt[i] = s;
    return;
  }
  typedef T out4 __attribute__((ext_vector_type(4)));
  const size_t rows = (size_t)a.B * a.G * a.T, i = (size_t)(blk - n_ddt) * 256 + threadIdx.x;
  const size_t row = i / (N / 4);
  if (row >= rows) return;
  const int c = (int)(i % (N / 4)) * 4;
  const size_t bg = row / a.T, t = row % a.T, b = bg / a.G, grp = bg % a.G;
  f32x4 sb = zero4(), scv = zero4();
  for (int k = 0; k < a.nsplit; ++k) {
    sb += *reinterpret_cast<const f32x4*>(a.part_b + ((size_t)k * rows + row) * N + c);
    scv += *reinterpret_cast<const f32x4*>(a.part_c + ((size_t)k * rows + row) * N + c);
  }
  out4 ob, oc;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    ob[r] = (T)sb[r];
    oc[r] = (T)scv[r];
  }
  *reinterpret_cast<out4*>(reinterpret_cast<T*>(a.dbm) + b * a.dbs.b + grp * a.dbs.h + (long long)t * a.dbs.t + c) = ob;
  *reinterpret_cast<out4*>(reinterpret_cast<T*>(a.dcm) + b * a.dcs.b + grp * a.dcs.h + (long long)t * a.dcs.t + c) = oc;
}

// One token: S' = e^{d A} S + d B x^T in place, y = S'^T C + D x.  Bound by reading and writing S: 83 us for 256 x 24
// states of 128 x 64, 4.9 TB/s.  One workgroup per
// (b, h): P / 4 threads across the columns (16-byte state accesses), 256 / (P / 4) groups of rows whose shares of y
// are summed in LDS.
template <class T, int N, int P>
__global__ __launch_bounds__(256) void step_kernel(SsmStepArgs a) {
  constexpr int TC = P / 4, RG = 256 / TC, RPT = N >= RG ? N / RG : 1;
  __shared__ float sY[RG][P];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, grp = h / (a.H / a.G);
  const int c = (threadIdx.x % TC) * 4, rg = threadIdx.x / TC;
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h;
  const T* Bm = reinterpret_cast<const T*>(a.bm) + b * a.bs.b + grp * a.bs.h;
  const T* Cm = reinterpret_cast<const T*>(a.cm) + b * a.cs.b + grp * a.cs.h;
  const float z = a.dt[b * a.ts.b + h * a.ts.h] + (a.dt_bias != nullptr ? a.dt_bias[h] : 0.f);
  const float d = a.softplus ? softplus_f(z) : z;
  const float dec = expf(d * a.A[h]);
  float* S = a.S + (size_t)blockIdx.x * N * P + c;
  f32x4 xv, acc = zero4();
#pragma unroll
  for (int k = 0; k < 4; ++k) xv[k] = d * (float)x[c + k];
  f32x4 s[RPT];
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int n = rg + k * RG;
    if (n < N) s[k] = *reinterpret_cast<const f32x4*>(S + (size_t)n * P);
  }
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int n = rg + k * RG;
    if (n < N) {
      const f32x4 u = s[k] * dec + xv * (float)Bm[n];
      *reinterpret_cast<f32x4*>(S + (size_t)n * P) = u;
      acc += u * (float)Cm[n];
    }
  }
  *reinterpret_cast<f32x4*>(&sY[rg][c]) = acc;
  __syncthreads();
  if (threadIdx.x < P) {
    float y = a.D != nullptr ? a.D[h] * (float)x[threadIdx.x] : 0.f;
#pragma unroll
    for (int k = 0; k < RG; ++k) y += sY[k][threadIdx.x];
    reinterpret_cast<T*>(a.y)[(size_t)blockIdx.x * P + threadIdx.x] = (T)y;
  }
}

}  // namespace ssm
}  // namespace prism
