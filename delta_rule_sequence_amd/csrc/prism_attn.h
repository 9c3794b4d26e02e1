// prism_attn.h - softmax attention of a prompt's rows (gfx950), forward.
//
//   s_ij = scale <q_i, k_j>,  o_i = sum_j e^(s_ij - m_i) v_j / l_i,  l_i = sum_j e^(s_ij - m_i),  lse_i = m_i + log l_i
// over the keys j <= i of i's sequence (causal), j > i - window, in one pass over the keys with a running m and l.
//
// A wave owns 32 queries and forms transposed tiles: S^T = K Q^T puts one query into a lane (and its partner 32 lanes on),
// so that m, l and the rescaling of o are single registers, and the tile's accumulators are, rounded, the second
// operand of O^T = V^T P^T without leaving their lane.  Q stays in registers; tiles of K and V go through LDS, read by
// rows (K) and transposed on the way (V).
#pragma once
#include <climits>
#include <type_traits>

#include "prism_attn_args.h"
#include "prism_tile.h"

namespace prism {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kInf = __builtin_inff();

// ---- 32 x 32 tiles ---------------------------------------------------------------------------------
// An operand's piece: 16 bytes of row l % 32; of the two pieces of a step, lane half h = l / 32 holds the h-th.  An
// accumulator's register i in lane l is row 8 (i / 4) + 4 h + i % 4, column l % 32.
__device__ __forceinline__ void mma(f32x16& acc, const u32x4& a, const u32x4& b, bf16_t) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16& acc, const u32x4& a, const u32x4& b, float) {
  const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[r], y[r], acc, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Rows of D values in LDS.  32 bytes between rows spread both kinds of reads over the banks.
template <class T, int D> struct Rows {
  static constexpr int kBytes = D * (int)sizeof(T), kStride = kBytes + 32;
  static constexpr int kPieces = kBytes / 16, kSteps = kPieces / 2;
  static constexpr int kPer = 16 / (int)sizeof(T);   // values of a piece
  // This lane's place in a tile of 32 rows, read by rows or transposed.
  static __device__ __forceinline__ int by_rows(int l) { return (l & 31) * kStride + (l >> 5) * 16; }
  static __device__ __forceinline__ int transposed(int l) {
    if constexpr (sizeof(T) == 2)
      return (4 * (l >> 5) + ((l & 15) >> 2)) * kStride + ((l >> 4) & 1) * 32 + (l & 3) * 8;
    else
      return 4 * (l >> 5) * kStride + (l & 31) * 4;
  }
};

__device__ __forceinline__ u32x4 lds16(const char* p) { return *reinterpret_cast<const u32x4*>(p); }

// Four rows of 16 columns, a column per lane: lane 4 r + c of 16 points at values 4 c .. 4 c + 3 of row r.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 lds_column4(const char* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
}

// A tile as the second operand of a product that contracts over its rows.  PARTS = 2: bfloat16 halves whose sum keeps 16 bits.
template <class T, int PARTS> struct Operand {
  bf16x8 part[PARTS][2];
  __device__ __forceinline__ void set(const f32x16& x) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bf16_t hi = (bf16_t)x[i];
      part[0][i >> 3][i & 7] = hi;
      if constexpr (PARTS == 2) part[1][i >> 3][i & 7] = (bf16_t)(x[i] - (float)hi);
    }
  }
};
template <int PARTS> struct Operand<float, PARTS> {
  f32x16 x;
  __device__ __forceinline__ void set(const f32x16& v) { x = v; }
};

// acc[j][] += (32 rows of D values at `rows`, transposed) * x[j];  at: this lane's place, Rows::transposed.
template <int D, int PARTS, int N>
__device__ __forceinline__ void mul_transposed(f32x16 (&acc)[N][D / 32], const char* rows, const Operand<bf16_t, PARTS> (&x)[N]) {
  constexpr int S = Rows<bf16_t, D>::kStride;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const char* p = rows + 16 * kb * S + d * 64;
      const s16x4 lo = lds_column4(p), up = lds_column4(p + 8 * S);
      const bf16x8 a = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int q = 0; q < PARTS; ++q) acc[j][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, x[j].part[q][kb], acc[j][d], 0, 0, 0);
    }
}
template <int D, int PARTS, int N>
__device__ __forceinline__ void mul_transposed(f32x16 (&acc)[N][D / 32], const char* rows, const Operand<float, PARTS> (&x)[N]) {
  constexpr int S = Rows<float, D>::kStride;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const float a = *reinterpret_cast<const float*>(rows + (8 * (i >> 2) + (i & 3)) * S + d * 128);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j][d] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, x[j].x[i], acc[j][d], 0, 0, 0);
    }
}

// ---- rows in memory -----------------------------------------------------------------------------------
// n rows from p on, `stride` bytes apart; reads past the last one give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* p, int n, int stride, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, n > 0 ? (n - 1) * stride + bytes : 0, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int at) { return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0); }

// The largest of x over a lane and its partner 32 lanes on, and their sum.
__device__ __forceinline__ float both_max(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
__device__ __forceinline__ float both_sum(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}

// ---- sequences and their tiles ------------------------------------------------------------------------
struct Seq {
  int b, first, n;     // batch, first token, tokens
  int tile, id;        // row tile within it; the sequence's number (-1: none)
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Tile `slot` of all sequences' tiles of `rows` rows, a sequence's last tile first if `back`.  With starts, a wave adds up
// the tiles of 64 sequences at a time.
__device__ __forceinline__ Seq find_tile(const AttnArgs& a, int slot, int rows, bool back) {
  Seq s;
  s.id = -1;
  if (a.starts == nullptr) {
    const int per = (int)(((unsigned)a.T + rows - 1) / rows);
    s.b = slot / per;
    s.first = 0;
    s.n = a.T;
    if (a.lens != nullptr) s.n = min(max(uniform(a.lens[s.b]), 0), a.T);
    s.tile = slot - s.b * per;
    if (back) s.tile = per - 1 - s.tile;
    if ((long long)s.tile * rows < s.n) s.id = s.b;
    return s;
  }
  s.b = 0;
  int left = slot;
  for (int base = 0; base < a.S; base += 64) {
    const int i = base + lane_id();
    int first = 0, n = 0;
    if (i < a.S) {
      first = min(max(a.starts[i], 0), a.T);
      n = max(min(a.starts[i + 1], a.T) - first, 0);
    }
    const int tiles = (int)(((unsigned)n + rows - 1) / rows);
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(upto, o, 64);
      if (lane_id() >= o) upto += u;
    }
    const unsigned long long past = __ballot(upto > left);
    if (past != 0) {
      const int j = __ffsll((unsigned long long)past) - 1;
      s.first = __builtin_amdgcn_readlane(first, j);
      s.n = __builtin_amdgcn_readlane(n, j);
      const int end = __builtin_amdgcn_readlane(upto, j);
      s.tile = back ? end - 1 - left : left - end + (int)(((unsigned)s.n + rows - 1) / rows);
      s.id = base + j;
      return s;
    }
    left -= __builtin_amdgcn_readlane(upto, 63);
  }
  return s;
}

// ---- forward ------------------------------------------------------------------------------------------
// NW waves of 32 QT queries; keys in tiles of BN, two of them in LDS: a tile is stored while the one before is
// computed on, and its successor is already on the way to registers.
template <class T, int D, int QT, int NW, int BN, int PARTS>
struct FwdTile {
  using R = Rows<T, D>;
  static constexpr int kThreads = 64 * NW, kRows = 32 * QT * NW;
  static constexpr int kEach = BN * R::kPieces / kThreads;           // pieces per thread of one tile
  static constexpr int kTile = BN * R::kStride;
  static constexpr int kLds = 4 * kTile;
  static_assert(BN * R::kPieces % kThreads == 0, "whole pieces");
};

// The running maximum moves only when it grows by more than this (in powers of 2): p stays below 2^8, and o is rescaled
// a few times per row rather than with every tile.
constexpr float kSlack = 8.f;

template <class T, int D, int QT, int NW, int BN, int PARTS>
__global__ __launch_bounds__(64 * NW, QT * D * (int)sizeof(T) > 256 ? 1 : 2) void fwd_kernel(AttnArgs a) {
  using F = FwdTile<T, D, QT, NW, BN, PARTS>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  // heads of a group lie S G blocks apart (or G): with a multiple of 8 they share an XCD and the keys in its L2
  const int heads = a.H, slot0 = (int)(blockIdx.x / heads), pair = (int)(blockIdx.x - (unsigned)slot0 * heads);
  const int rep = a.H / a.G, head = (pair % a.G) * rep + pair / a.G, group = pair % a.G;
  const Seq s = find_tile(a, slot0, F::kRows, a.causal);
  if (s.id < 0) return;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int q0 = s.tile * F::kRows, qw = q0 + w * 32 * QT;            // the block's and the wave's first query
  const long long e = sizeof(T);

  // Q: the second operand of S^T = K Q^T
  u32x4 qf[QT][R::kSteps];
  {
    const char* p = (const char*)a.q + (s.b * a.qs.b + head * a.qs.h + (long long)(s.first + qw) * a.qs.t) * e;
    const int stride = (int)(a.qs.t * e);
    const auto r = rows_of(p, min(32 * QT, s.n - qw), stride, R::kBytes);
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int k = 0; k < R::kSteps; ++k) qf[t][k] = load16(r, (32 * t + (l & 31)) * stride + (2 * k + h) * 16);
  }

  const int qlast = min(q0 + F::kRows, s.n) - 1;
  const int jend = a.causal ? qlast + 1 : s.n;                        // the block's keys: jbeg .. jend - 1
  const int jbeg = a.window > 0 ? max(q0 - a.window + 1, 0) : 0;
  const int t0 = jbeg / BN, t1 = (jend + BN - 1) / BN;

  u32x4 sk[F::kEach], sv[F::kEach];
  const int srow = tid / R::kPieces, spiece = tid % R::kPieces;
  constexpr int kStep = F::kThreads / R::kPieces;                     // rows between a thread's pieces
  const int kst = (int)(a.ks.t * e), vst = (int)(a.vs.t * e);
  const char* kp = (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)s.first * a.ks.t) * e;
  const char* vp = (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)s.first * a.vs.t) * e;
  const auto load = [&](int t) {
    const int n = min(BN, s.n - t * BN);
    const auto rk = rows_of(kp + (long long)t * BN * kst, n, kst, R::kBytes);
    const auto rv = rows_of(vp + (long long)t * BN * vst, n, vst, R::kBytes);
#pragma unroll
    for (int i = 0; i < F::kEach; ++i) sk[i] = load16(rk, (srow + i * kStep) * kst + spiece * 16);
#pragma unroll
    for (int i = 0; i < F::kEach; ++i) sv[i] = load16(rv, (srow + i * kStep) * vst + spiece * 16);
  };
  load(t0);

  f32x16 o[QT][D / 32];
  float m[QT], sum[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = -kInf, sum[t] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[t][d] = zero16();
  }
  const float c = a.scale * kLog2e;
  const int rrow = R::by_rows(l), rcol = R::transposed(l), wat = srow * R::kStride + spiece * 16;

  for (int t = t0; t < t1; ++t) {
    char* kt = lds + (t & 1) * F::kTile;
    char* vt = kt + 2 * F::kTile;
#pragma unroll
    for (int i = 0; i < F::kEach; ++i) {
      *reinterpret_cast<u32x4*>(kt + wat + i * kStep * R::kStride) = sk[i];
      *reinterpret_cast<u32x4*>(vt + wat + i * kStep * R::kStride) = sv[i];
    }
    __syncthreads();
    if (t + 1 < t1) load(t + 1);
    const int j0 = t * BN;
    if (a.causal && j0 > qw + 32 * QT - 1) continue;                  // nothing for this wave's queries

    f32x16 x[NT][QT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < QT; ++q) x[n][q] = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4 f = lds16(kt + rrow + n * 32 * R::kStride + k * 32);
#pragma unroll
        for (int q = 0; q < QT; ++q) mma(x[n][q], f, qf[q][k], T());
      }
    // keys that not all of the wave's queries see
    const bool edge = j0 + BN > s.n || (a.causal && j0 + BN - 1 > qw) || (a.window > 0 && j0 <= qw + 32 * QT - 1 - a.window);
    if (edge) {
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const int i = qw + 32 * q + (l & 31);
        const int last = (a.causal ? min(i, s.n - 1) : s.n - 1) - j0 - 4 * h;
        const int first = (a.window > 0 ? i - a.window + 1 : 0) - j0 - 4 * h;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = 32 * n + 8 * (r >> 2) + (r & 3);
            x[n][q][r] = j <= last && j >= first ? x[n][q][r] : -kInf;
          }
      }
    }
    Operand<T, PARTS> p[NT][QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      float top = -kInf;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, x[n][q][r]);
      top = both_max(top);
      const bool grows = top > m[q] && !((top - m[q]) * c <= kSlack);
      if (__any(grows)) {
        const float to = grows ? top : m[q];
        const float f = to == m[q] ? 1.f : __builtin_amdgcn_exp2f((m[q] - to) * c);
        m[q] = to;
        sum[q] *= f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[q][d] *= f;
      }
      const float shift = m[q] == -kInf ? 0.f : m[q] * c;
      float part = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          x[n][q][r] = __builtin_amdgcn_exp2f(fmaf(x[n][q][r], c, -shift));
          part += x[n][q][r];
        }
        p[n][q].set(x[n][q]);
      }
      sum[q] += part;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) mul_transposed<D, PARTS, QT>(o, vt + rcol + n * 32 * R::kStride, p[n]);
  }

#pragma unroll
  for (int q = 0; q < QT; ++q) {
    const int i = qw + 32 * q + (l & 31);
    const float total = both_sum(sum[q]), f = total > 0.f || total != total ? 1.f / total : 0.f;
    if (i >= s.n) continue;
    char* p = (char*)a.o + (s.b * a.os.b + head * a.os.h + (long long)(s.first + i) * a.os.t) * e;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        T y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = (T)(o[q][d][4 * r + u] * f);
        __builtin_memcpy(p + (32 * d + 8 * r + 4 * h) * e, y, sizeof(y));
      }
    if (a.lse != nullptr && h == 0)
      a.lse[((long long)s.b * a.H + head) * a.T + s.first + i] = total == 0.f ? -kInf : (m[q] * c + __builtin_amdgcn_logf(total)) * kLn2;
  }
}

}  // namespace attn
}  // namespace prism
