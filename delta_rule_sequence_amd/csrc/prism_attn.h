// prism_attn.h - softmax attention of a prompt's rows (gfx950), forward.
//
//   s_ij = scale <q_i, k_j>,  o_i = sum_j e^(s_ij - m_i) v_j / l_i,  l_i = sum_j e^(s_ij - m_i),  lse_i = m_i + log l_i
// over the keys j <= i of i's sequence (causal), j > i - window, in one pass over the keys with a running m and l.
//
// A wave owns 32 queries and forms transposed tiles: S^T = K Q^T puts one query into a lane (and its partner 32 lanes on),
// so that m, l and the rescaling of o are single registers, and the tile's accumulators are, rounded, the second
// operand of O^T = V^T P^T without leaving their lane.  Q stays in registers; tiles of K and V go through LDS, read by
// rows (K) and transposed on the way (V).
//
// Rounding: q, k, v are exact operands; p passes as one bfloat16 part in the kernel of many rows, off by 2^-8 of a term at most:
// o is then off by 0.0021 of its size where a float32 p would leave 0.0016, its own rounding.  Two parts (0.0017) take a second
// product with V: 1 x 16 x 16384 of 128 1.46 ms for 1.06, 2 x 16 x 8192 of 64 509 us for 320 (15 registers go to scratch), 4 x 16 x 4096
// of 128 399 for 294.  The kernel of few rows waits for bytes and passes two.
//
// Bounds, bfloat16: heads of 128 run at 0.87 of a large matrix product's rate (1 x 16 x 16384 causal, 1050 us: 1047 of 1200 TFLOP/s), the
// matrix cores busy for 42 % of the cycles at 2.4 GHz (that product's: 48).  Heads of 64 (860 TFLOP/s at 2 x 16 x 8192) spend as many cycles on a tile's 62 to 90
// vector instructions, 16 exponentials among them, as on its 8 matrix instructions, and the two overlap in part only.  64 queries to a wave (355
// for 900 TFLOP/s at 128: registers), wave priorities and a fixed interleaving of the two kinds gained nothing or lost 5 to 10 %.
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

// x, formed again at each place rather than held in a register from one to the next.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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

// Rows of D values in LDS, PAD bytes between them.  A read by rows wants 16 rows' 16-byte pieces in different ones of
// the 64 banks, a transposed one four rows' 64 bytes (float32: two rows' 128, four rows apart); kBoth is two-way for either.
constexpr int kBoth = 32, kByRows = 16;
template <class T, int D> constexpr int kTransposed = sizeof(T) == 4 ? 32 : D == 32 ? 0 : 64;
template <class T, int D, int PAD = kBoth> struct Rows {
  static constexpr int kBytes = D * (int)sizeof(T), kStride = kBytes + PAD;
  static constexpr int kPieces = kBytes / 16, kSteps = kPieces / 2;
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
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) part[q][i >> 3][i & 7] = (bf16_t)((float)part[q][i >> 3][i & 7] * f);
  }
};
template <int PARTS> struct Operand<float, PARTS> {
  f32x16 x;
  __device__ __forceinline__ void set(const f32x16& v) { x = v; }
  __device__ __forceinline__ void scale(float f) { x *= f; }
};

// acc += (32 rows of D values at `rows` + this lane's place, Rows::transposed) * x
template <int D, int PARTS, int PAD = kBoth>
__device__ __forceinline__ void mul_transposed(f32x16 (&acc)[D / 32], const char* rows, const Operand<bf16_t, PARTS>& x) {
  constexpr int S = Rows<bf16_t, D, PAD>::kStride;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const char* p = rows + 16 * kb * S + d * 64;
      const s16x4 lo = lds_column4(p), up = lds_column4(p + 8 * S);
      const bf16x8 a = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int q = 0; q < PARTS; ++q) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, x.part[q][kb], acc[d], 0, 0, 0);
    }
}
template <int D, int PARTS, int PAD = kBoth>
__device__ __forceinline__ void mul_transposed(f32x16 (&acc)[D / 32], const char* rows, const Operand<float, PARTS>& x) {
  constexpr int S = Rows<float, D, PAD>::kStride;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const float a = *reinterpret_cast<const float*>(rows + (8 * (i >> 2) + (i & 3)) * S + d * 128);
      acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, x.x[i], acc[d], 0, 0, 0);
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

// Rows of an accumulator tile whose columns are rows of the tensor: 4 values at a time.
template <class T, int D>
__device__ __forceinline__ void store_columns(char* row, const f32x16 (&acc)[D / 32], float f, int h) {
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      T y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) y[u] = (T)(acc[d][4 * r + u] * f);
      __builtin_memcpy(row + (32 * d + 8 * r + 4 * h) * (int)sizeof(T), y, sizeof(y));
    }
}

// ---- sequences and their tiles ------------------------------------------------------------------------
struct Seq {
  int b, first, n;     // batch, first token, tokens
  int tile, id;        // row tile within it; the sequence's number (-1: none)
  int head, group;     // head within its group, group
};

// Unit `unit` of all sequences' tiles of `rows` rows, `each` rows per token, times `rep` heads of G groups; a sequence's last tile first if `back`.
// The tiles that take longest come first, and blocks that read the same rows of a group lie a multiple of G (where the
// sequences are batches: of B G) apart: with a multiple of 8 they share an XCD and the rows in its L2.  With starts, a wave adds up
// the tiles of 64 sequences at a time.
__device__ __forceinline__ Seq find_tile(const AttnArgs& a, unsigned unit, int rows, int rep, bool back, int each = 1) {
  Seq s;
  s.id = -1;
  const unsigned G = (unsigned)a.G;
  if (a.starts == nullptr) {
    const unsigned per = ((unsigned)a.T * each + rows - 1) / rows, all = (unsigned)a.B * G, tile = unit / (all * rep);
    unit -= tile * all * rep;
    s.head = (int)(unit / all);
    unit -= s.head * all;
    s.b = (int)(unit / G);
    s.group = (int)(unit - s.b * G);
    s.first = 0;
    s.n = a.T;
    if (a.lens != nullptr) s.n = min(max(uniform(a.lens[s.b]), 0), a.T);
    s.tile = (int)(back ? per - 1 - tile : tile);
    if ((long long)s.tile * rows < (long long)s.n * each) s.id = s.b;
    return s;
  }
  const unsigned slot = unit / (G * rep);
  unit -= slot * G * rep;
  s.head = (int)(unit / G);
  s.group = (int)(unit - s.head * G);
  s.b = 0;
  int left = (int)slot;
  for (int base = 0; base < a.S; base += 64) {
    const int i = base + lane_id();
    int first = 0, n = 0;
    if (i < a.S) {
      first = min(max(a.starts[i], 0), a.T);
      n = max(min(a.starts[i + 1], a.T) - first, 0);
    }
    const int tiles = (int)(((unsigned)n * each + rows - 1) / rows);
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
      s.tile = back ? end - 1 - left : left - end + (int)(((unsigned)s.n * each + rows - 1) / rows);
      s.id = base + j;
      return s;
    }
    left -= __builtin_amdgcn_readlane(upto, 63);
  }
  return s;
}

// ---- forward ------------------------------------------------------------------------------------------
// Where the keys lie: kPrompt: rows of k and v; kCache: pages of the same type; kCache8: pages of e4m3 bytes with a scale
// per row.
enum Keys { kPrompt, kCache, kCache8 };

// NW waves of 32 queries; keys in tiles of BN, three of K and three of V in LDS.  Step t computes on tile t, stores
// tile t + 2 of K and t + 1 of V, and asks for the ones behind them.  (A spacing of 32 bytes for both kinds, two-way for either read,
// took 1 to 4 % longer: 1 x 16 x 16384 of 128 2 %.)
template <class T, int D, int NW, int BN, Keys KEYS>
struct FwdTile {
  using K = Rows<T, D, kByRows>;
  using V = Rows<T, D, kTransposed<T, D>>;
  static constexpr int kThreads = 64 * NW, kRows = 32 * NW;
  static constexpr int kKeys = BN * K::kStride, kValues = BN * V::kStride;
  static constexpr int kScales = KEYS == kCache8 ? 6 * BN * 4 : 0;
  static constexpr int kZero = 32 * V::kStride;                        // rows of zeros
  static constexpr int kValuesAt = 3 * kKeys, kZeroAt = kValuesAt + 3 * kValues, kScalesAt = kZeroAt + kZero;
  static constexpr int kLds = kScalesAt + kScales;
};

// Eight e4m3 values as bfloat16, exactly.
__device__ __forceinline__ u32x4 widen8(unsigned lo, unsigned hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 r;
  r[0] = __builtin_bit_cast(unsigned, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
  r[1] = __builtin_bit_cast(unsigned, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
  r[2] = __builtin_bit_cast(unsigned, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
  r[3] = __builtin_bit_cast(unsigned, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  return r;
}

// The pages of a tile's groups of 16 rows (a page has at least that many), asked for one tile ahead.
template <int BN> struct Pages {
  typedef int Ids __attribute__((ext_vector_type(BN / 16)));
  Ids id;
  // Tile t; t1: the tiles' end, n: the keys.
  __device__ __forceinline__ void ask(const AttnArgs& a, const int* table, int t, int t1, int n) {
#pragma unroll
    for (int g = 0; g < BN / 16; ++g) id[g] = t < t1 && t * BN + 16 * g < n ? table[(t * BN + 16 * g) >> a.page_shift] : -1;
  }
  __device__ __forceinline__ Pages now() const {
    Pages p;
#pragma unroll
    for (int g = 0; g < BN / 16; ++g) p.id[g] = uniform(id[g]);
    return p;
  }
  __device__ __forceinline__ int of(int row) const {
    int p = id[0];
#pragma unroll
    for (int g = 1; g < BN / 16; ++g) p = row >= 16 * g ? id[g] : p;
    return p;
  }
};

// A tile's pieces of K or V (and rows' scales) between memory and LDS.
template <class T, int D, int NT, int BN, Keys KEYS> struct KeyTile {
  using R = Rows<T, D>;
  static constexpr int kPieces = KEYS == kCache8 ? D / 16 : R::kPieces;    // 16-byte pieces of a row in memory
  static constexpr int kEach = (BN * kPieces + NT - 1) / NT;               // per thread
  static constexpr int kStep = NT / kPieces;                               // rows between a thread's pieces
  static constexpr bool kPart = BN * kPieces < NT;                         // not every thread has a piece
  static_assert(BN * kPieces % NT == 0 || kPart, "whole pieces");
  static_assert(BN <= NT, "a scale per thread");
  u32x4 x[kEach];
  float scale;

  // Rows from p on, n of them in the sequence; what lies behind is zeros.
  __device__ __forceinline__ void load_prompt(const char* p, int stride, int n, int tid) {
    const int row = tid / kPieces, at = tid % kPieces * 16;
    const auto r = rows_of(p, min(n, BN), stride, R::kBytes);
    if (kPart && row >= BN) return;
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = load16(r, (row + i * kStep) * stride + at);
  }
  // Rows from j0 on of the sequence's pages; rows from `n` on and those of pages outside the cache are zeros.  pages: those of
  // the tile's groups of 16 rows.
  __device__ __forceinline__ void load_cache(const AttnArgs& a, const void* cache, const float* scales, const Pages<BN>& pages,
                                             int group, int j0, int n, int tid) {
    const int row = tid / kPieces, at = tid % kPieces * 16, page = 1 << a.page_shift;
    constexpr int kBytes = kPieces * 16;
    if (page >= BN) {                                                 // one page
      const bool in = (unsigned)pages.id[0] < (unsigned)a.pages;
      const size_t first = ((size_t)(in ? pages.id[0] : 0) * a.G + group) * page + (j0 & (page - 1));
      const auto r = rows_of((const char*)cache + first * kBytes, in ? min(n - j0, BN) : 0, kBytes, kBytes);
      if (!kPart || row < BN) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) x[i] = load16(r, (row + i * kStep) * kBytes + at);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = row + i * kStep, j = j0 + r, p = pages.of(r);
        x[i] = u32x4{0, 0, 0, 0};
        if ((!kPart || row < BN) && j < n && (unsigned)p < (unsigned)a.pages)
          x[i] = *reinterpret_cast<const u32x4*>((const char*)cache + (((size_t)p * a.G + group) * page + (j & (page - 1))) * kBytes + at);
      }
    }
    if constexpr (KEYS == kCache8) {
      const int j = j0 + tid, p = pages.of(tid & (BN - 1));
      scale = 0.f;
      if (tid < BN && j < n && (unsigned)p < (unsigned)a.pages) scale = scales[((size_t)p * a.G + group) * page + (j & (page - 1))];
    }
  }
  template <int STRIDE> __device__ __forceinline__ void store(char* tile, float* scales, int tid) const {
    const int row = tid / kPieces, at = tid % kPieces;
    if (!kPart || row < BN) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        char* const p = tile + (row + i * kStep) * STRIDE;
        if constexpr (KEYS == kCache8) {
          *reinterpret_cast<u32x4*>(p + at * 32) = widen8(x[i][0], x[i][1]);
          *reinterpret_cast<u32x4*>(p + at * 32 + 16) = widen8(x[i][2], x[i][3]);
        } else {
          *reinterpret_cast<u32x4*>(p + at * 16) = x[i];
        }
      }
    }
    if constexpr (KEYS == kCache8)
      if (tid < BN) scales[tid] = scale;
  }
};

// Up to this the rounding of m c moves the exponent of a row's p, all alike, by 2^-8 at most (past 2^31: to infinity).
constexpr float kFar = 65536.f;

// The running maximum moves only when it grows by more than this (in powers of 2): p stays below 2^8, and o is rescaled
// a few times per row rather than with every tile.
constexpr float kSlack = 8.f;

// lse from the maximum score and the sum of a row.
__device__ __forceinline__ float row_lse(float m, float sum, float scale) {
  if (sum == 0.f) return -kInf;
  const float c = scale * kLog2e, log2 = __builtin_amdgcn_logf(sum);
  return fabsf(m * c) > kFar ? m * scale + log2 * kLn2 : (m * c + log2) * kLn2;
}

// Four neighbouring values of a row of keys or values, times its scale.
template <class T, Keys KEYS>
__device__ __forceinline__ f32x4 row4(const char* row, int d, float scale) {
  f32x4 r;
  if constexpr (KEYS == kCache8) {
    const int w = *reinterpret_cast<const int*>(row + d);
    r[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0), r[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
    r[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2), r[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] *= scale;
  } else {
    T x[4];
    __builtin_memcpy(x, row + d * (int)sizeof(T), sizeof(x));
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] = (float)x[u];
  }
  return r;
}

// A wave's rows once more, key by key: what a tile does to a row that its keys hide from it (0 times an infinity or a NaN),
// and scores beyond kFar, call for it.  The scores are those of the tiles, bit for bit: an lse of 10^9 has to meet the same
// ones in the backward.  The keys: tiles t0, t0 + step, ... < t1 of 32 keys, of n keys altogether, first .. last of them
// for this lane's row; kp, vp, table as in the kernels.  m, sum and o as the tiles leave them.
template <class T, int D, Keys KEYS, int STEPS>
__device__ __forceinline__ void careful_rows(const AttnArgs& a, const u32x4 (&qf)[STEPS], const char* kp, const char* vp, long long kst,
                                          long long vst, const int* table, int group, int t0, int t1, int step, int n,
                                          int first, int last, float& m, float& sum, f32x16 (&o)[D / 32]) {
  const int l = lane_id(), h = l >> 5, page = 1 << a.page_shift;
  constexpr int kBytes = KEYS == kCache8 ? D : D * (int)sizeof(T);
  const float c = a.scale * kLog2e;
  // a row of the cache; -1: of a page outside it
  const auto row_of = [&](int j) -> long long {
    const int id = table[j >> a.page_shift];
    return (unsigned)id < (unsigned)a.pages ? ((long long)id * a.G + group) * page + (j & (page - 1)) : -1;
  };
  m = -kInf, sum = 0.f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) o[d] = zero16();
  for (int t = t0; t < t1; t += step) {
    f32x16 x = zero16();
    {
      const int j = t * 32 + (l & 31);
      const char* k = j < n ? kp + j * kst : nullptr;
      float f = 0.f;
      if constexpr (KEYS != kPrompt) {
        const long long r = j < n ? row_of(j) : -1;
        k = r >= 0 ? (const char*)a.cache_k + r * kBytes : nullptr;
        if constexpr (KEYS == kCache8) f = r >= 0 ? a.cache_ks[r] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        u32x4 y = {0, 0, 0, 0};
        if (k != nullptr) {
          if constexpr (KEYS == kCache8) {
            unsigned w[2];
            __builtin_memcpy(w, k + (2 * i + h) * 8, 8);
            y = widen8(w[0], w[1]);
          } else {
            y = *reinterpret_cast<const u32x4*>(k + (2 * i + h) * 16);
          }
        }
        mma(x, y, qf[i], T());
      }
      if constexpr (KEYS == kCache8) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] *= __shfl(f, 8 * (r >> 2) + 4 * h + (r & 3), 64);
      }
    }
    for (int jj = 0; jj < 32; ++jj) {
      const int j = t * 32 + jj;
      const bool in = j >= first && j <= last;
      if (!__any(in)) continue;
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) s = r == 4 * (jj >> 3) + (jj & 3) ? x[r] : s;
      s = __shfl(s, (l & 31) + 32 * (jj >> 2 & 1), 64);
      const char* v = vp + j * vst;
      float vs = 1.f;
      if constexpr (KEYS != kPrompt) {
        const long long r = row_of(j);
        v = r >= 0 ? (const char*)a.cache_v + r * kBytes : nullptr;
        if constexpr (KEYS == kCache8) vs = r >= 0 ? a.cache_vs[r] : 0.f;
      }
      if (!in) continue;
      const float to = fmaxf(m, s), ref = to == -kInf ? 0.f : to;
      const float f = to == m ? 1.f : __builtin_amdgcn_exp2f((m - ref) * c), p = __builtin_amdgcn_exp2f((s - ref) * c);
      m = to;
      sum = fmaf(sum, f, p);
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f32x4 y = zero4();
          if (v != nullptr) y = row4<T, KEYS>(v, 32 * d + 8 * r + 4 * h, vs);
#pragma unroll
          for (int u = 0; u < 4; ++u) o[d][4 * r + u] = o[d][4 * r + u] * f + p * y[u];
        }
    }
  }
  sum = h == 0 ? sum : 0.f;                                           // both lanes of a row have all of it
}
template <int N>
__device__ __forceinline__ bool finite(const f32x16 (&o)[N]) {
  bool ok = true;
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) ok &= fabsf(o[d][r]) < kInf;
  return ok;
}

// Shares of a row's result that the join kernel adds up: o before its division, and the maximum score and
// sum behind all rows' o: part = [splits][B H T][D], then [splits][B H T][2].
__device__ __forceinline__ size_t share(const AttnArgs& a, int split, const Seq& s, int head, int i) {
  return (((size_t)split * a.B + s.b) * a.H + head) * a.T + s.first + i;
}
__device__ __forceinline__ float* share_stats(const AttnArgs& a, int D, size_t row) {
  return a.part + (size_t)a.splits * a.B * a.H * a.T * D + 2 * row;
}

template <class T, int D, int NW, int BN, Keys KEYS>
__global__ __launch_bounds__(64 * NW, D * (int)sizeof(T) > 256 ? 1 : D * (int)sizeof(T) <= 128 && KEYS == kPrompt ? 4 : 2) void fwd_kernel(AttnArgs a) {
  using F = FwdTile<T, D, NW, BN, KEYS>;
  using R = Rows<T, D>;
  extern __shared__ __align__(16) char lds[];
  constexpr int NT = BN / 32;
  const unsigned unit = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - unit * a.splits;
  const int rep = a.H / a.G;
  const Seq s = find_tile(a, unit, F::kRows, rep, a.causal);
  if (s.id < 0) return;
  const int group = s.group, head = group * rep + s.head;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int q0 = s.tile * F::kRows, qw = q0 + w * 32;                 // the block's and the wave's first query
  const long long e = sizeof(T);
  // tokens in front of the first query, and keys altogether
  int past = 0, keys = s.n;
  if constexpr (KEYS != kPrompt) {
    const int room = a.max_pages << a.page_shift;
    past = min(max(uniform(a.past[s.b]), 0), room);
    keys = min(past + s.n, room);
  }

  // Q: the second operand of S^T = K Q^T
  u32x4 qf[R::kSteps];
  {
    const char* p = (const char*)a.q + (s.b * a.qs.b + head * a.qs.h + (long long)(s.first + qw) * a.qs.t) * e;
    const int stride = (int)(a.qs.t * e);
    const auto r = rows_of(p, min(32, s.n - qw), stride, R::kBytes);
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) qf[k] = load16(r, (l & 31) * stride + (2 * k + h) * 16);
  }

  // the block's keys jbeg .. jend - 1, and its share of their tiles
  const int qlast = min(q0 + F::kRows, s.n) - 1;
  const int jend = a.causal ? min(past + qlast + 1, keys) : keys;
  const int jbeg = a.window > 0 ? max(past + q0 - a.window + 1, 0) : 0;
  int t0 = jbeg / BN, t1 = max((jend + BN - 1) / BN, t0);
  if (a.splits > 1) {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + (int)split * per, t1);
    t1 = min(t0 + per, t1);
  }

  const int kst = (int)(a.ks.t * e), vst = (int)(a.vs.t * e);
  const char *kp = nullptr, *vp = nullptr;
  const int* table = nullptr;
  if constexpr (KEYS == kPrompt) {
    kp = (const char*)a.k + (s.b * a.ks.b + group * a.ks.h + (long long)s.first * a.ks.t) * e;
    vp = (const char*)a.v + (s.b * a.vs.b + group * a.vs.h + (long long)s.first * a.vs.t) * e;
  } else {
    table = a.table + (size_t)s.b * a.max_pages;
  }
  KeyTile<T, D, F::kThreads, BN, KEYS> nk, nv;
  Pages<BN> coming, of_v;                                             // pages of the tile after the last asked for, and of that one
  if constexpr (KEYS != kPrompt) coming.ask(a, table, t0, t1, keys);
  const auto load_k = [&](int t) {                                    // in the order of the tiles
    if constexpr (KEYS == kPrompt) {
      nk.load_prompt(kp + (long long)t * BN * kst, kst, keys - t * BN, tid);
    } else {
      of_v = coming.now();
      nk.load_cache(a, a.cache_k, a.cache_ks, of_v, group, t * BN, keys, tid);
      coming.ask(a, table, t + 1, t1, keys);
    }
  };
  const auto load_v = [&](int t) {                                    // behind load_k of the same tile
    if constexpr (KEYS == kPrompt) nv.load_prompt(vp + (long long)t * BN * vst, vst, keys - t * BN, tid);
    else nv.load_cache(a, a.cache_v, a.cache_vs, of_v, group, t * BN, keys, tid);
  };
  char* const v_tiles = lds + F::kValuesAt;
  float* const scales = reinterpret_cast<float*>(lds + F::kScalesAt);  // three of K, three of V

  f32x16 o[D / 32];
  float m = -kInf, sum = 0.f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) o[d] = zero16();
  const float c = a.scale * kLog2e;
  const int rrow = F::K::by_rows(l), rcol = F::V::transposed(l), pw = past + qw;
  // the keys first .. last that this lane's position sees, formed where they are needed: registers are short
  const auto seen = [&](int& first, int& last) {
    const int i = pw + (anew(l) & 31);
    last = a.causal ? min(i, keys - 1) : keys - 1, first = a.window > 0 ? i - a.window + 1 : 0;
  };
  const int wlast = a.causal ? min(pw + 31, keys - 1) : keys - 1;     // of all of the wave's positions
  const auto scores = [&](f32x16& x, const char* tile) {
    x = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(tile + rrow + k * 32), qf[k], T());
  };

  // 32 keys after another: while the exponentials of some are formed, the matrix cores form the scores of the next and the
  // products of the ones before with their values.
  f32x16 x[2];                                                        // scores of these keys, and of the next
  Operand<T, 1> p;                                             // p of the keys before
  p.set(zero16());
  // and their values: before the first ones and where p is empty, zeros (0 times an infinity would be NaN)
  char* const zeros = lds + F::kZeroAt;
  for (int z = tid * 16; z < F::kZero; z += F::kThreads * 16) *reinterpret_cast<u32x4*>(zeros + z) = u32x4{0, 0, 0, 0};
  const char* pv = zeros + rcol;
  int buf = 0;                                                        // tile t's place in LDS
  if (t0 < t1) {
    load_k(t0);
    load_v(t0);
    nk.template store<F::K::kStride>(lds, scales, tid);
    nv.template store<F::V::kStride>(v_tiles, scales + 3 * BN, tid);
    if (t0 + 1 < t1) {
      load_k(t0 + 1);
      nk.template store<F::K::kStride>(lds + F::kKeys, scales + BN, tid);
      load_v(t0 + 1);
    }
    if (t0 + 2 < t1) load_k(t0 + 2);
  }
  __syncthreads();
  if (t0 < t1) scores(x[0], lds);
  const auto stage = [&](int t, int buf1, int buf2) {
    if (t + 2 < t1) nk.template store<F::K::kStride>(lds + buf2 * F::kKeys, scales + buf2 * BN, tid);
    if (t + 1 < t1) nv.template store<F::V::kStride>(v_tiles + buf1 * F::kValues, scales + (3 + buf1) * BN, tid);
    if (t + 2 < t1) load_v(t + 2);
    if (t + 3 < t1) load_k(t + 3);
  };
  const int tw = min(t1, max(t0, wlast / BN + 1));                    // the wave's own tiles
  const auto tile = [&](int t, auto odd) {                            // odd: x[1] has the scores of the tile's first keys
    constexpr int X = decltype(odd)::value;
    if (t > t0) __syncthreads();
    const int buf1 = buf == 2 ? 0 : buf + 1, buf2 = buf1 == 2 ? 0 : buf1 + 1;
    stage(t, buf1, buf2);
    const char *kt = lds + buf * F::kKeys, *kn = lds + buf1 * F::kKeys, *vt = v_tiles + buf * F::kValues;
    const float *ks = scales + buf * BN, *vs = scales + (3 + buf) * BN;
    buf = buf1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j0 = t * BN + 32 * n;
      f32x16& y = x[(n + X) & 1];
      if constexpr (KEYS == kCache8) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(ks + 32 * n + 8 * r + 4 * h);
#pragma unroll
          for (int u = 0; u < 4; ++u) y[4 * r + u] *= f[u];
        }
      }
      // keys that not all of the wave's queries see
      if (j0 + 31 > (a.causal ? min(pw, keys - 1) : keys - 1) || (a.window > 0 && j0 <= pw + 31 - a.window)) {
        int first, last;
        seen(first, last);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = 8 * (r >> 2) + (r & 3) + j0 + 4 * h;
          y[r] = j <= last && j >= first ? y[r] : -kInf;
        }
      }
      float top = -kInf;
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, y[r]);
      top = both_max(top);
      const bool grows = top > m && !((top - m) * c <= kSlack);
      if (__any(grows)) {
        const float to = grows ? top : m;
        const float f = to == m ? 1.f : __builtin_amdgcn_exp2f((m - to) * c);
        m = to;
        sum *= f;
        p.scale(f);                                                // rounded once more, at 2^-8 of what comes now
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[d] *= f;
      }
      const float shift = m == -kInf ? 0.f : m * c;
      // behind the last keys: scores of whatever lies there, unused
      scores(x[(n + X + 1) & 1], n + 1 < NT ? kt + (n + 1) * 32 * F::K::kStride : kn);
      mul_transposed<D, 1, kTransposed<T, D>>(o, pv, p);
      pv = vt + rcol + n * 32 * F::V::kStride;
      float part = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        y[r] = __builtin_amdgcn_exp2f(fmaf(y[r], c, -shift));
        part += y[r];
      }
      sum += part;
      if constexpr (KEYS == kCache8) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(vs + 32 * n + 8 * r + 4 * h);
#pragma unroll
          for (int u = 0; u < 4; ++u) y[4 * r + u] *= f[u];
        }
      }
      p.set(y);
    }
  };
  int t = t0;
  if constexpr (NT % 2 == 1) {
    for (; t + 1 < tw; t += 2) {
      tile(t, std::integral_constant<int, 0>());
      tile(t + 1, std::integral_constant<int, 1>());
    }
  }
  for (; t < tw; ++t) tile(t, std::integral_constant<int, 0>());
  mul_transposed<D, 1, kTransposed<T, D>>(o, pv, p);
  for (; t < t1; ++t) {                                               // those of the block's other waves
    if (t > t0) __syncthreads();
    const int buf1 = buf == 2 ? 0 : buf + 1, buf2 = buf1 == 2 ? 0 : buf1 + 1;
    stage(t, buf1, buf2);
    buf = buf1;
  }
  const int iq = qw + (l & 31);
  int first, last;
  seen(first, last);
  if (__any(iq < s.n && (!finite(o) || !(fabsf(m * c) <= kFar || m == -kInf)))) {
    careful_rows<T, D, KEYS>(a, qf, kp, vp, kst, vst, table, group, t0 * NT, t1 * NT, 1, keys, first, iq < s.n ? last : -1, m, sum, o);
  }

  const float total = both_sum(sum);
  if (iq >= s.n) return;
  if (a.splits > 1) {
    const size_t row = share(a, split, s, head, iq);
    if (h == 0) share_stats(a, D, row)[0] = m, share_stats(a, D, row)[1] = total;
    store_columns<float, D>(reinterpret_cast<char*>(a.part + row * D), o, 1.f, h);
    return;
  }
  // a row without keys: zeros, and a logarithm of -infinity
  store_columns<T, D>((char*)a.o + (s.b * a.os.b + head * a.os.h + (long long)(s.first + iq) * a.os.t) * e, o,
                      total == 0.f ? 0.f : 1.f / total, h);
  if (a.lse != nullptr && h == 0) a.lse[((long long)s.b * a.H + head) * a.T + s.first + iq] = row_lse(m, total, a.scale);
}

// ---- few rows of queries --------------------------------------------------------------------------------
// The rows of a group's heads, token by token, lie in tiles of 32 rows, so that keys are read once for all of them.  Four
// waves take every fourth tile of 32 keys each, in LDS of their own, with a maximum, a sum and an o of their own, and join them
// at the end.  For single tokens, and for prompts that are too short to fill the device with a workgroup per 128 rows.
// Single tokens are bound by the cache's bytes (5.17 of the copy's 5.19 TB/s over 800 MB); a workgroup keeps 4 x 16 KB of loads in flight.
template <class T, int D, Keys KEYS> struct FewTile {
  using K = Rows<T, D, kByRows>;
  using V = Rows<T, D, kTransposed<T, D>>;
  static constexpr int kKeys = 32 * K::kStride, kTiles = kKeys + 32 * V::kStride;
  static constexpr int kOut = (D + 4) * 4, kJoin = 32 * kOut + 64 * 4;        // a row of o on its way to the join; all, and m, l
  static constexpr int kUsed = kTiles + (KEYS == kCache8 ? 64 * 4 : 0);       // keys, values, scales
  static constexpr int kWave = kUsed > kJoin ? kUsed : kJoin, kLds = 4 * kWave;
};

template <class T, int D, Keys KEYS>
__global__ __launch_bounds__(256, D * (int)sizeof(T) > 256 ? 1 : 2) void few_kernel(AttnArgs a) {
  using F = FewTile<T, D, KEYS>;
  using R = Rows<T, D>;
  constexpr int PARTS = 2;                                             // bound by bytes or latency: both are free
  extern __shared__ __align__(16) char lds[];
  const unsigned unit = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - unit * a.splits;
  const int rep = a.H / a.G;
  const Seq s = find_tile(a, unit, 32, 1, a.causal, rep);
  if (s.id < 0) return;
  const int group = s.group, tile = s.tile, b = s.b;
  const int first = tile * 32 / rep, lastq = min((tile * 32 + 31) / rep, s.n - 1);
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int r = tile * 32 + (l & 31), tq = r / rep, head = group * rep + (r - tq * rep);
  int past = 0, keys = s.n;
  if constexpr (KEYS != kPrompt) {
    const int room = a.max_pages << a.page_shift;
    past = min(max(uniform(a.past[b]), 0), room);
    keys = min(past + s.n, room);
  }
  const int jend = a.causal ? min(past + lastq + 1, keys) : keys, jbeg = a.window > 0 ? max(past + first - a.window + 1, 0) : 0;
  int t0 = jbeg / 32, t1 = max((jend + 31) / 32, t0);
  {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + (int)split * per, t1);
    t1 = min(t0 + per, t1);
  }
  const long long e = sizeof(T);
  const int kst = (int)(a.ks.t * e), vst = (int)(a.vs.t * e);
  const char *kp = nullptr, *vp = nullptr;
  const int* table = nullptr;
  if constexpr (KEYS == kPrompt) {
    kp = (const char*)a.k + (b * a.ks.b + group * a.ks.h + (long long)s.first * a.ks.t) * e;
    vp = (const char*)a.v + (b * a.vs.b + group * a.vs.h + (long long)s.first * a.vs.t) * e;
  } else {
    table = a.table + (size_t)b * a.max_pages;
  }

  u32x4 qf[R::kSteps];
#pragma unroll
  for (int k = 0; k < R::kSteps; ++k) {
    qf[k] = u32x4{0, 0, 0, 0};
    if (tq < s.n)
      qf[k] = *reinterpret_cast<const u32x4*>((const char*)a.q + (b * a.qs.b + head * a.qs.h + (long long)(s.first + tq) * a.qs.t) * e +
                                              (2 * k + h) * 16);
  }
  char* const kt = lds + w * F::kWave;
  char* const vt = kt + F::kKeys;
  float* const scales = reinterpret_cast<float*>(kt + F::kTiles);
  KeyTile<T, D, 64, 32, KEYS> nk, nv;
  Pages<32> coming;
  if constexpr (KEYS != kPrompt) coming.ask(a, table, t0 + w, t1, keys);
  const auto load = [&](int t) {
    if constexpr (KEYS == kPrompt) {
      nk.load_prompt(kp + (long long)t * 32 * kst, kst, keys - t * 32, l);
      nv.load_prompt(vp + (long long)t * 32 * vst, vst, keys - t * 32, l);
    } else {
      const Pages<32> pages = coming.now();
      nk.load_cache(a, a.cache_k, a.cache_ks, pages, group, t * 32, keys, l);
      nv.load_cache(a, a.cache_v, a.cache_vs, pages, group, t * 32, keys, l);
      coming.ask(a, table, t + 4, t1, keys);
    }
  };
  if (t0 + w < t1) load(t0 + w);

  f32x16 o[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) o[d] = zero16();
  float m = -kInf, sum = 0.f;
  const float c = a.scale * kLog2e;
  const int rrow = F::K::by_rows(l), rcol = F::V::transposed(l);
  const int i = tq < s.n ? past + tq : -1;                             // this lane's position
  for (int t = t0 + w; t < t1; t += 4) {
    nk.template store<F::K::kStride>(kt, scales, l);
    nv.template store<F::V::kStride>(vt, scales + 32, l);
    __builtin_amdgcn_wave_barrier();
    if (t + 4 < t1) load(t + 4);
    f32x16 x = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(kt + rrow + k * 32), qf[k], T());
    const int last = (a.causal ? min(i, keys - 1) : keys - 1) - t * 32 - 4 * h, from = (a.window > 0 ? i - a.window + 1 : 0) - t * 32 - 4 * h;
    float top = -kInf;
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      f32x4 f = {1.f, 1.f, 1.f, 1.f};
      if constexpr (KEYS == kCache8) f = *reinterpret_cast<const f32x4*>(scales + 8 * r4 + 4 * h);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = 8 * r4 + u, k = 4 * r4 + u;
        if constexpr (KEYS == kCache8) x[k] *= f[u];
        x[k] = j <= last && j >= from ? x[k] : -kInf;
        top = fmaxf(top, x[k]);
      }
    }
    top = both_max(top);
    const bool grows = top > m && !((top - m) * c <= kSlack);
    if (__any(grows)) {
      const float to = grows ? top : m;
      const float f = to == m ? 1.f : __builtin_amdgcn_exp2f((m - to) * c);
      m = to;
      sum *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= f;
    }
    const float shift = m == -kInf ? 0.f : m * c;
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      f32x4 f = {1.f, 1.f, 1.f, 1.f};
      if constexpr (KEYS == kCache8) f = *reinterpret_cast<const f32x4*>(scales + 32 + 8 * r4 + 4 * h);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = 4 * r4 + u;
        x[k] = __builtin_amdgcn_exp2f(fmaf(x[k], c, -shift));
        sum += x[k];
        if constexpr (KEYS == kCache8) x[k] *= f[u];
      }
    }
    Operand<T, PARTS> p;
    p.set(x);
    mul_transposed<D, PARTS, kTransposed<T, D>>(o, vt + rcol, p);
    __builtin_amdgcn_wave_barrier();
  }

  if (__any(tq < s.n && (!finite(o) || !(fabsf(m * c) <= kFar || m == -kInf)))) {
    careful_rows<T, D, KEYS>(a, qf, kp, vp, kst, vst, table, group, t0 + w, t1, 4, keys, a.window > 0 ? i - a.window + 1 : 0,
                          tq >= s.n ? -1 : a.causal ? min(i, keys - 1) : keys - 1, m, sum, o);
  }

  // the waves' shares through LDS
  const float total = both_sum(sum);
  store_columns<float, D>(kt + (l & 31) * F::kOut, o, 1.f, h);
  float* const stats = reinterpret_cast<float*>(kt + 32 * F::kOut);
  if (h == 0) stats[2 * (l & 31)] = m, stats[2 * (l & 31) + 1] = total;
  __syncthreads();
  const int row = tid >> 3, rr = tile * 32 + row, t = rr / rep, hd = group * rep + (rr - t * rep);
  if (t >= s.n) return;
  float mj = -kInf, sj = 0.f, f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float* st = reinterpret_cast<const float*>(lds + k * F::kWave + 32 * F::kOut) + 2 * row;
    if (st[1] != 0.f) mj = fmaxf(mj, st[0]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float* st = reinterpret_cast<const float*>(lds + k * F::kWave + 32 * F::kOut) + 2 * row;
    f[k] = st[1] == 0.f ? 0.f : __builtin_amdgcn_exp2f((st[0] - mj) * c);
    sj += f[k] * st[1];
  }
  const size_t at = share(a, split, s, hd, t);
  if (a.splits > 1 && (tid & 7) == 0) share_stats(a, D, at)[0] = mj, share_stats(a, D, at)[1] = sj;
  const float by = a.splits > 1 ? 1.f : sj == 0.f ? 0.f : 1.f / sj;
  if (a.splits == 1 && a.lse != nullptr && (tid & 7) == 0) a.lse[((long long)b * a.H + hd) * a.T + s.first + t] = row_lse(mj, sj, a.scale);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
    const int col = 32 * d + (tid & 7) * 4;
    f32x4 y = zero4();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(lds + k * F::kWave + row * F::kOut + col * 4);
#pragma unroll
      for (int u = 0; u < 4; ++u) y[u] = fmaf(f[k], v[u], y[u]);
    }
    if (a.splits > 1) {
      *reinterpret_cast<f32x4*>(a.part + at * D + col) = y;
    } else {
      T z[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) z[u] = (T)(y[u] * by);
      __builtin_memcpy((char*)a.o + (b * a.os.b + hd * a.os.h + (long long)(s.first + t) * a.os.t + col) * e, z, sizeof(z));
    }
  }
}

// Joins the shares of the rows, at most 64 of each: a wave per row, whose lanes weigh a share each and then take D / 4 columns of
// every (256 / D)-th share.  (Thread per four columns that walks the shares: 83 us for the two kernels where these take 39, 13 single
// tokens over 11610 in 22 shares.)
template <class T, int D>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a) {
  constexpr int L = D / 4, N = 64 / L;
  const size_t rows = (size_t)a.B * a.H * a.T, row = (size_t)blockIdx.x * 4 + wave_id();
  if (row >= rows) return;
  const int l = lane_id();
  const size_t bh = row / a.T;
  const int t = (int)(row - bh * a.T), b = (int)(bh / a.H), head = (int)(bh - (size_t)b * a.H);
  if (a.lens != nullptr && t >= uniform(a.lens[b])) return;
  const float* const stats = share_stats(a, D, row) + 2 * rows * l;
  float m = -kInf, total = 0.f;
  if (l < a.splits) m = stats[0], total = stats[1];
  if (total == 0.f) m = -kInf;
  float top = m;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  // an infinite maximum: what comes of it is NaN, as without shares
  const float f = total == 0.f ? 0.f : __builtin_amdgcn_exp2f((m - top) * (a.scale * kLog2e));
  float sum = f * total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
  const int at = l % L * 4;
  f32x4 o = zero4();
#pragma unroll 4
  for (int k = l / L; k < (a.splits + N - 1) / N * N; k += N) {
    const float w = __shfl(f, k, 64);                                  // 0 past the last share and of empty ones: not read
    f32x4 x = zero4();
    if (w != 0.f) x = *reinterpret_cast<const f32x4*>(a.part + (rows * k + row) * D + at);
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = fmaf(w, x[u], o[u]);
  }
#pragma unroll
  for (int d = L; d < 64; d <<= 1)
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] += __shfl_xor(o[u], d, 64);
  if (l >= L) return;
  T y[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) y[u] = (T)(sum == 0.f ? 0.f : o[u] / sum);
  __builtin_memcpy((char*)a.o + (b * a.os.b + head * a.os.h + (long long)t * a.os.t + at) * (long long)sizeof(T), y, sizeof(y));
}

}  // namespace attn
}  // namespace prism
