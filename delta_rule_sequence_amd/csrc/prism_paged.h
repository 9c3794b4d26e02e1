// prism_paged.h - the paged cache of keys and values (gfx950): rows are written to it, and few rows of queries read it.
//
// Position p of a sequence lies in page table[p / page], row p % page of its group.  With 8 bits a row x is held as e4m3
// bytes of x / scale, scale = max |x| / 448.
#pragma once
#include "prism_attn.h"
#include "prism_e4m3.h"

namespace prism {
namespace attn {

// ---- write ----------------------------------------------------------------------------------------------
// A workgroup takes kWriteTokens tokens of a sequence, all groups, keys and values; a row lies in D / 8 or D / 4 lanes.
constexpr int kWriteTokens = 16;

template <class T, int D, bool BITS8>
__global__ __launch_bounds__(256) void cache_write_kernel(AttnArgs a) {
  const int G = a.G;
  constexpr int V = 16 / (int)sizeof(T), L = D / V;
  typedef T vec __attribute__((ext_vector_type(V)));
  a.G = 1;                                                            // tiles of all groups at once
  const Seq s = find_tile(a, blockIdx.x, kWriteTokens, 1, false);
  if (s.id < 0) return;
  const int t0 = s.tile * kWriteTokens, n = min(kWriteTokens, s.n - t0), at = threadIdx.x % L;
  const long long past = max(a.past[s.id], 0);
  const int* table = a.table + (size_t)s.id * a.max_pages;
  const int page = 1 << a.page_shift;
  for (int r = threadIdx.x / L; r < n * 2 * G; r += 256 / L) {
    const int g = r % G, tk = r / G, t = t0 + (tk >> 1);
    const bool key = (tk & 1) == 0;
    const long long p = past + t;
    if (p >> a.page_shift >= a.max_pages) continue;
    const int id = table[p >> a.page_shift];
    if ((unsigned)id >= (unsigned)a.pages) continue;
    const prism_strides st = key ? a.ks : a.vs;
    const vec x = *reinterpret_cast<const vec*>((const T*)(key ? a.k : a.v) + (s.b * st.b + g * st.h + (long long)(s.first + t) * st.t) + at * V);
    const size_t row = ((size_t)id * G + g) * page + (p & (page - 1));
    void* const cache = key ? a.cache_k : a.cache_v;
    if constexpr (!BITS8) {
      *reinterpret_cast<vec*>((T*)cache + row * D + at * V) = x;
    } else {
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, norm::abs_bits((float)x[i]));
#pragma unroll
      for (int o = 1; o < L; o <<= 1) m = max(m, (unsigned)__shfl_xor((int)m, o, 64));
      float f;
      const float scale = norm::block_scale(m, &f);
      unsigned y[V / 4];
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32((float)x[4 * i] * f, (float)x[4 * i + 1] * f, 0, false);
        y[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32((float)x[4 * i + 2] * f, (float)x[4 * i + 3] * f, w, true);
      }
      __builtin_memcpy((char*)cache + row * D + at * V, y, sizeof(y));
      if (at == 0) (key ? a.cache_ks : a.cache_vs)[row] = scale;
    }
  }
}

// ---- few rows of queries --------------------------------------------------------------------------------
// The rows of a group's heads, token by token, are one tile of 32 rows, so the cache is read once for all of them.  Four
// waves take every fourth tile of 32 keys each, with a maximum, a sum and an o of their own, and join them at the end.
template <class T, int D, Keys KEYS> struct FewTile {
  using R = Rows<T, D>;
  static constexpr int kTile = 32 * R::kStride;
  static constexpr int kWave = 2 * kTile + (KEYS == kCache8 ? 64 * 4 : 0);   // keys, values, scales
  static constexpr int kOut = (D + 4) * 4;                                    // a row of o on its way to the join
  static constexpr int kLds = 4 * kWave;
  static_assert(32 * kOut + 64 * 4 <= kWave, "the join fits");
};

template <class T, int D, Keys KEYS>
__global__ __launch_bounds__(256, D * (int)sizeof(T) > 256 ? 1 : 2) void few_kernel(AttnArgs a) {
  using F = FewTile<T, D, KEYS>;
  using R = Rows<T, D>;
  constexpr int PARTS = 2;                                             // bound by the cache's bytes: both are free
  extern __shared__ __align__(16) char lds[];
  const unsigned unit = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - unit * a.splits;
  const unsigned bg = unit / (unsigned)a.tiles;
  const int tile = (int)(unit - bg * a.tiles), rep = a.H / a.G, b = (int)(bg / (unsigned)a.G), group = (int)(bg - (unsigned)b * a.G);
  Seq s;
  s.b = b, s.first = 0, s.id = b, s.tile = tile;
  s.n = a.lens != nullptr ? min(max(uniform(a.lens[b]), 0), a.T) : a.T;
  const int first = tile * 32 / rep, lastq = min((tile * 32 + 31) / rep, s.n - 1);
  if (first >= s.n) return;
  const int tid = threadIdx.x, l = lane_id(), h = l >> 5, w = uniform(wave_id());
  const int r = tile * 32 + (l & 31), tq = r / rep, head = group * rep + (r - tq * rep);
  const int room = a.max_pages << a.page_shift;
  const int past = min(max(uniform(a.past[b]), 0), room), keys = min(past + s.n, room);
  const int jend = min(past + lastq + 1, keys), jbeg = a.window > 0 ? max(past + first - a.window + 1, 0) : 0;
  int t0 = jbeg / 32, t1 = max((jend + 31) / 32, t0);
  {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + (int)split * per, t1);
    t1 = min(t0 + per, t1);
  }
  const int* table = a.table + (size_t)b * a.max_pages;

  u32x4 qf[R::kSteps];
#pragma unroll
  for (int k = 0; k < R::kSteps; ++k) {
    qf[k] = u32x4{0, 0, 0, 0};
    if (tq < s.n)
      qf[k] = *reinterpret_cast<const u32x4*>((const char*)a.q + (b * a.qs.b + head * a.qs.h + (long long)tq * a.qs.t) * (long long)sizeof(T) +
                                              (2 * k + h) * 16);
  }
  char* const kt = lds + w * F::kWave;
  char* const vt = kt + F::kTile;
  float* const scales = reinterpret_cast<float*>(kt + 2 * F::kTile);
  KeyTile<T, D, 64, 32, KEYS> nk, nv;
  const auto page_of = [&](int t) { return t < t1 && a.page_shift >= 5 ? table[t * 32 >> a.page_shift] : 0; };
  int id = page_of(t0 + w);
  const auto load = [&](int t) {
    nk.load_cache(a, a.cache_k, a.cache_ks, table, uniform(id), group, t * 32, keys, l);
    nv.load_cache(a, a.cache_v, a.cache_vs, table, uniform(id), group, t * 32, keys, l);
    id = page_of(t + 4);
  };
  if (t0 + w < t1) load(t0 + w);

  f32x16 o[1][D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) o[0][d] = zero16();
  float m = -kInf, sum = 0.f;
  const float c = a.scale * kLog2e;
  const int rrow = R::by_rows(l), rcol = R::transposed(l);
  const int i = tq < s.n ? past + tq : -1;                             // this lane's position
  for (int t = t0 + w; t < t1; t += 4) {
    nk.store(kt, scales, l);
    nv.store(vt, scales + 32, l);
    __builtin_amdgcn_wave_barrier();
    if (t + 4 < t1) load(t + 4);
    f32x16 x = zero16();
#pragma unroll
    for (int k = 0; k < R::kSteps; ++k) mma(x, lds16(kt + rrow + k * 32), qf[k], T());
    const int last = min(i, keys - 1) - t * 32 - 4 * h, from = (a.window > 0 ? i - a.window + 1 : 0) - t * 32 - 4 * h;
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
      for (int d = 0; d < D / 32; ++d) o[0][d] *= f;
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
    Operand<T, PARTS> p[1];
    p[0].set(x);
    mul_transposed<D, PARTS, 1>(o, vt + rcol, p);
    __builtin_amdgcn_wave_barrier();
  }

  if (__any(tq < s.n && (!finite(o[0]) || !(fabsf(m * c) <= kFar || m == -kInf)))) {
    careful_rows<T, D, KEYS>(a, qf, nullptr, nullptr, 0, 0, table, group, t0 + w, t1, 4, keys, a.window > 0 ? i - a.window + 1 : 0,
                          tq < s.n ? min(i, keys - 1) : -1, m, sum, o[0]);
  }

  // the waves' shares through LDS
  const float total = both_sum(sum);
  store_columns<float, D>(kt + (l & 31) * F::kOut, o[0], 1.f, h);
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
      __builtin_memcpy((char*)a.o + (b * a.os.b + hd * a.os.h + (long long)t * a.os.t + col) * (long long)sizeof(T), z, sizeof(z));
    }
  }
}

}  // namespace attn
}  // namespace prism
