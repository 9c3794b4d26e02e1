// prism_paged.h - the paged cache of keys and values (gfx950): rows are written to it (prism_attn.h reads it).
//
// Position p of a sequence lies in page table[p / page], row p % page of its group.  With 8 bits a row x is held as e4m3
// bytes of x / scale, scale = max |x| / 448.
#pragma once
#include "prism_attn.h"
#include "prism_e4m3.h"

namespace prism {
namespace attn {

// ---- write ----------------------------------------------------------------------------------------------
// A workgroup takes kWriteTokens tokens of a sequence, all groups, keys and values; a row lies in D / 8 or D / 4 lanes, and 8 rows are
// in flight.  With 8 bits bound by instructions (1100 vector instructions per wave, addresses and the divisions by the group count
// among them: 7 us of issue) and the latency of the row maximum's exchange: 16 us where a copy of the bytes of 8 x 2048 tokens of
// 4 groups of 128 takes 7.4; a token's step is a launch (3.4 us).
constexpr int kWriteTokens = 16;

template <class T, int D, bool BITS8>
__global__ __launch_bounds__(256) void cache_write_kernel(AttnArgs a, unsigned first_tile) {
  const int G = a.G;
  constexpr int V = 16 / (int)sizeof(T), L = D / V;
  typedef T vec __attribute__((ext_vector_type(V)));
  a.G = 1;                                                            // tiles of all groups at once
  const Seq s = find_tile(a, first_tile + blockIdx.x, kWriteTokens, 1, false);
  if (s.id < 0) return;
  const int t0 = s.tile * kWriteTokens, n = min(kWriteTokens, s.n - t0), at = threadIdx.x % L;
  const long long past = max(a.past[s.id], 0);
  const int* table = a.table + (size_t)s.id * a.max_pages;
  const int page = 1 << a.page_shift;
  constexpr int U = 8;                                                 // rows in flight
  for (int first = threadIdx.x / L; first < n * 2 * G; first += U * (256 / L)) {
    vec x[U];
    long long row[U];                                                  // -1: not written
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = first + u * (256 / L), g = r % G, tk = r / G, t = t0 + (tk >> 1);
      const bool key = (tk & 1) == 0;
      const long long p = past + t;
      row[u] = -1;
      if (r >= n * 2 * G || p >> a.page_shift >= a.max_pages) continue;
      const int id = table[p >> a.page_shift];
      const prism_strides st = key ? a.ks : a.vs;
      x[u] = *reinterpret_cast<const vec*>((const T*)(key ? a.k : a.v) + (s.b * st.b + g * st.h + (long long)(s.first + t) * st.t) + at * V);
      if ((unsigned)id < (unsigned)a.pages) row[u] = ((long long)id * G + g) * page + (p & (page - 1));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool key = ((first + u * (256 / L)) / G & 1) == 0;
      if (row[u] < 0) continue;                                        // all lanes of a row alike
      void* const cache = key ? a.cache_k : a.cache_v;
      if constexpr (!BITS8) {
        *reinterpret_cast<vec*>((T*)cache + row[u] * D + at * V) = x[u];
      } else {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, norm::abs_bits((float)x[u][i]));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) m = max(m, (unsigned)__shfl_xor((int)m, o, 64));
        float f;
        const float scale = norm::block_scale(m, &f);
        unsigned y[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const int w = __builtin_amdgcn_cvt_pk_fp8_f32((float)x[u][4 * i] * f, (float)x[u][4 * i + 1] * f, 0, false);
          y[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32((float)x[u][4 * i + 2] * f, (float)x[u][4 * i + 3] * f, w, true);
        }
        __builtin_memcpy((char*)cache + row[u] * D + at * V, y, sizeof(y));
        if (at == 0) (key ? a.cache_ks : a.cache_vs)[row[u]] = scale;
      }
    }
  }
}

}  // namespace attn
}  // namespace prism
