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

}  // namespace attn
}  // namespace prism
