// attn_paged.hip - launches of the paged cache's write and of the attention over it (prism_paged.h, prism_attn.h)
#include <algorithm>

#include "prism_paged.h"

namespace prism {
namespace host {
namespace {

prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }
int row_tiles(const AttnArgs& a, int rows) { return a.starts != nullptr ? a.T / rows + a.S : a.B * ((a.T + rows - 1) / rows); }

template <class T, int D, bool BITS8>
prism_status write(const AttnArgs& a, hipStream_t s) {
  // at most 2^24 tiles, 2^23 of them to a launch
  const unsigned tiles = row_tiles(a, attn::kWriteTokens), most = 1u << 23;
  for (unsigned first = 0; first < tiles; first += most) {
    attn::cache_write_kernel<T, D, BITS8><<<dim3(std::min(tiles - first, most)), 256, 0, s>>>(a, first);
    if (launched() != PRISM_OK) return PRISM_ERR_HIP;
  }
  return PRISM_OK;
}

template <class T, int D, attn::Keys KEYS>
prism_status few(const AttnArgs& a, hipStream_t s) {
  using F = attn::FewTile<T, D, KEYS>;
  return launch_wide<attn::few_kernel<T, D, KEYS>>((unsigned)(a.B * a.G * ((a.T * (a.H / a.G) + 31) / 32) * a.splits), 256, F::kLds, a, s);
}
template <class T, int D, attn::Keys KEYS, int NW>
prism_status many(const AttnArgs& a, hipStream_t s) {
  constexpr int BN = sizeof(T) == 2 || D == 32 ? 64 : 32;
  using F = attn::FwdTile<T, D, NW, BN, KEYS>;
  return launch_wide<attn::fwd_kernel<T, D, NW, BN, KEYS>>((unsigned)(row_tiles(a, F::kRows) * a.H * a.splits), F::kThreads, F::kLds, a, s);
}
template <class T, int D, attn::Keys KEYS>
prism_status paged(int rows, const AttnArgs& a, hipStream_t s) {
  prism_status st;
  if (rows == 32) {
    st = few<T, D, KEYS>(a, s);
  } else {
    if constexpr (D == 128 && sizeof(T) == 2) st = rows == 256 ? many<T, D, KEYS, 8>(a, s) : many<T, D, KEYS, 4>(a, s);
    else st = many<T, D, KEYS, 4>(a, s);
  }
  if (st != PRISM_OK || a.splits == 1) return st;
  attn::join_kernel<T, D><<<dim3((unsigned)(((size_t)a.B * a.H * a.T + 3) / 4)), 256, 0, s>>>(a);
  return launched();
}

}  // namespace

prism_status launch_cache_write(prism_dtype dt, int D, bool bits8, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_F32) return D == 32 ? write<float, 32, false>(a, s) : D == 64 ? write<float, 64, false>(a, s) : write<float, 128, false>(a, s);
  if (bits8) return D == 32 ? write<bf16_t, 32, true>(a, s) : D == 64 ? write<bf16_t, 64, true>(a, s) : write<bf16_t, 128, true>(a, s);
  return D == 32 ? write<bf16_t, 32, false>(a, s) : D == 64 ? write<bf16_t, 64, false>(a, s) : write<bf16_t, 128, false>(a, s);
}

prism_status launch_attn_paged(prism_dtype dt, int D, bool bits8, int rows, const AttnArgs& a, hipStream_t s) {
  using namespace attn;
  if (dt == PRISM_F32)
    return D == 32 ? paged<float, 32, kCache>(rows, a, s) : D == 64 ? paged<float, 64, kCache>(rows, a, s) : paged<float, 128, kCache>(rows, a, s);
  if (bits8)
    return D == 32 ? paged<bf16_t, 32, kCache8>(rows, a, s) : D == 64 ? paged<bf16_t, 64, kCache8>(rows, a, s) : paged<bf16_t, 128, kCache8>(rows, a, s);
  return D == 32 ? paged<bf16_t, 32, kCache>(rows, a, s) : D == 64 ? paged<bf16_t, 64, kCache>(rows, a, s) : paged<bf16_t, 128, kCache>(rows, a, s);
}

}  // namespace host
}  // namespace prism
