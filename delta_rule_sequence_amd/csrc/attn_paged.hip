// attn_paged.hip - launches of the paged cache's write and of the attention over it (prism_paged.h, prism_attn.h)
#include "prism_paged.h"

namespace prism {
namespace host {
namespace {

prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }
int row_tiles(const AttnArgs& a, int rows) { return a.starts != nullptr ? a.T / rows + a.S : a.B * ((a.T + rows - 1) / rows); }

template <class T, int D, bool BITS8>
prism_status write(const AttnArgs& a, hipStream_t s) {
  attn::cache_write_kernel<T, D, BITS8><<<dim3(row_tiles(a, attn::kWriteTokens)), 256, 0, s>>>(a);
  return launched();
}

template <class T, int D, attn::Keys KEYS>
prism_status paged(bool few, const AttnArgs& a, hipStream_t s) {
  using W = attn::FewTile<T, D, KEYS>;
  constexpr int BN = sizeof(T) == 2 || D == 32 ? 64 : 32;
#ifndef MW
#define MW 4
#endif
  constexpr int NW = D == 128 && sizeof(T) == 2 ? MW : 4;
  using M = attn::FwdTile<T, D, NW, BN, KEYS>;
  const auto few_rows = attn::few_kernel<T, D, KEYS>;
  const auto many_rows = attn::fwd_kernel<T, D, NW, BN, 1, KEYS>;
  static const bool ok =
      hipFuncSetAttribute(reinterpret_cast<const void*>(few_rows), hipFuncAttributeMaxDynamicSharedMemorySize, W::kLds) == hipSuccess &&
      hipFuncSetAttribute(reinterpret_cast<const void*>(many_rows), hipFuncAttributeMaxDynamicSharedMemorySize, M::kLds) == hipSuccess;
  if (!ok) return PRISM_ERR_HIP;
  if (few) few_rows<<<dim3(a.B * a.G * ((a.T * (a.H / a.G) + 31) / 32) * a.splits), 256, W::kLds, s>>>(a);
  else many_rows<<<dim3(row_tiles(a, M::kRows) * a.H * a.splits), M::kThreads, M::kLds, s>>>(a);
  if (a.splits > 1) {
    const size_t rows = (size_t)a.B * a.H * a.T;
    attn::join_kernel<T, D><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a);
  }
  return launched();
}

}  // namespace

prism_status launch_cache_write(prism_dtype dt, int D, bool bits8, AttnArgs a, hipStream_t s) {
  if (dt == PRISM_F32) return D == 32 ? write<float, 32, false>(a, s) : D == 64 ? write<float, 64, false>(a, s) : write<float, 128, false>(a, s);
  if (bits8) return D == 32 ? write<bf16_t, 32, true>(a, s) : D == 64 ? write<bf16_t, 64, true>(a, s) : write<bf16_t, 128, true>(a, s);
  return D == 32 ? write<bf16_t, 32, false>(a, s) : D == 64 ? write<bf16_t, 64, false>(a, s) : write<bf16_t, 128, false>(a, s);
}

prism_status launch_attn_paged(prism_dtype dt, int D, bool bits8, bool few, AttnArgs a, hipStream_t s) {
  using namespace attn;
  if (dt == PRISM_F32)
    return D == 32 ? paged<float, 32, kCache>(few, a, s) : D == 64 ? paged<float, 64, kCache>(few, a, s) : paged<float, 128, kCache>(few, a, s);
  if (bits8)
    return D == 32 ? paged<bf16_t, 32, kCache8>(few, a, s) : D == 64 ? paged<bf16_t, 64, kCache8>(few, a, s) : paged<bf16_t, 128, kCache8>(few, a, s);
  return D == 32 ? paged<bf16_t, 32, kCache>(few, a, s) : D == 64 ? paged<bf16_t, 64, kCache>(few, a, s) : paged<bf16_t, 128, kCache>(few, a, s);
}

}  // namespace host
}  // namespace prism
