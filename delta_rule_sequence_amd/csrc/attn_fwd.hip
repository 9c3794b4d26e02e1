// attn_fwd.hip - launches of the attention forward (prism_attn.h)
#include "prism_attn.h"

namespace prism {
namespace host {
namespace {

template <class K>
bool room(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess;
}
size_t row_tiles(const AttnArgs& a, size_t rows, size_t each) {
  return a.starts != nullptr ? a.T * each / rows + a.S : a.B * ((a.T * each + rows - 1) / rows);
}

template <class T, int D, int NW, int BN>
prism_status many(const AttnArgs& a, hipStream_t stream) {
  using F = attn::FwdTile<T, D, NW, BN, attn::kPrompt>;
  const auto kernel = attn::fwd_kernel<T, D, NW, BN, 1, attn::kPrompt>;
  static const bool ok = room(kernel, F::kLds);
  if (!ok) return PRISM_ERR_HIP;
  kernel<<<dim3((unsigned)(row_tiles(a, F::kRows, 1) * a.H)), F::kThreads, F::kLds, stream>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}
template <class T, int D>
prism_status few(const AttnArgs& a, hipStream_t stream) {
  using F = attn::FewTile<T, D, attn::kPrompt>;
  const auto kernel = attn::few_kernel<T, D, attn::kPrompt>;
  static const bool ok = room(kernel, F::kLds);
  if (!ok) return PRISM_ERR_HIP;
  kernel<<<dim3((unsigned)(row_tiles(a, 32, a.H / a.G) * a.G)), 256, F::kLds, stream>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

#ifndef FORCE
#define FORCE -1
#endif
// Workgroups of 128 rows, or of 256 for wide heads, where there are enough of them for the device; else tiles of 32 rows whose
// keys four waves share.
template <class T, int D>
prism_status run(const AttnArgs& a, hipStream_t s) {
  const size_t blocks = row_tiles(a, 128, 1) * a.H;
  int how = blocks < 256 ? 0 : D == 128 && sizeof(T) == 2 && blocks >= 1024 ? 2 : 1;
  if (FORCE >= 0) how = FORCE;
  if (how == 0) return few<T, D>(a, s);
  if constexpr (D == 128 && sizeof(T) == 2) if (how == 2) return many<T, D, 8, 64>(a, s);
  return many<T, D, 4, (sizeof(T) == 4 && D > 32 ? 32 : 64)>(a, s);
}

}  // namespace

prism_status launch_attn_fwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return D == 32 ? run<bf16_t, 32>(a, s) : D == 64 ? run<bf16_t, 64>(a, s) : run<bf16_t, 128>(a, s);
  return D == 32 ? run<float, 32>(a, s) : D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace host
}  // namespace prism
