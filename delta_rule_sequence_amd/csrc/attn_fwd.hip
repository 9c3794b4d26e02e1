// attn_fwd.hip - launches of the attention forward (prism_attn.h)
#include "prism_attn.h"

namespace prism {
namespace host {
namespace {

#ifndef NW_
#define NW_ 8
#define BN_ 64
#define PARTS_ 1
#endif

template <class T, int D, int NW, int BN, int PARTS>
prism_status run(AttnArgs a, hipStream_t stream) {
  using F = attn::FwdTile<T, D, NW, BN, attn::kPrompt>;
  const auto kernel = attn::fwd_kernel<T, D, NW, BN, PARTS, attn::kPrompt>;
  a.tiles = a.starts != nullptr ? a.T / F::kRows + a.S : a.B * ((a.T + F::kRows - 1) / F::kRows);
  static const bool ok = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             F::kLds) == hipSuccess;
  if (!ok) return PRISM_ERR_HIP;
  kernel<<<dim3(a.tiles * a.H), F::kThreads, F::kLds, stream>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

}  // namespace

prism_status launch_attn_fwd(prism_dtype dt, int D, AttnArgs a, hipStream_t s) {
  if (dt == PRISM_BF16)
    return D == 32 ? run<bf16_t, 32, 4, 64, 1>(a, s) : D == 64 ? run<bf16_t, 64, NW_, BN_, PARTS_>(a, s) : run<bf16_t, 128, NW_, BN_, PARTS_>(a, s);
  return D == 32 ? run<float, 32, 4, 64, 1>(a, s) : D == 64 ? run<float, 64, 4, 32, 1>(a, s) : run<float, 128, 4, 32, 1>(a, s);
}

}  // namespace host
}  // namespace prism
