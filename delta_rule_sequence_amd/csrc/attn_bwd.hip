// attn_bwd.hip - launches of the attention backward (prism_attn_bwd.h)
#include "prism_attn_bwd.h"

namespace prism {
namespace host {
namespace {

#ifndef NQ_
#define NQ_ 4
#define BQ_ 64
#define NK_ 4
#define BK_ 64
#endif

template <class F>
bool room(const void* kernel) { return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, F::kLds) == hipSuccess; }

int row_tiles(const AttnArgs& a, int rows) { return a.starts != nullptr ? a.T / rows + a.S : a.B * ((a.T + rows - 1) / rows); }

template <class T, int D, int NQ, int BQ, int NK, int BK>
prism_status run(const AttnArgs& a, hipStream_t stream) {
  using Q = attn::BwdTile<T, D, NQ, BQ>;
  using K = attn::BwdTile<T, D, NK, BK>;
  static const bool ok = room<Q>(reinterpret_cast<const void*>(attn::dq_kernel<T, D, NQ, BQ>)) &&
                         room<K>(reinterpret_cast<const void*>(attn::dkv_kernel<T, D, NK, BK>));
  if (!ok) return PRISM_ERR_HIP;
  attn::dq_kernel<T, D, NQ, BQ><<<dim3(row_tiles(a, Q::kRows) * a.H), Q::kThreads, Q::kLds, stream>>>(a);
  attn::dkv_kernel<T, D, NK, BK><<<dim3(row_tiles(a, K::kRows) * a.G), K::kThreads, K::kLds, stream>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

}  // namespace

prism_status launch_attn_bwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16)
    return D == 32 ? run<bf16_t, 32, 4, 64, 4, 64>(a, s) : D == 64 ? run<bf16_t, 64, NQ_, BQ_, NK_, BK_>(a, s) : run<bf16_t, 128, NQ_, BQ_, NK_, BK_>(a, s);
  return D == 32 ? run<float, 32, 4, 32, 4, 32>(a, s) : D == 64 ? run<float, 64, 4, 32, 4, 32>(a, s) : run<float, 128, 4, 32, 4, 32>(a, s);
}

}  // namespace host
}  // namespace prism
