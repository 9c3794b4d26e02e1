// attn_bwd.hip - launches of the attention backward (prism_attn_bwd.h)
#include "prism_attn_bwd.h"

namespace prism {
namespace host {
namespace {

#ifndef NQ_
#define NQ_ 8
#define BQ_ 64
#define KW_ 4
#define QW_ 1
#define BK_ 64
#endif
#ifndef AK_
#define AK_ false
#endif
#ifndef N6_
#define N6_ 4
#define K6_ 4
#define Q6_ 2
#define B6_ 128
#endif
#ifndef ONE_
#define ONE_ 3
#endif

template <class F>
bool room(const void* kernel) { return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, F::kLds) == hipSuccess; }

int row_tiles(const AttnArgs& a, int rows) { return a.starts != nullptr ? a.T / rows + a.S : a.B * ((a.T + rows - 1) / rows); }

// PASS: parts of a pass by keys, dk and dv at once (3) or one after the other.
template <class T, int D, int NQ, int BQ, int KW, int QW, int BK, int PASS, bool AQ, bool AK>
prism_status run(const AttnArgs& a, hipStream_t stream) {
  using Q = attn::BwdTile<T, D, NQ, BQ, AQ>;
  using K = attn::KeyPass<T, D, KW, QW, BK, AK>;
  constexpr int FIRST = PASS == 3 ? 3 : attn::kDk;
  static const bool ok = room<Q>(reinterpret_cast<const void*>(attn::dq_kernel<T, D, NQ, BQ, AQ>)) &&
                         room<K>(reinterpret_cast<const void*>(attn::dkv_kernel<T, D, KW, QW, BK, FIRST, AK>)) &&
                         (PASS == 3 || room<K>(reinterpret_cast<const void*>(attn::dkv_kernel<T, D, KW, QW, BK, attn::kDv, AK>)));
  if (!ok) return PRISM_ERR_HIP;
  attn::dq_kernel<T, D, NQ, BQ, AQ><<<dim3(row_tiles(a, Q::kRows) * a.H), Q::kThreads, Q::kLds, stream>>>(a);
  const dim3 grid(row_tiles(a, K::kKeys) * a.G * a.splits);
  attn::dkv_kernel<T, D, KW, QW, BK, FIRST, AK><<<grid, K::kThreads, K::kLds, stream>>>(a);
  if constexpr (PASS != 3) attn::dkv_kernel<T, D, KW, QW, BK, attn::kDv, AK><<<grid, K::kThreads, K::kLds, stream>>>(a);
  if (a.splits > 1) {
    const size_t rows = 2 * (size_t)a.B * a.G * a.T, per = 256 / (D / 4);
    attn::sum_kernel<T, D><<<dim3((unsigned)((rows + per - 1) / per)), 256, 0, stream>>>(a);
  }
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

}  // namespace

prism_status launch_attn_bwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16)
    return D == 32 ? run<bf16_t, 32, 4, 64, 4, 1, 64, 3, true, true>(a, s) : D == 64 ? run<bf16_t, 64, N6_, 64, K6_, Q6_, B6_, 3, true, true>(a, s) : run<bf16_t, 128, NQ_, BQ_, KW_, QW_, BK_, ONE_, true, AK_>(a, s);
  return D == 32 ? run<float, 32, 4, 32, 2, 2, 64, 3, false, false>(a, s) : D == 64 ? run<float, 64, 4, 32, 2, 2, 64, 3, false, false>(a, s) : run<float, 128, 4, 32, 2, 2, 64, 3, false, false>(a, s);
}

}  // namespace host
}  // namespace prism
