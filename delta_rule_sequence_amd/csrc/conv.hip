// conv.hip - launches of the causal convolution (prism_conv.h)
#include "prism_conv.h"

namespace prism {
namespace host {
namespace {

prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }

// V channels per thread.
dim3 strip_grid(const ConvArgs& a, int V) {
  const int cols = (a.D + V - 1) / V;
  return dim3((cols + 63) / 64, (a.nstrip + 3) / 4, a.B * a.H);
}

template <class T, int K, bool SILU>
void fwd_act(const ConvArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (conv_group<V>(a.D) == 1) conv::fwd_kernel<T, K, 1, 8, SILU, false><<<strip_grid(a, 1), 256, 0, s>>>(a);
  else if (a.D % V == 0) conv::fwd_kernel<T, K, V, 8, SILU, false><<<strip_grid(a, V), 256, 0, s>>>(a);
  else conv::fwd_kernel<T, K, V, 8, SILU, true><<<strip_grid(a, V), 256, 0, s>>>(a);
}
template <class T, int K>
prism_status fwd(const ConvArgs& a, hipStream_t s) {
  if (a.silu) fwd_act<T, K, true>(a, s);
  else fwd_act<T, K, false>(a, s);
  return launched();
}

template <class T, int K, bool SILU>
void bwd_act(const ConvArgs& a, hipStream_t s) {
  constexpr int V = 4;
  if (conv_group<V>(a.D) == 1) conv::bwd_kernel<T, K, 1, 4, SILU, false><<<strip_grid(a, 1), 256, 0, s>>>(a);
  else if (a.D % V == 0) conv::bwd_kernel<T, K, V, 4, SILU, false><<<strip_grid(a, V), 256, 0, s>>>(a);
  else conv::bwd_kernel<T, K, V, 4, SILU, true><<<strip_grid(a, V), 256, 0, s>>>(a);
}
template <class T, int K>
prism_status bwd(const ConvArgs& a, hipStream_t s) {
  if (a.silu) bwd_act<T, K, true>(a, s);
  else bwd_act<T, K, false>(a, s);
  conv::wsum_kernel<K><<<dim3((a.D + 31) / 32, K + 1, a.H), 1024, 0, s>>>(a);
  return launched();
}

template <class T, int K>
prism_status step(const ConvArgs& a, hipStream_t s) {
  const size_t n = (size_t)a.B * a.H * a.D;
  conv::step_kernel<T, K><<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(a);
  return launched();
}

}  // namespace

prism_status launch_conv_fwd(prism_dtype dt, int K, const ConvArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return K == 2 ? fwd<bf16_t, 2>(a, s) : K == 3 ? fwd<bf16_t, 3>(a, s) : fwd<bf16_t, 4>(a, s);
  return K == 2 ? fwd<float, 2>(a, s) : K == 3 ? fwd<float, 3>(a, s) : fwd<float, 4>(a, s);
}
prism_status launch_conv_bwd(prism_dtype dt, int K, const ConvArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return K == 2 ? bwd<bf16_t, 2>(a, s) : K == 3 ? bwd<bf16_t, 3>(a, s) : bwd<bf16_t, 4>(a, s);
  return K == 2 ? bwd<float, 2>(a, s) : K == 3 ? bwd<float, 3>(a, s) : bwd<float, 4>(a, s);
}
prism_status launch_conv_step(prism_dtype dt, int K, const ConvArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return K == 2 ? step<bf16_t, 2>(a, s) : K == 3 ? step<bf16_t, 3>(a, s) : step<bf16_t, 4>(a, s);
  return K == 2 ? step<float, 2>(a, s) : K == 3 ? step<float, 3>(a, s) : step<float, 4>(a, s);
}

}  // namespace host
}  // namespace prism
