// norm.hip - launches of the root-mean-square norm (prism_norm.h)
#include "prism_norm.h"

namespace prism {
namespace host {
namespace {

prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }

template <class T>
prism_status bwd(const NormArgs& a, hipStream_t s) {
  norm::bwd_kernel<T><<<dim3(a.nblk), 256, 0, s>>>(a);
  if (a.dw != nullptr) norm::wsum_kernel<<<dim3((a.D + 63) / 64), 256, 0, s>>>(a);
  return launched();
}

}  // namespace

prism_status launch_norm_fwd(prism_dtype dt, bool, const NormArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) norm::fwd_kernel<bf16_t><<<dim3(a.rows), 256, 0, s>>>(a);
  else norm::fwd_kernel<float><<<dim3(a.rows), 256, 0, s>>>(a);
  return launched();
}
prism_status launch_norm_bwd(prism_dtype dt, bool, const NormArgs& a, hipStream_t s) {
  return dt == PRISM_BF16 ? bwd<bf16_t>(a, s) : bwd<float>(a, s);
}

}  // namespace host
}  // namespace prism
