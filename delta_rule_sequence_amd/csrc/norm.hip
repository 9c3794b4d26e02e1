// norm.hip - launches of the root-mean-square norm (prism_norm.h)
#include "prism_norm.h"

namespace prism {
namespace host {
namespace {

prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }

// n workgroups over x and y (a dimension holds 2^32 threads).
dim3 blocks(size_t n) {
  const size_t x = n < 1 << 20 ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

template <class T, int TPR, int NV>
void fwd_row(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = norm::row_threads(TPR) / TPR;
  norm::fwd_row_kernel<T, TPR, NV><<<blocks(((size_t)a.rows + RPB - 1) / RPB), norm::row_threads(TPR), 0, s>>>(a);
}
template <class T, int TPR, int NV>
void bwd_row(const NormArgs& a, hipStream_t s) {
  if (a.gate != nullptr) norm::bwd_row_kernel<T, TPR, NV, true><<<dim3(a.nblk), norm::row_threads(TPR), 0, s>>>(a);
  else norm::bwd_row_kernel<T, TPR, NV, false><<<dim3(a.nblk), norm::row_threads(TPR), 0, s>>>(a);
}

// Lanes and pieces of a row of n 16-byte pieces: a part of a wave up to 32 pieces, a wave up to 256, 256 lanes up to 1024,
// else 1024.
#define PRISM_NORM_ROWS(F, n)                                                                          \
  ((n) <= 8 ? F<T, 8, 1>(a, s) : (n) <= 16 ? F<T, 16, 1>(a, s) : (n) <= 32 ? F<T, 32, 1>(a, s)         \
   : (n) <= 64 ? F<T, 64, 1>(a, s) : (n) <= 128 ? F<T, 64, 2>(a, s) : (n) <= 192 ? F<T, 64, 3>(a, s)   \
   : (n) <= 256 ? F<T, 64, 4>(a, s) : (n) <= 512 ? F<T, 256, 2>(a, s) : (n) <= 768 ? F<T, 256, 3>(a, s) \
   : (n) <= 1024 ? F<T, 256, 4>(a, s) : F<T, 1024, 2>(a, s))

template <class T>
prism_status fwd(bool rows, const NormArgs& a, hipStream_t s) {
  const int n = (a.D + norm::Piece<T>::V - 1) / norm::Piece<T>::V;
  if (rows) PRISM_NORM_ROWS(fwd_row, n);
  else norm::fwd_long_kernel<T><<<blocks(a.rows), 256, 0, s>>>(a);
  return launched();
}
template <class T>
prism_status bwd(bool rows, const NormArgs& a, hipStream_t s) {
  const int n = (a.D + norm::Piece<T>::V - 1) / norm::Piece<T>::V;
  if (rows) PRISM_NORM_ROWS(bwd_row, n);
  else norm::bwd_long_kernel<T><<<dim3(a.nblk), 256, 0, s>>>(a);
  if (a.dw != nullptr) norm::wsum_kernel<<<dim3((a.D + 31) / 32), 1024, 0, s>>>(a);
  return launched();
}

}  // namespace

prism_status launch_norm_fwd(prism_dtype dt, bool rows, const NormArgs& a, hipStream_t s) {
  return dt == PRISM_BF16 ? fwd<bf16_t>(rows, a, s) : fwd<float>(rows, a, s);
}
prism_status launch_norm_bwd(prism_dtype dt, bool rows, const NormArgs& a, hipStream_t s) {
  return dt == PRISM_BF16 ? bwd<bf16_t>(rows, a, s) : bwd<float>(rows, a, s);
}

}  // namespace host
}  // namespace prism
