// rope.hip - launches of the norm and rotation of queries and keys (prism_rope.h)
#include "prism_rope.h"

namespace prism {
namespace host {
namespace {

template <class T, int V, int L, int NU, bool INTER>
prism_status run(bool bwd, const RopeArgs& a, hipStream_t s) {
  if (bwd) {
    rope::bwd_kernel<T, V, L, NU, INTER><<<dim3(a.nblk), 256, 0, s>>>(a);
    if (a.part != nullptr) rope::sum_kernel<<<dim3((2 * a.D + 31) / 32), 1024, 0, s>>>(a);
  } else {
    const size_t units = (size_t)a.B * a.T * a.groups, per = 256 / L;
    rope::fwd_kernel<T, V, L, NU, INTER><<<dim3((unsigned)((units + per - 1) / per)), 256, 0, s>>>(a);
  }
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

// Lane groups: 4 pairs (8 values) per lane where the row and its rotated part are whole multiples of that, else single
// pairs on a wave.
template <class T, bool INTER>
prism_status by_width(bool bwd, const RopeArgs& a, hipStream_t s) {
  if (a.D % 8 != 0 || a.rot % 8 != 0) return a.D <= 128 ? run<T, 1, 64, 1, INTER>(bwd, a, s) : run<T, 1, 64, 4, INTER>(bwd, a, s);
  return a.D <= 32 ? run<T, 4, 4, 1, INTER>(bwd, a, s) : a.D <= 64 ? run<T, 4, 8, 1, INTER>(bwd, a, s)
       : a.D <= 128 ? run<T, 4, 16, 1, INTER>(bwd, a, s) : a.D <= 256 ? run<T, 4, 32, 1, INTER>(bwd, a, s)
                                                          : run<T, 4, 64, 1, INTER>(bwd, a, s);
}

template <class T>
prism_status by_layout(bool bwd, const RopeArgs& a, hipStream_t s) {
  return a.interleaved ? by_width<T, true>(bwd, a, s) : by_width<T, false>(bwd, a, s);
}

}  // namespace

prism_status launch_rope(prism_dtype dt, bool bwd, const RopeArgs& a, hipStream_t s) {
  return dt == PRISM_BF16 ? by_layout<bf16_t>(bwd, a, s) : by_layout<float>(bwd, a, s);
}

}  // namespace host
}  // namespace prism
