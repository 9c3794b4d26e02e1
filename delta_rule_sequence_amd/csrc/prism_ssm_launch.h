// prism_ssm_launch.h - launches of the state space scan for one tensor type and state width N (one
// translation unit each, ssm_<type>_n<N>.hip).
#pragma once
#include "prism_ssm_bf16.h"

namespace prism {
namespace host {

inline prism_status launched() { return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP; }

// The scan over the segments, 16 of them per thread.
template <int N, int PW, bool TRANS>
void seg_scan(const SsmArgs& a, int dirs, hipStream_t stream) {
  int groups = 1;
  while (groups * 16 < a.nseg) groups *= 2;
  ssm::seg_scan_kernel<N, PW, TRANS><<<dim3(N * PW / 256 * groups, a.B * a.H * a.nsl, dirs), 256, 0, stream>>>(a, groups);
}

// HP: virtual heads of a group per workgroup (two where their number is even: they share the rows of B and C).
// PTW: column tiles per wave.
template <int N, int PW, int PTW, int HP>
void ssm_fwd_mx(const SsmArgs& a, hipStream_t stream) {
  const int bh = a.B * a.H * a.nsl, nth = ssm::mx::waves_per_head<PW, PTW>() * HP * 64;
  if (a.nseg > 1) {
    ssm::mx::state_kernel<N, PW, PTW, HP, false, false><<<dim3(bh / HP * (a.nseg - 1), 1), nth, 0, stream>>>(a);
    if (!a.fold) seg_scan<N, PW, false>(a, 1, stream);
  }
  ssm::mx::sweep_kernel<N, PW, PTW, HP><<<dim3(bh / HP * a.nseg), nth, 0, stream>>>(a);
}
template <int N, int PW, int PTW, int HP>
void ssm_bwd_states_mx(const SsmArgs& a, hipStream_t stream) {
  const int bh = a.B * a.H * a.nsl, nth = ssm::mx::waves_per_head<PW, PTW>() * HP * 64;
  if (a.nseg > 1) {
    ssm::mx::state_kernel<N, PW, PTW, HP, true, false><<<dim3(bh / HP * (a.nseg - 1), 2), nth, 0, stream>>>(a);
    if (!a.fold) seg_scan<N, PW, true>(a, 2, stream);
  }
  ssm::mx::state_kernel<N, PW, PTW, HP, true, true><<<dim3(bh / HP * a.nseg, 2), nth, 0, stream>>>(a);
}

template <class T, int N, int PW>
prism_status ssm_fwd_pw(const SsmArgs& a, hipStream_t stream) {
  const int bh = a.B * a.H * a.nsl;
  if constexpr (std::is_same<T, bf16_t>::value) {
    constexpr int PTW = PW >= 32 ? 2 : 1;
    if (a.H / a.G * a.nsl % 2 == 0) ssm_fwd_mx<N, PW, PTW, 2>(a, stream);
    else ssm_fwd_mx<N, PW, PTW, 1>(a, stream);
  } else {
    if (a.nseg > 1) {
      ssm::state_kernel<N, PW, false><<<dim3(a.nseg, bh, 1), PW * 4, 0, stream>>>(a);
      seg_scan<N, PW, true>(a, 1, stream);
    }
    ssm::sweep_kernel<N, PW><<<dim3(a.nseg, bh), PW * 4, 0, stream>>>(a);
  }
  return launched();
}

template <class T, int N, int PW>
prism_status ssm_bwd_pw(const SsmArgs& a, hipStream_t stream) {
  const int bh = a.B * a.H * a.nsl;
  if constexpr (std::is_same<T, bf16_t>::value) {
    constexpr int PTW = PW >= 32 ? 2 : 1;
    if (a.H / a.G * a.nsl % 2 == 0) ssm_bwd_states_mx<N, PW, PTW, 2>(a, stream);
    else ssm_bwd_states_mx<N, PW, PTW, 1>(a, stream);
    ssm::mx::grad_kernel<N, PW><<<dim3(a.nch, a.nsplit, a.B * a.G), 512, 0, stream>>>(a);
  } else {
    if (a.nseg > 1) ssm::state_kernel<N, PW, false><<<dim3(a.nseg, bh, 2), PW * 4, 0, stream>>>(a);
    seg_scan<N, PW, true>(a, 2, stream);
    ssm::state_kernel<N, PW, true><<<dim3(a.nseg, bh, 2), PW * 4, 0, stream>>>(a);
    ssm::grad_kernel<N, PW><<<dim3(a.nch, a.nsplit, a.B * a.G), 256, 0, stream>>>(a);
  }
  const auto blocks = [](size_t n) { return (unsigned)((n + 255) / 256); };
  const unsigned n_ddt = a.nsl > 1 ? blocks((size_t)a.B * a.H * a.T) : 0;
  const unsigned n_split = a.nsplit > 1 ? blocks((size_t)a.B * a.G * a.T * (N / 4)) : 0;
  ssm::finish_kernel<T, N><<<dim3(3 * a.H + n_ddt + n_split), 256, 0, stream>>>(a, n_ddt);
  return launched();
}

template <class T, int N, int P>
prism_status ssm_step_p(int B, const SsmStepArgs& a, hipStream_t stream) {
  ssm::step_kernel<T, N, P><<<dim3((unsigned)((size_t)B * a.H)), 256, 0, stream>>>(a);
  return launched();
}

// The entry points of one (type, N): PW in {16, 32, 64}, P in {16, 32, 64, 128}.
#define PRISM_SSM_UNIT(NAME, T, N)                                                                  \
  prism_status NAME##_fwd(int pw, const SsmArgs& a, hipStream_t s) {                                \
    return pw == 16 ? ssm_fwd_pw<T, N, 16>(a, s) : pw == 32 ? ssm_fwd_pw<T, N, 32>(a, s)            \
                                                            : ssm_fwd_pw<T, N, 64>(a, s);           \
  }                                                                                                 \
  prism_status NAME##_bwd(int pw, const SsmArgs& a, hipStream_t s) {                                \
    return pw == 16 ? ssm_bwd_pw<T, N, 16>(a, s) : pw == 32 ? ssm_bwd_pw<T, N, 32>(a, s)            \
                                                            : ssm_bwd_pw<T, N, 64>(a, s);           \
  }                                                                                                 \
  prism_status NAME##_step(int p, int B, const SsmStepArgs& a, hipStream_t s) {                     \
    return p == 16 ? ssm_step_p<T, N, 16>(B, a, s) : p == 32 ? ssm_step_p<T, N, 32>(B, a, s)        \
         : p == 64 ? ssm_step_p<T, N, 64>(B, a, s) : ssm_step_p<T, N, 128>(B, a, s);                \
  }

}  // namespace host
}  // namespace prism
