// prism_ssm_args.h - arguments of the state space layer's kernels (prism_ssm.h, prism_conv.h, prism_norm.h)
// and their launch functions.
#pragma once
#include <hip/hip_runtime.h>

#include "prism.h"

namespace prism {

// The scan.  A head's P columns are cut into nsl slices of PW columns ("virtual heads"): slices
// share decays and Bm / Cm and are otherwise independent.  hv = h * nsl + slice.
struct SsmArgs {
  const void *x, *bm, *cm, *dy;
  prism_strides xs, bs, cs, ts, dys;  // element strides (batch, head / group, token)
  const float *dt, *dt_bias, *A, *D;
  const int* lens;
  int B, H, G, T, P, softplus;
  int nsl;                        // slices per head
  int nch, seg_chunks, nseg;      // 64-token chunks, chunks per segment, segments
  int fold;                       // entering states are formed by their readers (few segments), not by a scan of their own
  const float* S0;
  void* y;
  prism_strides ys;
  float* S_final;
  float* seg;                     // [dirs][B * HV][nseg][N * PW]: states at segment borders
  float* seg_dec;                 // [dirs][B * HV][nseg]: decay over each segment
  // backward
  float* st;                      // [2][B * HV][nch][N * PW]: state entering / adjoint leaving each chunk
  const float* dS;
  void *dx, *dbm, *dcm;
  prism_strides dxs, dbs, dcs;
  float *ddt, *dA, *dD, *ddt_bias;
  int nsplit, per_split;          // splits of a group's virtual heads in the gradient pass
  float *part_b, *part_c;         // [nsplit][B][G][T][N] (nsplit > 1)
  float* part_ddt;                // [nsl][B][H][T] (nsl > 1)
  float* part_sum;                // [3][B * HV][nch]: shares of dA, dD, ddt_bias
};

struct SsmStepArgs {
  const void *x, *bm, *cm;
  prism_strides xs, bs, cs, ts;
  const float *dt, *dt_bias, *A, *D;
  int H, G, softplus;
  float* S;
  void* y;
};

// Channels per thread of the convolution: V, or 1 where V would leave more than three quarters of a wave without any.
// One strip per wave; at 16 x 12000 x 64, V against 1: 44 and 13 us (bf16, V 8), 23 and 17 (f32, V 4), backward 60 and
// 30, 56 and 33; at 16 x 4800 x 160: 21 and 21, 17 and 20, 31 and 32, 39 and 36; at 400 channels V leads by a tenth or
// more.
template <int V> inline int conv_group(int D) { return D > 16 * V ? V : 1; }

struct ConvArgs {
  const void *x, *dy;
  prism_strides xs, ys, dys;
  const float *w, *bias;
  const void* conv_in;
  const int* lens;
  int B, H, T, D, silu;
  void* y;                        // forward: y, backward: dx
  void* conv_out;
  int strip, nstrip;              // tokens per thread, strips of a sequence
  float* part;                    // backward: [B * ceil(nstrip / 4)][H][K + 1][D]
  float *dw, *dbias;
};

struct NormArgs {
  const void *x, *residual, *gate, *dy, *dh_in;
  long long xs, gs;
  const float* w;
  int rows, D;
  float eps;
  void* y;
  float* scales;
  void* h;                        // forward: h_out, backward: dh
  void* dgate;
  float* part;                    // backward: [nblk][D] shares of dweight
  int nblk;
  float* dw;
};

namespace host {
// Each enqueues on `stream` and reports launch failures.  rows: the norm's rows fit a workgroup's registers.
prism_status launch_ssm_fwd(prism_dtype ty, int N, int PW, const SsmArgs& a, hipStream_t stream);
prism_status launch_ssm_bwd(prism_dtype ty, int N, int PW, const SsmArgs& a, hipStream_t stream);
prism_status launch_ssm_step(prism_dtype ty, int N, int P, int B, const SsmStepArgs& a, hipStream_t stream);
prism_status launch_conv_fwd(prism_dtype dt, int K, const ConvArgs& a, hipStream_t stream);
prism_status launch_conv_bwd(prism_dtype dt, int K, const ConvArgs& a, hipStream_t stream);
prism_status launch_conv_step(prism_dtype dt, int K, const ConvArgs& a, hipStream_t stream);
prism_status launch_norm_fwd(prism_dtype dt, bool rows, const NormArgs& a, hipStream_t stream);
prism_status launch_norm_bwd(prism_dtype dt, bool rows, const NormArgs& a, hipStream_t stream);
}  // namespace host
}  // namespace prism
