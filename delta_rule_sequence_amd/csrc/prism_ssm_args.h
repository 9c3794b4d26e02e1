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

// Channels per thread of the convolution: V, or 1 where V would leave more than half of a wave without any.  One strip per
// wave.  16 x 768000 / D x D, V against 1, us: forward bf16 (V 8) 45 and 14 at 64 channels, 20 and 16 at 160, 14.6 and 13.7 at 256,
// 13.5 and 13.6 at 320, 13.2 and 15.7 at 400; f32 (V 4) 27 and 17 at 64, 18 and 17 at 128, 17 and 19 at 160, 19 and 21 at 400;
// backward (V 4) bf16 55 and 31, 33 and 28, 30 and 31, 25 and 31; f32 62 and 40, 42 and 38, 41 and 41, 40 and 42.
template <int V> inline int conv_group(int D) { return D > 32 * V ? V : 1; }

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
