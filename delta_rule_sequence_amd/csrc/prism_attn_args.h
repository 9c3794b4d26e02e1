// prism_attn_args.h - arguments of the attention layer's kernels (prism_attn.h, prism_attn_bwd.h, prism_paged.h,
// prism_rope.h) and their launch functions.
#pragma once
#include <hip/hip_runtime.h>

#include "prism.h"

namespace prism {

// Sequences: the B batches of T tokens, of lens[b] tokens each where lens is given; or, with starts, S stretches
// starts[s] .. starts[s + 1] - 1 of one batch's tokens.
struct AttnArgs {
  const void *q, *k, *v;
  prism_strides qs, ks, vs, os;   // element strides (batch, head / group, token)
  const int *lens, *starts;
  int B, H, G, T, S;
  int causal, window;             // window 0: none
  float scale;
  int tiles;                      // row tiles of all sequences, at most
  void* o;
  float* lse;                     // [B][H][T]; may be null in the forward
  // backward
  const void* dout;
  prism_strides dos, dqs, dks, dvs;
  float* delta;                   // [B][H][T]: <do, o> of each row
  void *dq, *dk, *dv;
  // paged cache: k, v are [pages][G][page][D], of q's type or e4m3 with a scale per row
  const float *k_scale, *v_scale; // [pages][G][page]
  const int *table, *past;        // [B][max_pages], [B]
  int pages, page_shift, max_pages;
  int splits;                     // key ranges of a sequence, joined afterwards
  float* part;                    // their shares of o, and m, l behind them
};

namespace host {
// Each enqueues on `stream` and reports launch failures.
prism_status launch_attn_fwd(prism_dtype dt, int D, AttnArgs a, hipStream_t stream);
prism_status launch_attn_bwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t stream);
}  // namespace host
}  // namespace prism
