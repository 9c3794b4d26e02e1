// prism_attn_args.h - arguments of the attention layer's kernels (prism_attn.h, prism_attn_bwd.h, prism_paged.h,
// prism_rope.h) and their launch functions.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>

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
  void* o;
  float* lse;                     // [B][H][T]; may be null in the forward
  // backward
  const void* dout;
  prism_strides dos, dqs, dks, dvs;
  float* delta;                   // [B][H][T]: <do, o> of each row
  void *dq, *dk, *dv;
  // paged cache: [pages][G][page][D], of q's type or e4m3 with a scale per row
  void *cache_k, *cache_v;
  float *cache_ks, *cache_vs;     // [pages][G][page]
  const int *table, *past;        // [S][max_pages], [S]
  int pages, page_shift, max_pages;
  int splits;                     // key ranges of a sequence, joined afterwards
  float* part;                    // their shares of o, and m, l behind them
};

// Norm and rotation of the rows of two tensors: x[0] with H heads, x[1] with G.
struct RopeArgs {
  const void *x[2], *dy[2];
  void* y[2];                     // forward: y, backward: dx
  prism_strides xs[2], dys[2], ys[2];
  const float *w[2], *freq;
  float* dw[2];
  const int* pos;                 // [B][T]; null: the token's index
  int B, T, D, heads[2], rot, interleaved;
  float factor, eps;
  int per, groups;                // heads per lane group, groups of a token
  float* part;                    // [nblk][2][D]
  int nblk;
};

namespace host {
// A launch holds less than 2^32 threads.
constexpr size_t kMostThreads = ((size_t)1 << 32) - 1;

// A launch with `lds` bytes of dynamic LDS, which may be more than a kernel has by default: each device is told once.
template <auto KERNEL>
prism_status launch_wide(unsigned blocks, unsigned threads, int lds, const AttnArgs& a, hipStream_t stream) {
  static std::atomic<unsigned long long> told{0};                     // the devices, by bits
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return PRISM_ERR_HIP;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if ((told.load(std::memory_order_relaxed) & bit) == 0) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
      return PRISM_ERR_HIP;
    told.fetch_or(bit, std::memory_order_relaxed);
  }
  KERNEL<<<dim3(blocks), dim3(threads), lds, stream>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

// Each enqueues on `stream` and reports launch failures.
prism_status launch_cache_write(prism_dtype dt, int D, bool bits8, const AttnArgs& a, hipStream_t stream);
prism_status launch_attn_paged(prism_dtype dt, int D, bool bits8, int rows, const AttnArgs& a, hipStream_t stream);
prism_status launch_rope(prism_dtype dt, bool bwd, const RopeArgs& a, hipStream_t stream);
prism_status launch_attn_fwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t stream);
prism_status launch_attn_bwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t stream);
}  // namespace host
}  // namespace prism
