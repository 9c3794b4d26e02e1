// attn_api.hip - C ABI of the attention layer (include/prism.h): argument checks, plans and workspace layout.
// Host side only; every check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "prism.h"
#include "prism_attn_args.h"
#include "prism_checks.h"

namespace {

using namespace prism;
using namespace prism::checks;

bool attn_width(int D) { return D == 32 || D == 64 || D == 128; }

// What the forward and the backward share.  Row tiles hold at least 32 rows, so the launches' counts stay below
// 2^32 threads with fewer than 2^23 tiles of all heads.
prism_status attn_check(int B, int H, int G, int T, int D, int S, const int* lens, const int* starts, float scale, int window,
                        prism_dtype dt) {
  if (B <= 0 || H <= 0 || G <= 0 || T <= 0 || D <= 0 || !known(dt) || H % G != 0) return PRISM_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0) return PRISM_ERR_INVALID_ARG;
  if (starts != nullptr ? (S <= 0 || B != 1 || lens != nullptr) : S != 0) return PRISM_ERR_INVALID_ARG;
  if (!attn_width(D) || T > INT_MAX - 4096) return PRISM_ERR_UNSUPPORTED;
  const size_t tiles = starts != nullptr ? (size_t)T / 32 + S : (size_t)B * (((size_t)T + 31) / 32);
  return tiles > ((size_t)1 << 23) / H ? PRISM_ERR_UNSUPPORTED : PRISM_OK;
}

}  // namespace

extern "C" {

prism_status prism_attn_fwd(const void* q, const prism_strides* q_strides, const void* k, const prism_strides* k_strides,
                            const void* v, const prism_strides* v_strides, const int* lens, const int* starts, int S,
                            int B, int H, int G, int T, int D, float scale, int causal, int window, prism_dtype dt,
                            void* o, const prism_strides* o_strides, float* lse, hipStream_t stream) {
  const prism_status st = attn_check(B, H, G, T, D, S, lens, starts, scale, window, dt);
  if (st != PRISM_OK) return st;
  if (!q || !k || !v || !o) return PRISM_ERR_INVALID_ARG;
  if (window > 0 && !causal) return PRISM_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (!make_strides(q_strides, B, H, T, D, &a.qs) || !make_strides(k_strides, B, G, T, D, &a.ks) ||
      !make_strides(v_strides, B, G, T, D, &a.vs) || !make_strides(o_strides, B, H, T, D, &a.os) || !rows_apart(a.os, B, H, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(q, a.qs, D, dt) || !scan_rows(k, a.ks, D, dt) || !scan_rows(v, a.vs, D, dt) || !scan_rows(o, a.os, D, dt))
    return PRISM_ERR_UNSUPPORTED;
  a.q = q, a.k = k, a.v = v, a.lens = lens, a.starts = starts;
  a.B = B, a.H = H, a.G = G, a.T = T, a.S = S, a.causal = causal != 0, a.window = window, a.scale = scale;
  a.o = o, a.lse = lse;
  return host::launch_attn_fwd(dt, D, a, stream);
}

size_t prism_attn_bwd_workspace_bytes(int B, int H, int G, int T, int D, prism_dtype dt) {
  if (attn_check(B, H, G, T, D, 0, nullptr, nullptr, 1.f, 0, dt) != PRISM_OK) return 0;
  Layout ly;
  ly.add((size_t)B * H, (size_t)T * 4);
  return ly.ok() ? ly.total : 0;
}

prism_status prism_attn_bwd(const void* q, const prism_strides* q_strides, const void* k, const prism_strides* k_strides,
                            const void* v, const prism_strides* v_strides, const void* o, const prism_strides* o_strides,
                            const float* lse, const void* d_o, const prism_strides* do_strides,
                            const int* lens, const int* starts, int S, int B, int H, int G, int T, int D, float scale,
                            int causal, int window, prism_dtype dt, void* dq, const prism_strides* dq_strides,
                            void* dk, const prism_strides* dk_strides, void* dv, const prism_strides* dv_strides,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const prism_status st = attn_check(B, H, G, T, D, S, lens, starts, scale, window, dt);
  if (st != PRISM_OK) return st;
  if (!q || !k || !v || !o || !lse || !d_o || !dq || !dk || !dv) return PRISM_ERR_INVALID_ARG;
  if (window > 0 && !causal) return PRISM_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (!make_strides(q_strides, B, H, T, D, &a.qs) || !make_strides(k_strides, B, G, T, D, &a.ks) ||
      !make_strides(v_strides, B, G, T, D, &a.vs) || !make_strides(o_strides, B, H, T, D, &a.os) ||
      !make_strides(do_strides, B, H, T, D, &a.dos) || !make_strides(dq_strides, B, H, T, D, &a.dqs) ||
      !make_strides(dk_strides, B, G, T, D, &a.dks) || !make_strides(dv_strides, B, G, T, D, &a.dvs) ||
      !rows_apart(a.dqs, B, H, T, D) || !rows_apart(a.dks, B, G, T, D) || !rows_apart(a.dvs, B, G, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(q, a.qs, D, dt) || !scan_rows(k, a.ks, D, dt) || !scan_rows(v, a.vs, D, dt) || !scan_rows(o, a.os, D, dt) ||
      !scan_rows(d_o, a.dos, D, dt) || !scan_rows(dq, a.dqs, D, dt) || !scan_rows(dk, a.dks, D, dt) || !scan_rows(dv, a.dvs, D, dt))
    return PRISM_ERR_UNSUPPORTED;
  const size_t need = prism_attn_bwd_workspace_bytes(B, H, G, T, D, dt);
  if (need == 0) return PRISM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  // dq is written before the other kernel reads q, k, v and do; dk before other workgroups have read k
  for (const void* in : {q, k, v, o, d_o})
    if (dq == in || dk == in || dv == in) return PRISM_ERR_INVALID_ARG;
  a.q = q, a.k = k, a.v = v, a.o = const_cast<void*>(o), a.lse = const_cast<float*>(lse), a.dout = d_o;
  a.lens = lens, a.starts = starts, a.B = B, a.H = H, a.G = G, a.T = T, a.S = S;
  a.causal = causal != 0, a.window = window, a.scale = scale;
  a.delta = reinterpret_cast<float*>(workspace), a.dq = dq, a.dk = dk, a.dv = dv;
  return host::launch_attn_bwd(dt, D, a, stream);
}

}  // extern "C"
