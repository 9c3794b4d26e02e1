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
  if (H > 65535 || (long long)T * (H / G) > INT_MAX - 4096) return PRISM_ERR_UNSUPPORTED;  // a group's rows are counted in 31 bits
  return tiles > ((size_t)1 << 23) / H ? PRISM_ERR_UNSUPPORTED : PRISM_OK;
}

// Norm and rotation: sizes, and the lane groups' share of a token's heads.
int rope_lanes(int D, int rot) { return D % 8 != 0 || rot % 8 != 0 ? 64 : D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// An output's rows may be those of its own input, with its strides.
bool same(const prism_strides& x, const prism_strides& y) { return x.b == y.b && x.h == y.h && x.t == y.t; }
bool in_place(const void* const* x, const prism_strides* xs, void* const* y, const prism_strides* ys) {
  if (y[0] == y[1] || y[0] == x[1] || y[1] == x[0]) return false;
  return (y[0] != x[0] || same(xs[0], ys[0])) && (y[1] != x[1] || same(xs[1], ys[1]));
}

prism_status rope_plan(int B, int H, int G, int T, int D, int rot, float factor, float eps, prism_dtype dt, RopeArgs* a) {
  if (B <= 0 || H <= 0 || G <= 0 || T <= 0 || D <= 0 || rot <= 0 || rot > D || !known(dt)) return PRISM_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(factor)) return PRISM_ERR_INVALID_ARG;
  if (D % 2 != 0 || rot % 2 != 0 || D > 512 || H > 65535 || G > 65535) return PRISM_ERR_UNSUPPORTED;
  const size_t tokens = (size_t)B * T, heads = (size_t)H + G, lanes = rope_lanes(D, rot);
  if (tokens > ((size_t)1 << 31) / lanes / heads) return PRISM_ERR_UNSUPPORTED;
  // heads of a token that share their sines and cosines, as long as every CU keeps 8 waves
  a->per = (int)std::min(heads, std::max<size_t>(1, tokens * heads * lanes / 64 / (8 * kCUs)));
  a->groups = (int)((heads + a->per - 1) / a->per);
  a->per = (int)((heads + a->groups - 1) / a->groups);
  const size_t slots = 256 / lanes;
  a->nblk = (int)std::min<size_t>((tokens * a->groups + slots - 1) / slots, 4 * kCUs);
  a->B = B, a->T = T, a->D = D, a->heads[0] = H, a->heads[1] = G, a->rot = rot, a->factor = factor, a->eps = eps;
  return PRISM_OK;
}

// The paged cache's sizes; page: a power of two.
prism_status cache_check(int G, int D, int pages, int page, int max_pages, int T, bool bits8, prism_dtype dt) {
  if (pages <= 0 || page <= 0 || max_pages <= 0) return PRISM_ERR_INVALID_ARG;
  if (bits8 && dt != PRISM_BF16) return PRISM_ERR_UNSUPPORTED;
  if ((page & (page - 1)) != 0 || page < 16 || page > 1024) return PRISM_ERR_UNSUPPORTED;
  return (long long)max_pages * page + T > INT_MAX - 8192 ? PRISM_ERR_UNSUPPORTED : PRISM_OK;
}

// How new tokens read the cache.  Few rows of a group's heads: tiles of 32 rows that share the cache's keys; else 128 rows of a head to a
// workgroup, 256 of wide heads.  A sequence's keys are split until the device is full, into ranges of 512 keys or more (128 where
// that leaves CUs without any) of the max_pages * page keys that its table has room for: the host does not know how many a sequence
// holds, nor is the window reckoned with, and a kernel deals out what a sequence has to all the ranges evenly.
// Measured, us: 256 rows (8 x 16 heads x 32 tokens over 4096 of 128) 46 as few, 75 as many, 512 rows (2 x 16 x 128 over 8192) 39 as many
// with one workgroup per CU, 48 with two (of 64 wide heads two fit a CU: 512 tokens 63 with two, 83 with one); 1 x 32 x 512 tokens over
// 4096: 88 with 128 rows, 62 with 256; single tokens of 13 x 2 over 11610: 38 with ranges of 512, 40 of 256; 4 x 8 over 500: 13.5 and
// 11.2 with 128.
struct PagedPlan {
  int rows, splits;               // rows of a tile: 32 (few), 128 or 256
  size_t total;
};
PagedPlan paged_plan(int B, int H, int G, int T, int D, int page, int max_pages, prism_dtype dt) {
  PagedPlan pl;
  const size_t rows = (size_t)T * (H / G), keys = (size_t)max_pages * page;
  const bool wide = D == 128 && dt == PRISM_BF16 && T >= 256;
  pl.rows = rows <= 256 ? 32 : wide ? 256 : 128;
  const size_t units = pl.rows == 32 ? (size_t)B * G * ((rows + 31) / 32) : (size_t)B * H * ((T + pl.rows - 1) / pl.rows);
  const size_t want = ((pl.rows == 32 ? 4 : D == 128 ? 1 : 2) * kCUs + units - 1) / units;
  size_t range = 512;
  while (range > 128 && units * (keys / range) < kCUs) range /= 2;
  pl.splits = (int)std::min<size_t>(std::min(want, std::max<size_t>(1, keys / range)), 64);
  Layout ly;
  if (pl.splits > 1) ly.add((size_t)pl.splits * B * H * T, (size_t)(D + 2) * 4);
  pl.total = ly.ok() ? std::max<size_t>(ly.total, 256) : 0;
  return pl;
}

}  // namespace

extern "C" {

prism_status prism_attn_fwd(const void* q, const prism_strides* q_strides, const void* k, const prism_strides* k_strides,
                            const void* v, const prism_strides* v_strides, const int* lens, const int* starts, int S,
                            int B, int H, int G, int T, int D, float scale, int causal, int window, prism_dtype dt,
                            void* o, const prism_strides* o_strides, float* lse, hipStream_t stream) {
  const prism_status st = attn_check(B, H, G, T, D, S, lens, starts, scale, window, dt);
  if (st != PRISM_OK) return st;
  if (!q || !k || !v || !o || o == q || o == k || o == v) return PRISM_ERR_INVALID_ARG;
  if (window > 0 && !causal) return PRISM_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (!make_strides(q_strides, B, H, T, D, &a.qs) || !make_strides(k_strides, B, G, T, D, &a.ks) ||
      !make_strides(v_strides, B, G, T, D, &a.vs) || !make_strides(o_strides, B, H, T, D, &a.os) || !rows_apart(a.os, B, H, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(q, a.qs, D, dt) || !scan_rows(k, a.ks, D, dt) || !scan_rows(v, a.vs, D, dt) || !scan_rows(o, a.os, D, dt))
    return PRISM_ERR_UNSUPPORTED;
  a.q = q, a.k = k, a.v = v, a.lens = lens, a.starts = starts;
  a.B = B, a.H = H, a.G = G, a.T = T, a.S = S, a.causal = causal != 0, a.window = window, a.scale = scale;
  a.splits = 1, a.o = o, a.lse = lse;
  return host::launch_attn_fwd(dt, D, a, stream);
}

// The pass by keys: a group's heads go to `splits` workgroups where the key tiles alone leave the device empty.
struct BwdPlan {
  int splits;
  size_t part, total;
};
static BwdPlan bwd_plan(int B, int H, int G, int T, int D) {
  BwdPlan pl;
  const size_t units = (size_t)B * G * (((size_t)T + 127) / 128), rep = (size_t)(H / G);
  const size_t want = std::min(rep, (2 * kCUs + units - 1) / units), each = (rep + want - 1) / want;
  pl.splits = (int)((rep + each - 1) / each);
  Layout ly;
  ly.add((size_t)B * H, (size_t)T * 4);
  pl.part = ly.add(pl.splits > 1 ? 2 * (size_t)pl.splits * B * G : 0, (size_t)T * D * 4);
  pl.total = ly.ok() ? ly.total : 0;
  return pl;
}

size_t prism_attn_bwd_workspace_bytes(int B, int H, int G, int T, int D, prism_dtype dt) {
  if (attn_check(B, H, G, T, D, 0, nullptr, nullptr, 1.f, 0, dt) != PRISM_OK) return 0;
  return bwd_plan(B, H, G, T, D).total;
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
  const BwdPlan pl = bwd_plan(B, H, G, T, D);
  if (pl.total == 0) return PRISM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < pl.total) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  // dq is written before the other kernel reads q, k, v and do; dk before other workgroups have read k
  for (const void* in : {q, k, v, o, d_o})
    if (dq == in || dk == in || dv == in) return PRISM_ERR_INVALID_ARG;
  if (dq == dk || dq == dv || dk == dv) return PRISM_ERR_INVALID_ARG;
  a.q = q, a.k = k, a.v = v, a.o = const_cast<void*>(o), a.lse = const_cast<float*>(lse), a.dout = d_o;
  a.lens = lens, a.starts = starts, a.B = B, a.H = H, a.G = G, a.T = T, a.S = S;
  a.causal = causal != 0, a.window = window, a.scale = scale;
  a.delta = reinterpret_cast<float*>(workspace), a.part = at<float>(workspace, pl.part), a.splits = pl.splits;
  a.dq = dq, a.dk = dk, a.dv = dv;
  return host::launch_attn_bwd(dt, D, a, stream);
}

prism_status prism_rope_fwd(const void* q, const prism_strides* q_strides, const void* k, const prism_strides* k_strides,
                            const float* freq, const int* pos, const float* wq, const float* wk,
                            int B, int H, int G, int T, int D, int rot, int interleaved, float factor, float eps,
                            prism_dtype dt, void* yq, const prism_strides* yq_strides, void* yk,
                            const prism_strides* yk_strides, hipStream_t stream) {
  RopeArgs a = {};
  const prism_status st = rope_plan(B, H, G, T, D, rot, factor, eps, dt, &a);
  if (st != PRISM_OK) return st;
  if (!q || !k || !freq || !yq || !yk || (wq == nullptr) != (wk == nullptr)) return PRISM_ERR_INVALID_ARG;
  if (!make_strides(q_strides, B, H, T, D, &a.xs[0]) || !make_strides(k_strides, B, G, T, D, &a.xs[1]) ||
      !make_strides(yq_strides, B, H, T, D, &a.ys[0]) || !make_strides(yk_strides, B, G, T, D, &a.ys[1]) ||
      !rows_apart(a.ys[0], B, H, T, D) || !rows_apart(a.ys[1], B, G, T, D))
    return PRISM_ERR_INVALID_ARG;
  a.x[0] = q, a.x[1] = k, a.y[0] = yq, a.y[1] = yk, a.w[0] = wq, a.w[1] = wk, a.freq = freq, a.pos = pos;
  a.interleaved = interleaved != 0;
  if (!in_place(a.x, a.xs, a.y, a.ys)) return PRISM_ERR_INVALID_ARG;
  return host::launch_rope(dt, false, a, stream);
}

size_t prism_rope_bwd_workspace_bytes(int B, int H, int G, int T, int D, int rot, prism_dtype dt) {
  RopeArgs a = {};
  if (rope_plan(B, H, G, T, D, rot, 1.f, 0.f, dt, &a) != PRISM_OK) return 0;
  Layout ly;
  ly.add((size_t)a.nblk * 2, (size_t)D * 4);
  return ly.total;
}

prism_status prism_rope_bwd(const void* q, const prism_strides* q_strides, const void* k, const prism_strides* k_strides,
                            const void* dyq, const prism_strides* dyq_strides, const void* dyk,
                            const prism_strides* dyk_strides, const float* freq, const int* pos, const float* wq,
                            const float* wk, int B, int H, int G, int T, int D, int rot, int interleaved, float factor,
                            float eps, prism_dtype dt, void* dq, const prism_strides* dq_strides, void* dk,
                            const prism_strides* dk_strides, float* dwq, float* dwk, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  RopeArgs a = {};
  const prism_status st = rope_plan(B, H, G, T, D, rot, factor, eps, dt, &a);
  if (st != PRISM_OK) return st;
  const bool norm = wq != nullptr;
  if (!dyq || !dyk || !freq || !dq || !dk || norm != (wk != nullptr) || (norm && (!q || !k))) return PRISM_ERR_INVALID_ARG;
  if (!norm && (dwq || dwk)) return PRISM_ERR_INVALID_ARG;
  if (!make_strides(q_strides, B, H, T, D, &a.xs[0]) || !make_strides(k_strides, B, G, T, D, &a.xs[1]) ||
      !make_strides(dyq_strides, B, H, T, D, &a.dys[0]) || !make_strides(dyk_strides, B, G, T, D, &a.dys[1]) ||
      !make_strides(dq_strides, B, H, T, D, &a.ys[0]) || !make_strides(dk_strides, B, G, T, D, &a.ys[1]) ||
      !rows_apart(a.ys[0], B, H, T, D) || !rows_apart(a.ys[1], B, G, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (norm && (dwq || dwk)) {
    if (!workspace || workspace_bytes < prism_rope_bwd_workspace_bytes(B, H, G, T, D, rot, dt)) return PRISM_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
    a.part = reinterpret_cast<float*>(workspace);
  }
  a.x[0] = q, a.x[1] = k, a.dy[0] = dyq, a.dy[1] = dyk, a.y[0] = dq, a.y[1] = dk, a.w[0] = wq, a.w[1] = wk;
  a.dw[0] = dwq, a.dw[1] = dwk, a.freq = freq, a.pos = pos, a.interleaved = interleaved != 0;
  if (!in_place(a.dy, a.dys, a.y, a.ys)) return PRISM_ERR_INVALID_ARG;
  if (norm && (dq == q || dq == k || dk == q || dk == k)) return PRISM_ERR_INVALID_ARG;
  return host::launch_rope(dt, true, a, stream);
}

prism_status prism_cache_write(const void* k, const prism_strides* k_strides, const void* v, const prism_strides* v_strides,
                               const int* table, const int* past, const int* lens, const int* starts, int S,
                               int B, int G, int T, int D, int pages, int page, int max_pages, prism_dtype dt,
                               void* cache_k, void* cache_v, float* scale_k, float* scale_v, hipStream_t stream) {
  prism_status st = attn_check(B, G, G, T, D, S, lens, starts, 1.f, 0, dt);
  if (st == PRISM_OK) st = cache_check(G, D, pages, page, max_pages, T, scale_k != nullptr, dt);
  if (st != PRISM_OK) return st;
  if (!k || !v || !table || !past || !cache_k || !cache_v || (scale_k == nullptr) != (scale_v == nullptr)) return PRISM_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (!make_strides(k_strides, B, G, T, D, &a.ks) || !make_strides(v_strides, B, G, T, D, &a.vs)) return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(k, a.ks, D, dt) || !scan_rows(v, a.vs, D, dt) || !aligned16(cache_k) || !aligned16(cache_v)) return PRISM_ERR_UNSUPPORTED;
  if (cache_k == cache_v || (scale_k != nullptr && scale_k == scale_v)) return PRISM_ERR_INVALID_ARG;
  a.k = k, a.v = v, a.lens = lens, a.starts = starts, a.B = B, a.H = G, a.G = G, a.T = T, a.S = S;
  a.cache_k = cache_k, a.cache_v = cache_v, a.cache_ks = scale_k, a.cache_vs = scale_v, a.table = table, a.past = past;
  a.pages = pages, a.page_shift = __builtin_ctz((unsigned)page), a.max_pages = max_pages;
  return host::launch_cache_write(dt, D, scale_k != nullptr, a, stream);
}

size_t prism_attn_paged_workspace_bytes(int B, int H, int G, int T, int D, int page, int max_pages, prism_dtype dt) {
  if (attn_check(B, H, G, T, D, 0, nullptr, nullptr, 1.f, 0, dt) != PRISM_OK) return 0;
  if (cache_check(G, D, 1, page, max_pages, T, false, dt) != PRISM_OK) return 0;
  return paged_plan(B, H, G, T, D, page, max_pages, dt).total;
}

prism_status prism_attn_paged(const void* q, const prism_strides* q_strides, const void* cache_k, const void* cache_v,
                              const float* scale_k, const float* scale_v, const int* table, const int* past,
                              const int* lens, int B, int H, int G, int T, int D, int pages, int page, int max_pages,
                              float scale, int window, prism_dtype dt, void* o, const prism_strides* o_strides,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  prism_status st = attn_check(B, H, G, T, D, 0, lens, nullptr, scale, window, dt);
  if (st == PRISM_OK) st = cache_check(G, D, pages, page, max_pages, T, scale_k != nullptr, dt);
  if (st != PRISM_OK) return st;
  if (!q || !cache_k || !cache_v || !table || !past || !o || o == q || (scale_k == nullptr) != (scale_v == nullptr))
    return PRISM_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (!make_strides(q_strides, B, H, T, D, &a.qs) || !make_strides(o_strides, B, H, T, D, &a.os) || !rows_apart(a.os, B, H, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(q, a.qs, D, dt) || !scan_rows(o, a.os, D, dt) || !aligned16(cache_k) || !aligned16(cache_v)) return PRISM_ERR_UNSUPPORTED;
  const PagedPlan pl = paged_plan(B, H, G, T, D, page, max_pages, dt);
  if (pl.total == 0) return PRISM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < pl.total) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  a.q = q, a.lens = lens, a.B = B, a.H = H, a.G = G, a.T = T, a.causal = 1, a.window = window, a.scale = scale;
  a.cache_k = const_cast<void*>(cache_k), a.cache_v = const_cast<void*>(cache_v);
  a.cache_ks = const_cast<float*>(scale_k), a.cache_vs = const_cast<float*>(scale_v), a.table = table, a.past = past;
  a.pages = pages, a.page_shift = __builtin_ctz((unsigned)page), a.max_pages = max_pages;
  a.o = o, a.splits = pl.splits, a.part = reinterpret_cast<float*>(workspace);
  return host::launch_attn_paged(dt, D, scale_k != nullptr, pl.rows, a, stream);
}

}  // extern "C"
