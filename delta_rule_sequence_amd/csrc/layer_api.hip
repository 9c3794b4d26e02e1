// layer_api.hip - C ABI of the state space layer (include/prism.h): argument checks, plans and workspace
// layout of the convolution, the selective scan and the norm.  Host side only; every check runs before anything
// is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <stdint.h>

#include "prism.h"
#include "prism_ssm_args.h"

namespace prism {
namespace host {
#define PRISM_DECL_SSM(NAME)                                              \
  prism_status NAME##_fwd(int pw, const SsmArgs& a, hipStream_t s);       \
  prism_status NAME##_bwd(int pw, const SsmArgs& a, hipStream_t s);       \
  prism_status NAME##_step(int p, int B, const SsmStepArgs& a, hipStream_t s);
PRISM_DECL_SSM(ssm_bf16_n16)
PRISM_DECL_SSM(ssm_bf16_n32)
PRISM_DECL_SSM(ssm_bf16_n64)
PRISM_DECL_SSM(ssm_bf16_n128)
PRISM_DECL_SSM(ssm_f32_n16)
PRISM_DECL_SSM(ssm_f32_n32)
PRISM_DECL_SSM(ssm_f32_n64)
PRISM_DECL_SSM(ssm_f32_n128)
#undef PRISM_DECL_SSM

#define PRISM_BY_TYPE_AND_N(OP, ...)                                                              \
  (ty == PRISM_BF16 ? (N == 16   ? ssm_bf16_n16_##OP(__VA_ARGS__)                                 \
                       : N == 32 ? ssm_bf16_n32_##OP(__VA_ARGS__)                                 \
                       : N == 64 ? ssm_bf16_n64_##OP(__VA_ARGS__) : ssm_bf16_n128_##OP(__VA_ARGS__)) \
                    : (N == 16   ? ssm_f32_n16_##OP(__VA_ARGS__)                                  \
                       : N == 32 ? ssm_f32_n32_##OP(__VA_ARGS__)                                  \
                       : N == 64 ? ssm_f32_n64_##OP(__VA_ARGS__) : ssm_f32_n128_##OP(__VA_ARGS__)))

prism_status launch_ssm_fwd(prism_dtype ty, int N, int PW, const SsmArgs& a, hipStream_t stream) {
  return PRISM_BY_TYPE_AND_N(fwd, PW, a, stream);
}
prism_status launch_ssm_bwd(prism_dtype ty, int N, int PW, const SsmArgs& a, hipStream_t stream) {
  return PRISM_BY_TYPE_AND_N(bwd, PW, a, stream);
}
prism_status launch_ssm_step(prism_dtype ty, int N, int P, int B, const SsmStepArgs& a, hipStream_t stream) {
  return PRISM_BY_TYPE_AND_N(step, P, B, a, stream);
}
#undef PRISM_BY_TYPE_AND_N
}  // namespace host
}  // namespace prism

namespace {

using namespace prism;

constexpr int kChunk = 64;       // tokens per chunk of the scan (ssm::Q)
constexpr size_t kCUs = 256;     // compute units of an MI355X
constexpr int kMaxWidth = 1 << 26;  // channels of the convolution and the norm: the launches' 32-bit thread counts
constexpr int kFold = 8;         // most segments whose entering states their readers form (bfloat16)

size_t elem(prism_dtype dt) { return dt == PRISM_BF16 ? 2 : 4; }
bool known(prism_dtype dt) { return dt == PRISM_F32 || dt == PRISM_BF16; }
bool width_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

// A workspace layout: offsets of 256-byte aligned regions; total stays SIZE_MAX after an overflow.
struct Layout {
  size_t total = 0;
  size_t add(size_t count, size_t size) {
    const size_t at = total;
    if (total == SIZE_MAX || (size != 0 && count > (SIZE_MAX / 2 - total) / size)) {
      total = SIZE_MAX;
      return 0;
    }
    total += (count * size + 255) / 256 * 256;
    return at;
  }
  bool ok() const { return total != SIZE_MAX; }
};

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Strides of a [B, H, T, width] tensor: the caller's, or dense ones.  Checks signs and that the largest offset fits
// in 63 bits.
bool make_strides(const prism_strides* given, int B, int H, int T, int width, prism_strides* out) {
  if (given == nullptr) {
    out->t = width;
    out->h = (long long)T * width;
    if (out->h > LLONG_MAX / 8 / H) return false;
    out->b = out->h * H;
  } else {
    *out = *given;
    if ((B > 1 && out->b <= 0) || (H > 1 && out->h <= 0) || (T > 1 && out->t <= 0)) return false;
    if (B == 1) out->b = 0;
    if (H == 1) out->h = 0;
    if (T == 1) out->t = width;
  }
  const long long lim = LLONG_MAX / 64;
  return out->b <= lim / B && out->h <= lim / H && out->t <= lim / T;
}

// Whether rows of an output [B, H, T, width] cannot overlap: sorted by stride, each axis steps over the ones below.
bool rows_apart(const prism_strides& s, int B, int H, int T, int width) {
  struct Axis { long long st; long long n; } ax[3] = {{s.b, B}, {s.h, H}, {s.t, T}};
  std::sort(ax, ax + 3, [](const Axis& p, const Axis& q) { return p.st < q.st; });
  long long span = width;
  for (const Axis& a : ax) {
    if (a.n == 1) continue;
    if (a.st < span) return false;
    span += a.st * (a.n - 1);
  }
  return true;
}

// Rows of the scan's tensors: on 16-byte boundaries, not overlapping, and at most 16 MB apart (a chunk's rows are
// addressed with 32-bit byte offsets).
bool rows16(const void* p, const prism_strides& s, prism_dtype dt);
bool scan_rows(const void* p, const prism_strides& s, int width, prism_dtype dt) {
  return rows16(p, s, dt) && s.t >= width && s.t * (long long)elem(dt) <= (1 << 24);
}

bool rows16(const void* p, const prism_strides& s, prism_dtype dt) {
  const long long e = (long long)elem(dt);
  return aligned16(p) && s.b * e % 16 == 0 && s.h * e % 16 == 0 && s.t * e % 16 == 0;
}

// ---- scan ------------------------------------------------------------------------------------
struct SsmPlan {
  int PW, nsl, HV, nch, seg_chunks, nseg, nsplit, per_split;
  size_t seg, seg_dec, st, part_b, part_c, part_ddt, part_sum, total;
};

prism_status ssm_plan(int B, int H, int G, int T, int N, int P, prism_dtype ty, bool bwd, SsmPlan* pl) {
  if (B <= 0 || H <= 0 || G <= 0 || T <= 0 || N <= 0 || P <= 0) return PRISM_ERR_INVALID_ARG;
  if (!known(ty) || H % G != 0) return PRISM_ERR_INVALID_ARG;
  if (!width_ok(N) || !width_ok(P) || T > INT_MAX - 4096) return PRISM_ERR_UNSUPPORTED;
  pl->PW = std::min(P, 64);
  pl->nsl = P / pl->PW;
  if ((size_t)B * (size_t)H * (size_t)pl->nsl > 65535) return PRISM_ERR_UNSUPPORTED;  // (b, virtual head) pairs map to grid.y
  pl->HV = H * pl->nsl;
  pl->nch = (int)(((long long)T + kChunk - 1) / kChunk);
  // Segments until the device is full: each costs a state in the workspace and a second read of its inputs; up to kFold of
  // them the passes form their entering states themselves, more take a scan over them.  Forward: two workgroups of two
  // heads per CU and some more, since a batch may be ragged (8 x 24 x 2048 tokens, N = 128: 148 us with 2 segments, 110 with
  // 4, 97 with 5, 99 with 6, 104 with 8, but ragged 92 with 5, 86 with 6, 94 with 8; 32 x 8 x 1024: 69 with 4, 84 with 8), no
  // more than those two per CU where the scan comes on top (8 x 12 x 2048: 62 with 8, 72 with 11; 2 x 4 x 16384, N = 64: 42 with
  // 64, 39 with 128).  Half as many for float32 where they are more than kFold (4 x 8 x 2048, N = 64: 55 with 16, 59 with 32; else
  // not: 8 x 12 x 2048, N = 128: 317 with 5, 283 with 8) and for the backward, whose two directions fill the device sooner (8 x 12 x
  // 2048: 191 with 5, 204 with 8; 2 x 4 x 16384: 110 with 64, 125 with 128) and which takes one rather than two (8 x 24 x 2048:
  // 338 and 354; 32 x 8 x 1024: 224 and 244).
  // Least chunks of a segment: two for bfloat16; a float32 chunk takes longer than a segment costs (3 x 6 x 509 tokens,
  // N = P = 32: a call of 29 us with two, 26 with one).
  const int least = ty == PRISM_BF16 || pl->nch <= 2 ? 2 : 1;
  const size_t bh = (size_t)B * pl->HV;
  const auto cut = [&](size_t want) {
    pl->seg_chunks = std::max(std::min(pl->nch, least), (int)((pl->nch + want - 1) / want));
    pl->nseg = (pl->nch + pl->seg_chunks - 1) / pl->seg_chunks;
  };
  const size_t half = std::max<size_t>(1, 2 * kCUs / bh);
  if (bwd) {
    cut(half == 2 ? 1 : half);
  } else {
    cut(std::max<size_t>(1, 9 * kCUs / 2 / bh));
    if (pl->nseg > kFold) cut(4 * kCUs / bh);
    if (pl->nseg > kFold && ty == PRISM_F32) cut(half);
  }
  const size_t mat = (size_t)N * pl->PW;
  Layout ly;
  const int dirs = bwd ? 2 : 1;
  const bool segs = bwd || pl->nseg > 1;
  pl->seg = ly.add(segs ? dirs * bh * pl->nseg : 0, mat * 4);
  pl->seg_dec = ly.add(segs ? dirs * bh * pl->nseg : 0, 4);
  if (bwd) {
    // The gradient pass: a workgroup walks per_split of a group's virtual heads, and loads and sums outside the heads cost
    // it about one more.  Splits for the least time over the rounds that the device needs; a CU holds one workgroup, or two
    // of float32 with small tiles.  (float32, 24 heads of 128 in 4 groups, 2464 tokens, N = 16: 157 us with 2 splits, 124 with
    // 3, 150 with 4; 16 heads of 64 in 2 groups, N = 128, 1733 tokens: 175 with 2, 125 with 4, 141 with 8;
    // bfloat16, 3 x 8 of 64, N = 64, 4000 tokens: 95 with 1, 103 with 2, 102 with 4.)
    const unsigned per_group = (unsigned)(pl->HV / G);
    const size_t units = (size_t)pl->nch * B * G, slots = ty == PRISM_F32 && N + pl->PW <= 96 ? 2 * kCUs : kCUs;
    size_t least_time = SIZE_MAX;
    for (unsigned ns = 1; ns <= std::min(per_group, 64u); ++ns) {
      const unsigned per = (per_group + ns - 1) / ns, n = (per_group + per - 1) / per;
      const size_t time = (units * n + slots - 1) / slots * (per + 1);
      if (time < least_time) least_time = time, pl->per_split = (int)per, pl->nsplit = (int)n;
    }
    const size_t rows = (size_t)B * G * T;
    pl->st = ly.add(2 * bh * pl->nch, mat * 4);
    pl->part_b = ly.add(pl->nsplit > 1 ? pl->nsplit * rows : 0, (size_t)N * 4);
    pl->part_c = ly.add(pl->nsplit > 1 ? pl->nsplit * rows : 0, (size_t)N * 4);
    pl->part_ddt = ly.add(pl->nsl > 1 ? (size_t)pl->nsl * B * H : 0, (size_t)T * 4);
    pl->part_sum = ly.add(3 * bh, (size_t)pl->nch * 4);
    // the launches cover these with 32-bit grids
    const size_t most = (size_t)UINT_MAX - 768 * (size_t)H - 1024;
    if (rows * (N / 4) + (size_t)B * H * T > most || (size_t)pl->nch * 512 > most) return PRISM_ERR_UNSUPPORTED;
  }
  if (!ly.ok()) return PRISM_ERR_INVALID_ARG;
  pl->total = std::max<size_t>(ly.total, 256);
  return PRISM_OK;
}

template <class P> P* at(void* ws, size_t off) { return reinterpret_cast<P*>(reinterpret_cast<char*>(ws) + off); }

// ---- convolution -------------------------------------------------------------------------------
prism_status conv_check(int B, int H, int T, int D, int K, prism_dtype dt) {
  if (B <= 0 || H <= 0 || T <= 0 || D <= 0 || !known(dt)) return PRISM_ERR_INVALID_ARG;
  if (K < 2 || K > 4) return PRISM_ERR_UNSUPPORTED;
  if ((size_t)B * (size_t)H > 65535) return PRISM_ERR_UNSUPPORTED;  // (b, h) pairs map to grid.z / grid.y
  if ((size_t)B * H > (size_t)INT_MAX / (size_t)D) return PRISM_ERR_UNSUPPORTED;
  if (D > kMaxWidth || T > INT_MAX - 4096) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

// Tokens per thread: long strips read their K - 1 border rows (and, backward, leave their shares of dw) once for
// more tokens, short ones fill the device when there are few channels.
int conv_strip(int B, int H, int T, int D, prism_dtype dt, bool bwd) {
  const size_t per = bwd || elem(dt) == 4 ? conv_group<4>(D) : conv_group<8>(D), cols = (size_t)B * H * (((size_t)D + per - 1) / per);
  int strip = bwd ? 64 : 32;
  while (strip > 8 && cols * (((size_t)T + strip - 1) / strip) < (bwd ? 8 : 16) * 64 * kCUs) strip /= 2;
  // workgroups of four strips map to grid.y
  while (((size_t)T + strip - 1) / strip / 4 + 1 > 65535) strip *= 2;
  return strip;
}

}  // namespace

extern "C" {

size_t prism_ssm_fwd_workspace_bytes(int B, int H, int G, int T, int N, int P, prism_dtype ty) {
  SsmPlan pl;
  return ssm_plan(B, H, G, T, N, P, ty, false, &pl) == PRISM_OK ? pl.total : 0;
}

prism_status prism_ssm_fwd(const void* x, const prism_strides* x_strides, const void* Bm,
                           const prism_strides* b_strides, const void* Cm, const prism_strides* c_strides,
                           const float* dt, const prism_strides* dt_strides, const float* dt_bias, const float* A,
                           const float* D, const float* S0, const int* lens,
                           int B, int H, int G, int T, int N, int P, int softplus, prism_dtype ty,
                           void* y, const prism_strides* y_strides, float* S_final,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  SsmPlan pl;
  const prism_status st = ssm_plan(B, H, G, T, N, P, ty, false, &pl);
  if (st != PRISM_OK) return st;
  if (!x || !Bm || !Cm || !dt || !A || !y || !S_final) return PRISM_ERR_INVALID_ARG;
  SsmArgs a = {};
  if (!make_strides(x_strides, B, H, T, P, &a.xs) || !make_strides(b_strides, B, G, T, N, &a.bs) ||
      !make_strides(c_strides, B, G, T, N, &a.cs) || !make_strides(dt_strides, B, H, T, 1, &a.ts) ||
      !make_strides(y_strides, B, H, T, P, &a.ys) || !rows_apart(a.ys, B, H, T, P))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(x, a.xs, P, ty) || !scan_rows(Bm, a.bs, N, ty) || !scan_rows(Cm, a.cs, N, ty) || !scan_rows(y, a.ys, P, ty))
    return PRISM_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < pl.total) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  a.x = x, a.bm = Bm, a.cm = Cm, a.dt = dt, a.dt_bias = dt_bias, a.A = A, a.D = D, a.lens = lens, a.S0 = S0;
  a.B = B, a.H = H, a.G = G, a.T = T, a.P = P, a.softplus = softplus != 0;
  a.nsl = pl.nsl, a.nch = pl.nch, a.seg_chunks = pl.seg_chunks, a.nseg = pl.nseg, a.fold = pl.nseg <= kFold;
  a.y = y, a.S_final = S_final;
  a.seg = at<float>(workspace, pl.seg), a.seg_dec = at<float>(workspace, pl.seg_dec);
  return host::launch_ssm_fwd(ty, N, pl.PW, a, stream);
}

size_t prism_ssm_bwd_workspace_bytes(int B, int H, int G, int T, int N, int P, prism_dtype ty) {
  SsmPlan pl;
  return ssm_plan(B, H, G, T, N, P, ty, true, &pl) == PRISM_OK ? pl.total : 0;
}

prism_status prism_ssm_bwd(const void* x, const prism_strides* x_strides, const void* Bm,
                           const prism_strides* b_strides, const void* Cm, const prism_strides* c_strides,
                           const float* dt, const prism_strides* dt_strides, const float* dt_bias, const float* A,
                           const float* D, const void* dy, const prism_strides* dy_strides, const float* dS_final,
                           int B, int H, int G, int T, int N, int P, int softplus, prism_dtype ty,
                           void* dx, const prism_strides* dx_strides, void* dBm, const prism_strides* db_strides,
                           void* dCm, const prism_strides* dc_strides, float* ddt, float* dA, float* dD,
                           float* ddt_bias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  SsmPlan pl;
  const prism_status st = ssm_plan(B, H, G, T, N, P, ty, true, &pl);
  if (st != PRISM_OK) return st;
  if (!x || !Bm || !Cm || !dt || !A || !dy || !dx || !dBm || !dCm || !ddt || !dA) return PRISM_ERR_INVALID_ARG;
  SsmArgs a = {};
  if (!make_strides(x_strides, B, H, T, P, &a.xs) || !make_strides(b_strides, B, G, T, N, &a.bs) ||
      !make_strides(c_strides, B, G, T, N, &a.cs) || !make_strides(dt_strides, B, H, T, 1, &a.ts) ||
      !make_strides(dy_strides, B, H, T, P, &a.dys) || !make_strides(dx_strides, B, H, T, P, &a.dxs) ||
      !make_strides(db_strides, B, G, T, N, &a.dbs) || !make_strides(dc_strides, B, G, T, N, &a.dcs) ||
      !rows_apart(a.dxs, B, H, T, P) || !rows_apart(a.dbs, B, G, T, N) || !rows_apart(a.dcs, B, G, T, N))
    return PRISM_ERR_INVALID_ARG;
  if (!scan_rows(x, a.xs, P, ty) || !scan_rows(Bm, a.bs, N, ty) || !scan_rows(Cm, a.cs, N, ty) || !scan_rows(dy, a.dys, P, ty) ||
      !scan_rows(dx, a.dxs, P, ty) || !scan_rows(dBm, a.dbs, N, ty) || !scan_rows(dCm, a.dcs, N, ty))
    return PRISM_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < pl.total) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  a.x = x, a.bm = Bm, a.cm = Cm, a.dy = dy, a.dt = dt, a.dt_bias = dt_bias, a.A = A, a.D = D;
  a.B = B, a.H = H, a.G = G, a.T = T, a.P = P, a.softplus = softplus != 0;
  a.nsl = pl.nsl, a.nch = pl.nch, a.seg_chunks = pl.seg_chunks, a.nseg = pl.nseg, a.fold = pl.nseg <= kFold;
  a.seg = at<float>(workspace, pl.seg), a.seg_dec = at<float>(workspace, pl.seg_dec);
  a.st = at<float>(workspace, pl.st), a.dS = dS_final;
  a.dx = dx, a.dbm = dBm, a.dcm = dCm, a.ddt = ddt, a.dA = dA, a.dD = dD, a.ddt_bias = ddt_bias;
  a.nsplit = pl.nsplit, a.per_split = pl.per_split;
  a.part_b = at<float>(workspace, pl.part_b), a.part_c = at<float>(workspace, pl.part_c);
  a.part_ddt = at<float>(workspace, pl.part_ddt), a.part_sum = at<float>(workspace, pl.part_sum);
  return host::launch_ssm_bwd(ty, N, pl.PW, a, stream);
}

prism_status prism_ssm_step(const void* x, const prism_strides* x_strides, const void* Bm,
                            const prism_strides* b_strides, const void* Cm, const prism_strides* c_strides,
                            const float* dt, const prism_strides* dt_strides, const float* dt_bias, const float* A,
                            const float* D, int B, int H, int G, int N, int P, int softplus, prism_dtype ty,
                            float* S, void* y, hipStream_t stream) {
  if (B <= 0 || H <= 0 || G <= 0 || N <= 0 || P <= 0 || !known(ty) || H % G != 0) return PRISM_ERR_INVALID_ARG;
  if (!width_ok(N) || !width_ok(P)) return PRISM_ERR_UNSUPPORTED;
  if ((size_t)B * (size_t)H > (size_t)INT_MAX / 256) return PRISM_ERR_UNSUPPORTED;
  if (!x || !Bm || !Cm || !dt || !A || !S || !y) return PRISM_ERR_INVALID_ARG;
  SsmStepArgs a = {};
  if (!make_strides(x_strides, B, H, 1, P, &a.xs) || !make_strides(b_strides, B, G, 1, N, &a.bs) ||
      !make_strides(c_strides, B, G, 1, N, &a.cs) || !make_strides(dt_strides, B, H, 1, 1, &a.ts))
    return PRISM_ERR_INVALID_ARG;
  if (!aligned16(S)) return PRISM_ERR_UNSUPPORTED;
  a.x = x, a.bm = Bm, a.cm = Cm, a.dt = dt, a.dt_bias = dt_bias, a.A = A, a.D = D;
  a.H = H, a.G = G, a.softplus = softplus != 0, a.S = S, a.y = y;
  return host::launch_ssm_step(ty, N, P, B, a, stream);
}

prism_status prism_conv_fwd(const void* x, const prism_strides* x_strides, const float* conv_w, const float* bias,
                            const void* conv_in, const int* lens, int B, int H, int T, int D, int K, int silu,
                            prism_dtype dt, void* y, const prism_strides* y_strides, void* conv_out,
                            hipStream_t stream) {
  const prism_status st = conv_check(B, H, T, D, K, dt);
  if (st != PRISM_OK) return st;
  if (!x || !conv_w || !y) return PRISM_ERR_INVALID_ARG;
  ConvArgs a = {};
  if (!make_strides(x_strides, B, H, T, D, &a.xs) || !make_strides(y_strides, B, H, T, D, &a.ys) ||
      !rows_apart(a.ys, B, H, T, D))
    return PRISM_ERR_INVALID_ARG;
  if (y == x) return PRISM_ERR_INVALID_ARG;  // a strip reads rows that its neighbour writes
  a.x = x, a.w = conv_w, a.bias = bias, a.conv_in = conv_in, a.lens = lens, a.y = y, a.conv_out = conv_out;
  a.B = B, a.H = H, a.T = T, a.D = D, a.silu = silu != 0;
  a.strip = conv_strip(B, H, T, D, dt, false);
  a.nstrip = (int)(((long long)T + a.strip - 1) / a.strip);
  return host::launch_conv_fwd(dt, K, a, stream);
}

size_t prism_conv_bwd_workspace_bytes(int B, int H, int T, int D, int K, prism_dtype dt) {
  if (conv_check(B, H, T, D, K, dt) != PRISM_OK) return 0;
  const int strip = conv_strip(B, H, T, D, dt, true);
  Layout ly;
  ly.add((size_t)B * (((size_t)T + 4 * strip - 1) / (4 * strip)) * H * (K + 1), (size_t)D * 4);  // one share per four strips
  return ly.ok() ? ly.total : 0;
}

prism_status prism_conv_bwd(const void* x, const prism_strides* x_strides, const float* conv_w, const float* bias,
                            const void* dy, const prism_strides* dy_strides,
                            int B, int H, int T, int D, int K, int silu, prism_dtype dt,
                            void* dx, const prism_strides* dx_strides, float* dconv_w, float* dbias,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const prism_status st = conv_check(B, H, T, D, K, dt);
  if (st != PRISM_OK) return st;
  if (!x || !conv_w || !dy || !dx || !dconv_w) return PRISM_ERR_INVALID_ARG;
  ConvArgs a = {};
  if (!make_strides(x_strides, B, H, T, D, &a.xs) || !make_strides(dy_strides, B, H, T, D, &a.dys) ||
      !make_strides(dx_strides, B, H, T, D, &a.ys) || !rows_apart(a.ys, B, H, T, D))
    return PRISM_ERR_INVALID_ARG;
  const size_t need = prism_conv_bwd_workspace_bytes(B, H, T, D, K, dt);
  if (need == 0) return PRISM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace) || dx == x || dx == dy) return PRISM_ERR_INVALID_ARG;
  a.x = x, a.w = conv_w, a.bias = bias, a.dy = dy, a.y = dx;
  a.B = B, a.H = H, a.T = T, a.D = D, a.silu = silu != 0;
  a.strip = conv_strip(B, H, T, D, dt, true);
  a.nstrip = (int)(((long long)T + a.strip - 1) / a.strip);
  a.part = reinterpret_cast<float*>(workspace), a.dw = dconv_w, a.dbias = dbias;
  return host::launch_conv_bwd(dt, K, a, stream);
}

prism_status prism_conv_step(const void* x, const prism_strides* x_strides, const float* conv_w, const float* bias,
                             int B, int H, int D, int K, int silu, prism_dtype dt, void* conv_state, void* y,
                             hipStream_t stream) {
  const prism_status st = conv_check(B, H, 1, D, K, dt);
  if (st != PRISM_OK) return st;
  if (!x || !conv_w || !conv_state || !y) return PRISM_ERR_INVALID_ARG;
  ConvArgs a = {};
  if (!make_strides(x_strides, B, H, 1, D, &a.xs)) return PRISM_ERR_INVALID_ARG;
  a.x = x, a.w = conv_w, a.bias = bias, a.conv_in = conv_state, a.y = y;
  a.B = B, a.H = H, a.T = 1, a.D = D, a.silu = silu != 0;
  return host::launch_conv_step(dt, K, a, stream);
}

static prism_status norm_check(int rows, int D, long long xs, const void* gate, long long gs, float eps, prism_dtype dt) {
  if (rows <= 0 || D <= 0 || !known(dt) || !(eps >= 0.f) || xs < D) return PRISM_ERR_INVALID_ARG;
  if (gate != nullptr && gs < D) return PRISM_ERR_INVALID_ARG;
  if (xs > LLONG_MAX / 8 / rows || gs > LLONG_MAX / 8 / rows) return PRISM_ERR_INVALID_ARG;
  if (D > kMaxWidth) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

// Whether rows fit the registers of a workgroup (2048 pieces of 16 bytes).  A longer row is read twice, a value per lane at a
// time: 218 rows of 7539 float32, gated, backward: 53 us that way, 19 in registers.
static bool norm_short(int D, prism_dtype dt) { return D * elem(dt) <= 32768; }

prism_status prism_norm_fwd(const void* x, long long x_stride, const void* residual, const float* weight,
                            const void* gate, long long gate_stride, int rows, int D, float eps, prism_dtype dt,
                            void* y, float* scales, void* h_out, hipStream_t stream) {
  const prism_status st = norm_check(rows, D, x_stride, gate, gate_stride, eps, dt);
  if (st != PRISM_OK) return st;
  if (!x || !y) return PRISM_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = x, a.xs = x_stride, a.residual = residual, a.w = weight, a.gate = gate, a.gs = gate_stride;
  a.rows = rows, a.D = D, a.eps = eps, a.y = y, a.scales = scales, a.h = h_out;
  return host::launch_norm_fwd(dt, norm_short(D, dt), a, stream);
}

// Workgroups of the backward: each sums its rows' share of dweight before the shares are joined.  Four rows or more to a
// workgroup, as long as every CU has one: a share is written and read again (1000 x 8192 bfloat16: 22 us with 256 shares, 39
// with 1000; gated 29 and 52; 2000 x 3000 float32: 21.1 with 500, 21.4 with 1024, 21.8 with 256).
static int norm_blocks(int rows, int D, prism_dtype dt) {
  const size_t pieces = ((size_t)D * elem(dt) + 15) / 16;
  const size_t at_once = pieces <= 8 ? 32 : pieces <= 16 ? 16 : pieces <= 32 ? 8 : pieces <= 256 ? 4 : 1;  // rows of a workgroup
  return (int)std::min((rows + at_once - 1) / at_once, std::max<size_t>(kCUs, std::min<size_t>(4 * kCUs, rows / 4)));
}

size_t prism_norm_bwd_workspace_bytes(int rows, int D, prism_dtype dt) {
  if (norm_check(rows, D, D, nullptr, 0, 0.f, dt) != PRISM_OK) return 0;
  Layout ly;
  ly.add((size_t)norm_blocks(rows, D, dt), (size_t)D * 4);
  return ly.ok() ? ly.total : 0;
}

prism_status prism_norm_bwd(const void* h, long long h_stride, const float* weight, const void* gate,
                            long long gate_stride, const void* dy, const void* dh_in, int rows, int D, float eps,
                            prism_dtype dt, void* dh, void* dgate, float* dweight,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const prism_status st = norm_check(rows, D, h_stride, gate, gate_stride, eps, dt);
  if (st != PRISM_OK) return st;
  if (!h || !dy || !dh || (gate != nullptr && !dgate)) return PRISM_ERR_INVALID_ARG;
  const size_t need = prism_norm_bwd_workspace_bytes(rows, D, dt);
  if (!workspace || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PRISM_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = h, a.xs = h_stride, a.w = weight, a.gate = gate, a.gs = gate_stride, a.dy = dy, a.dh_in = dh_in;
  a.rows = rows, a.D = D, a.eps = eps, a.h = dh, a.dgate = dgate;
  a.part = reinterpret_cast<float*>(workspace), a.nblk = norm_blocks(rows, D, dt), a.dw = dweight;
  return host::launch_norm_bwd(dt, norm_short(D, dt), a, stream);
}

}  // extern "C"
