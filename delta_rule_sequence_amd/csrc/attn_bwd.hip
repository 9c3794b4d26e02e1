// attn_bwd.hip - launches of the attention backward (prism_attn_bwd.h)
#include "prism_attn_bwd.h"

namespace prism {
namespace host {
namespace {

unsigned row_tiles(const AttnArgs& a, int rows) {
  return (unsigned)(a.starts != nullptr ? a.T / rows + a.S : (size_t)a.B * ((a.T + rows - 1) / rows));
}

// The pass by queries and the one by keys (waves that own rows, waves that share them, rows of a tile, ahead).
template <class T, int D, int OW, int SW, int BN, bool AHEAD>
prism_status by_queries(const AttnArgs& a, hipStream_t s) {
  using F = attn::Pass<T, D, OW, SW, BN, AHEAD>;
  return launch_wide<attn::dq_kernel<T, D, OW, SW, BN, AHEAD>>(row_tiles(a, F::kOwn) * a.H, F::kThreads, F::kLds, a, s);
}
template <class T, int D, int OW, int SW, int BN, bool AHEAD>
prism_status by_keys(const AttnArgs& a, hipStream_t s) {
  using F = attn::Pass<T, D, OW, SW, BN, AHEAD>;
  const prism_status st =
      launch_wide<attn::dkv_kernel<T, D, OW, SW, BN, AHEAD>>(row_tiles(a, F::kOwn) * a.G * a.splits, F::kThreads, F::kLds, a, s);
  if (st != PRISM_OK || a.splits == 1) return st;
  const size_t rows = 2 * (size_t)a.B * a.G * a.T, per = 256 / (D / 4);
  attn::sum_kernel<T, D><<<dim3((unsigned)((rows + per - 1) / per)), 256, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? PRISM_OK : PRISM_ERR_HIP;
}

// Where workgroups of 128 rows are few, each owns 32 (64 of wide float32 heads) and four (two) waves share them.  Measured at
// the sides of the borders, us, small / not: bfloat16 of 64: 1 x 16 x 1024 47 / 53, 1 x 16 x 2048 120 / 88, 1 x 8 x 1024 33 / 49,
// 4 x 16 x 256 34 / 30; of 32: 1 x 16 x 2048 53 / 69, 1 x 32 x 2048 83 / 82, 4 x 16 x 256 18 / 22, 4 x 16 x 512 32 / 32;
// float32 of 64: 1 x 16 x 2048 365 / 392, 1 x 32 x 2048 722 / 638, 4 x 16 x 256 61 / 66, 4 x 16 x 512 150 / 125; of 128:
// 1 x 16 x 2048 554 / 741, 1 x 32 x 2048 1074 / 1076.
template <class T, int D>
prism_status run(const AttnArgs& a, hipStream_t s) {
  const bool f32 = sizeof(T) == 4, long_rows = a.T >= 1024;
  const size_t small_most = f32 ? (D == 128 ? 512 : long_rows ? 256 : 160) : D == 32 ? (long_rows ? 384 : 192) : long_rows ? 128 : 96;
  const size_t blocks = (size_t)row_tiles(a, 128) * a.H;
  const bool small = blocks <= small_most || (!f32 && blocks > kMostThreads / 512);   // or more than a launch of eight waves each holds
  prism_status st;
  if constexpr (sizeof(T) == 4) {
    constexpr int SW = D == 128 ? 2 : 4;                              // 128 rows of 128 float32 twice do not fit
    if (small) st = by_queries<T, D, 4 / SW, SW, 32 * SW, false>(a, s);
    else st = by_queries<T, D, 4, 1, 32, false>(a, s);
    if (st != PRISM_OK) return st;
    return small ? by_keys<T, D, 4 / SW, SW, 32 * SW, false>(a, s) : by_keys<T, D, 2, 2, 64, false>(a, s);
  } else {
    if (small) st = by_queries<T, D, 1, 4, 128, false>(a, s);
    else if constexpr (D == 128) st = by_queries<T, D, 8, 1, 64, true>(a, s);
    else st = by_queries<T, D, 4, 1, 64, true>(a, s);
    if (st != PRISM_OK) return st;
    if (small) return by_keys<T, D, 1, 4, 128, false>(a, s);
    if constexpr (D == 128) return by_keys<T, D, 4, 1, 64, false>(a, s);
    else return by_keys<T, D, 4, 2, 128, true>(a, s);
  }
}

}  // namespace

prism_status launch_attn_bwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return D == 32 ? run<bf16_t, 32>(a, s) : D == 64 ? run<bf16_t, 64>(a, s) : run<bf16_t, 128>(a, s);
  return D == 32 ? run<float, 32>(a, s) : D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace host
}  // namespace prism
