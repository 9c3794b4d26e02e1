// attn_fwd.hip - launches of the attention forward (prism_attn.h)
#include "prism_attn.h"

namespace prism {
namespace host {
namespace {

size_t row_tiles(const AttnArgs& a, size_t rows, size_t each) {
  return a.starts != nullptr ? a.T * each / rows + a.S : a.B * ((a.T * each + rows - 1) / rows);
}

template <class T, int D, int NW, int BN>
prism_status many(const AttnArgs& a, hipStream_t stream) {
  using F = attn::FwdTile<T, D, NW, BN, attn::kPrompt>;
  return launch_wide<attn::fwd_kernel<T, D, NW, BN, attn::kPrompt>>((unsigned)(row_tiles(a, F::kRows, 1) * a.H), F::kThreads, F::kLds, a, stream);
}
template <class T, int D>
prism_status few(const AttnArgs& a, hipStream_t stream) {
  using F = attn::FewTile<T, D, attn::kPrompt>;
  return launch_wide<attn::few_kernel<T, D, attn::kPrompt>>((unsigned)(row_tiles(a, 32, a.H / a.G) * a.G), 256, F::kLds, a, stream);
}

// Workgroups of 128 rows, or of 256 for bfloat16 heads of 64 and 128 where there are many; else tiles of 32 rows whose keys four waves
// share.  Packed batches go by the tiles that all their tokens and sequences may take, whatever each holds: 1000 sequences of 16 tokens, 32 heads
// of 64, take 553 us in workgroups with one live wave of four or eight.  Measured at the sides of the borders, us, on rotating inputs, one length for all sequences, few rows / many rows: bfloat16 of 64: 1 x 16 x 2048 36 / 47,
// 1 x 32 x 2048 63 / 50, 4 x 16 x 256 13.5 / 12.6, 4 x 16 x 512 17.5 / 16.8; of 32: 1 x 16 x 2048 22 / 32, 1 x 32 x 2048 36 / 32; of 128:
// 1 x 16 x 2048 50 / 51, 1 x 32 x 2048 86 / 60; float32 of 64: 1 x 32 x 2048 184 / 212, 8 x 12 x 2048 485 / 447, 8 x 16 x 512 65 / 63,
// 32 x 16 x 256 87 / 71; of 128: 1 x 16 x 2048 195 / 294, 1 x 32 x 2048 384 / 327.  128 / 256 rows, bfloat16 of 128: 2 x 32 x 2048
// 114 / 88, 1 x 32 x 2048 62 / 67; of 64, four waves per SIMD each: 1 x 16 x 8192 204 / 226, 1 x 16 x 16384 658 / 615, 4 x 16 x 4096
// 178 / 172, 64 x 16 x 512 86 / 87 (128 rows with tiles of 64 keys, two waves per SIMD: 2 x 16 x 8192 349, where these take 337 / 315).
template <class T, int D>
prism_status run(const AttnArgs& a, hipStream_t s) {
  const size_t blocks = row_tiles(a, 128, 1) * a.H;
  const bool f32 = sizeof(T) == 4;
  const size_t few_most = f32 && D < 128 ? (a.T >= 1024 ? 1024 : 512) : a.T >= (f32 ? 512 : 1024) ? 320 : 192;
  if (blocks <= few_most) return few<T, D>(a, s);
  // 2^23 tiles of 32 rows, the most there are, may be as many of 256: a launch too large for eight waves each
  const bool eight_fit = row_tiles(a, 256, 1) * a.H <= kMostThreads / 512;
  if constexpr (sizeof(T) == 4) return many<T, D, 4, (D > 32 ? 32 : 64)>(a, s);
  else if constexpr (D == 128) return blocks >= 1024 && eight_fit ? many<T, D, 8, 64>(a, s) : many<T, D, 4, 64>(a, s);
  else if constexpr (D == 64) return blocks >= 2048 && a.T >= 2048 && eight_fit ? many<T, D, 8, 64>(a, s) : many<T, D, 4, 32>(a, s);
  else return many<T, D, 4, 64>(a, s);
}

}  // namespace

prism_status launch_attn_fwd(prism_dtype dt, int D, const AttnArgs& a, hipStream_t s) {
  if (dt == PRISM_BF16) return D == 32 ? run<bf16_t, 32>(a, s) : D == 64 ? run<bf16_t, 64>(a, s) : run<bf16_t, 128>(a, s);
  return D == 32 ? run<float, 32>(a, s) : D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace host
}  // namespace prism
