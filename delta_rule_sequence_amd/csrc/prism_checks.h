// prism_checks.h - argument checks and workspace layout shared by the C ABI of the state space and attention layers.
#pragma once
#include <algorithm>
#include <climits>
#include <cstddef>
#include <stdint.h>

#include "prism.h"

namespace prism {
namespace checks {

constexpr size_t kCUs = 256;     // compute units of an MI355X

inline size_t elem(prism_dtype dt) { return dt == PRISM_BF16 ? 2 : 4; }
inline bool known(prism_dtype dt) { return dt == PRISM_F32 || dt == PRISM_BF16; }
inline bool width_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

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

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Strides of a [B, H, T, width] tensor: the caller's, or dense ones.  Checks signs and that the largest offset fits
// in 63 bits.
inline bool make_strides(const prism_strides* given, int B, int H, int T, int width, prism_strides* out) {
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
inline bool rows_apart(const prism_strides& s, int B, int H, int T, int width) {
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

inline bool rows16(const void* p, const prism_strides& s, prism_dtype dt) {
  const long long e = (long long)elem(dt);
  return aligned16(p) && s.b * e % 16 == 0 && s.h * e % 16 == 0 && s.t * e % 16 == 0;
}

// Rows of the scan's tensors: on 16-byte boundaries, not overlapping, and at most 16 MB apart (a chunk's rows are
// addressed with 32-bit byte offsets).
inline bool scan_rows(const void* p, const prism_strides& s, int width, prism_dtype dt) {
  return rows16(p, s, dt) && s.t >= width && s.t * (long long)elem(dt) <= (1 << 24);
}

template <class P> P* at(void* ws, size_t off) { return reinterpret_cast<P*>(reinterpret_cast<char*>(ws) + off); }

}  // namespace checks
}  // namespace prism
