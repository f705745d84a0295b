// Argument checks shared by the entry points of include/flare_ops.h.
#pragma once

#include <cstdint>

#include "flare_ops.h"
#include "host_internal.h"

namespace flare {

constexpr int64_t kMaxInt = 2147483647;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool row_width_ok(int64_t D) { return D == 16 || D == 32 || D == 64 || D == 128; }

// Strides of a [B][H][N][D] tensor of bf16 rows: every row starts on a
// 16-byte boundary; a dimension of size one has no stride (0 is stored); rows
// of an output do not share memory through a zero stride.
inline flare_status fill_strides(long (&out)[3], const void* base, const int64_t* s, int64_t B, int64_t H, int64_t N,
                                 int64_t D, bool is_output) {
  const int64_t n[3] = {B, H, N};
  if (!aligned16(base)) return FLARE_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    out[i] = n[i] == 1 ? 0 : static_cast<long>(s[i]);
    if (n[i] == 1) continue;
    if (s[i] % 8 != 0) return FLARE_ERR_ALIGN;
    if (s[i] < 0 || (s[i] != 0 && s[i] < D) || (is_output && s[i] == 0)) return FLARE_ERR_SHAPE;
    if (s[i] > (int64_t(1) << 38)) return FLARE_ERR_UNSUPPORTED;
  }
  return FLARE_OK;
}

}  // namespace flare
