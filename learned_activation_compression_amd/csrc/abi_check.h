// Checks of arguments that several entry points make before anything is enqueued.
#pragma once

#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "../../include/mapl.h"

namespace mapl {

constexpr int64_t kMaxElems = int64_t(1) << 36;

inline bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

inline bool elem_misaligned(mapl_dtype dt, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p, dt == MAPL_BF16 ? 2 : 4)) return true;
  return false;
}

// rows, widths and gate rows that the norm kernels take
inline int check_norm_shape(int64_t N, int64_t d, int64_t gate_rows) {
  if (N < 0 || N > INT32_MAX || d < 1 || d > 8192 || gate_rows < 0) return MAPL_ERR_SHAPE;
  if (gate_rows > 0 && N % gate_rows != 0) return MAPL_ERR_SHAPE;
  if (gate_rows > N && N > 0) return MAPL_ERR_SHAPE;
  return MAPL_OK;
}

inline int check_norm_scalars(float res_scale, float eps, double p) {
  // a subnormal eps would count as zero in the reciprocal root of an empty row
  if (!std::isfinite(res_scale) || !(eps >= FLT_MIN) || !std::isfinite(eps) || !(p >= 0.0 && p <= 1.0)) return MAPL_ERR_ARG;
  return MAPL_OK;
}

inline int check_fp8_shape(int64_t a, int64_t b) {
  constexpr int64_t top = int64_t(1) << 27;  // a grid has fewer than 2^32 threads
  if (a < 0 || b < 0 || a > top || b > top || (b > 0 && a > kMaxElems / b)) return MAPL_ERR_SHAPE;
  return MAPL_OK;
}

}  // namespace mapl
