// Host-side argument checks shared by the C entry points.
#pragma once

#include <math.h>

#include "common.hpp"

namespace mao {

#define MAO_FAIL(code, ...)       \
  do {                            \
    ::mao::set_error(__VA_ARGS__); \
    return (code);                \
  } while (0)

inline size_t dtype_size(int dt) { return dt == MAO_BF16 ? 2 : 4; }
inline bool dtype_ok(int dt) { return dt == MAO_F32 || dt == MAO_BF16; }
inline bool finite(float x) { return isfinite(x) != 0; }

// Bytes a buffer touches: the interval [lo, hi), and for a strided matrix
// view whose every row starts at the same offset modulo the row pitch (one
// matrix, or a batch stride that is a multiple of the pitch) the pitch and the
// bytes each row covers, so that column views of one wider buffer (a fused
// QKV weight split into its logical matrices) are told apart exactly.
struct Range {
  uintptr_t lo, hi;
  uint64_t pitch = 0, span = 0;  // pitch 0: no row structure known
};

inline Range mat_range(const void* p, int64_t count, int64_t rows, int64_t cols, int64_t ld,
                int64_t stride, size_t es) {
  const int64_t last = (count - 1) * stride + (rows - 1) * ld + cols;
  Range r{(uintptr_t)p, (uintptr_t)p + (uintptr_t)(last * (int64_t)es)};
  if (count == 1 || stride % ld == 0) {
    r.pitch = (uint64_t)(ld * (int64_t)es);
    r.span = (uint64_t)(cols * (int64_t)es);
  }
  return r;
}

inline bool overlap(Range a, Range b) {
  if (!(a.lo < b.hi && b.lo < a.hi)) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  // rows of a cover [a.lo mod pitch, + a.span) on the circle of one pitch,
  // rows of b [b.lo mod pitch, + b.span): disjoint arcs never share a byte
  const uint64_t P = a.pitch;
  const uint64_t d = ((uint64_t)(b.lo % P) + P - (uint64_t)(a.lo % P)) % P;
  return !(d >= a.span && d + b.span <= P);
}

inline mao_status check_mat(const char* name, const void* data, int64_t rows, int64_t cols, int64_t ld,
                     int dtype, bool f32_only) {
  if (!data) MAO_FAIL(MAO_E_NULL, "%s: NULL data", name);
  if (rows < 1 || cols < 1) MAO_FAIL(MAO_E_SHAPE, "%s: rows=%lld cols=%lld", name, (long long)rows, (long long)cols);
  if (rows > (1 << 20) || cols > (1 << 20)) MAO_FAIL(MAO_E_SHAPE, "%s: dimension above 2^20", name);
  if (!dtype_ok(dtype) || (f32_only && dtype != MAO_F32)) MAO_FAIL(MAO_E_DTYPE, "%s: unsupported dtype %d", name, dtype);
  if (ld < cols || ld % 8 != 0) MAO_FAIL(MAO_E_LAYOUT, "%s: ld=%lld (cols=%lld) must be >= cols and a multiple of 8", name, (long long)ld, (long long)cols);
  if ((uintptr_t)data % 16 != 0) MAO_FAIL(MAO_E_LAYOUT, "%s: data not 16-byte aligned", name);
  return MAO_OK;
}

inline mao_status check_workspace(void* ws, size_t have, size_t need) {
  if (need == 0) return MAO_OK;
  if (!ws) MAO_FAIL(MAO_E_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if ((uintptr_t)ws % 256 != 0) MAO_FAIL(MAO_E_WORKSPACE, "workspace not 256-byte aligned");
  if (have < need) MAO_FAIL(MAO_E_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  return MAO_OK;
}

}  // namespace mao
