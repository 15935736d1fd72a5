// Checks that the host sides of the operators share: errors, types, workspaces
// and overlaps of tensors.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "layer_internal.h"
#include "muon_mi355x.h"

namespace muon {

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report(code, buf);
}
inline int ok() { return report(MUON_OK, ""); }
inline int hip_fail(hipError_t e, const char* what) { return fail(MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e)); }

inline bool dtype_ok(int32_t d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t esize(int32_t d) { return d == MUON_BF16 ? 2 : 4; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return MUON_OK;
  if (!ws) return fail(MUON_ERR_INVALID_ARG, "workspace is NULL");
  if ((uintptr_t)ws & 255) return fail(MUON_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (have < need) return fail(MUON_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, have);
  return MUON_OK;
}

// Bytes a strided set of rows reaches: rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const char* name;
  uintptr_t at;
  int64_t rows, width, stride;
};
inline Rows rows_of(const char* name, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  return {name, (uintptr_t)p, rows, cols * esize(dt), rows > 1 ? ld * esize(dt) : cols * esize(dt)};
}
// Whether two sets may share a byte.  Sets with one common stride are told
// apart by their place within it (columns of one packed buffer), others by
// their whole extent.
inline bool meet(const Rows& a, const Rows& b) {
  if (!a.at || !b.at || !a.rows || !b.rows || !a.width || !b.width) return false;
  const uintptr_t ae = a.at + (uintptr_t)((a.rows - 1) * a.stride + a.width);
  const uintptr_t be = b.at + (uintptr_t)((b.rows - 1) * b.stride + b.width);
  if (a.at >= be || b.at >= ae) return false;
  const int64_t S = a.rows > 1 ? a.stride : b.stride;
  if ((a.rows > 1 && b.rows > 1 && a.stride != b.stride) || a.width > S || b.width > S) return true;
  const int64_t d = (int64_t)((a.at >= b.at ? a.at - b.at : S - (int64_t)((b.at - a.at) % (uintptr_t)S)) % (uintptr_t)S);
  return !(d >= b.width && d + a.width <= S);
}

inline bool ranges_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  return a && b && na > 0 && nb > 0 && (uintptr_t)a < (uintptr_t)b + (uintptr_t)nb && (uintptr_t)b < (uintptr_t)a + (uintptr_t)na;
}

}  // namespace muon
