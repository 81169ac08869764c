// Checks of the arguments of the layer operators' host entry points: types,
// extents, and matrices that may not overlap.  Not part of the public ABI.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "layers_internal.h"

namespace vcoll {

inline int fail(int status, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return report_error(status, msg);
}

#define VCOLL_TRY(expr)   \
  do {                    \
    const int rc_ = expr; \
    if (rc_) return rc_;  \
  } while (0)

constexpr int64_t kMaxExtent = 0x7FFFFFFE;  // rows; tokens of a table
constexpr int64_t kMaxWidth = 1 << 30;      // columns: a chunk past the last fits 32 bits

inline int elem_size(int dtype) { return dtype == VCOLL_F32 ? 4 : dtype == VCOLL_BF16 ? 2 : 0; }

inline int check_type(int dtype, const char* what) {
  if (!elem_size(dtype)) return fail(VCOLL_ERR_INVALID_TYPE, "unknown %s %d", what, dtype);
  return VCOLL_OK;
}

inline int check_extent(int64_t v, const char* what, int64_t most = kMaxExtent) {
  if (v < 0) return fail(VCOLL_ERR_INVALID_ARG, "%s = %lld < 0", what, (long long)v);
  if (v > most)
    return fail(VCOLL_ERR_UNSUPPORTED, "%s = %lld is above %lld", what, (long long)v,
                (long long)most);
  return VCOLL_OK;
}

// One operand of a call: rows x cols elements of es bytes, ld elements apart.
struct Operand {
  const char* name;
  const void* ptr;
  int64_t rows, cols, ld;
  int es;
  bool out;
  const void* alias;  // the operand that it may coincide with, or NULL
};

inline int check_operand(const Operand& o) {
  if (o.rows == 0 || o.cols == 0) return VCOLL_OK;
  if (!o.ptr) return fail(VCOLL_ERR_INVALID_ARG, "%s is NULL", o.name);
  if ((uint64_t)o.ptr % o.es)
    return fail(VCOLL_ERR_INVALID_ARG, "%s is not aligned to the element size", o.name);
  if (o.ld < o.cols)
    return fail(VCOLL_ERR_INVALID_ARG, "%s: row stride %lld < %lld columns", o.name,
                (long long)o.ld, (long long)o.cols);
  if (o.ld > (INT64_MAX / 8 - o.cols) / o.rows)  // the byte extent must fit 64 bits
    return fail(VCOLL_ERR_INVALID_ARG, "%s: row stride %lld is out of range", o.name,
                (long long)o.ld);
  return VCOLL_OK;
}

inline bool overlap(const Operand& a, const Operand& b) {
  const uint64_t pa = (uint64_t)a.ptr, pb = (uint64_t)b.ptr;
  const uint64_t wa = (uint64_t)a.cols * a.es, wb = (uint64_t)b.cols * b.es;
  const uint64_t sa = (uint64_t)a.ld * a.es, sb = (uint64_t)b.ld * b.es;
  const uint64_t ea = pa + (uint64_t)(a.rows - 1) * sa + wa;
  const uint64_t eb = pb + (uint64_t)(b.rows - 1) * sb + wb;
  if (ea <= pb || eb <= pa) return false;
  if (sa == sb && a.rows > 1 && b.rows > 1) {  // column ranges of the same wider rows
    const uint64_t d = pb >= pa ? (pb - pa) % sa : (sa - (pa - pb) % sa) % sa;
    return d < wa || d + wb > sa;
  }
  return true;
}

// Pointers, strides, and that no output overlaps another operand.
inline int check_operands(const Operand* ops, int n) {
  for (int i = 0; i < n; ++i) VCOLL_TRY(check_operand(ops[i]));
  for (int i = 0; i < n; ++i)
    for (int k = i + 1; k < n; ++k) {
      const Operand &a = ops[i], &b = ops[k];
      if (!a.ptr || !b.ptr || !a.rows || !b.rows || !a.cols || !b.cols) continue;
      if (!a.out && !b.out) continue;
      if (a.ptr == b.ptr && a.ld == b.ld && a.es == b.es && (a.alias == b.ptr || b.alias == a.ptr))
        continue;
      if (overlap(a, b))
        return fail(VCOLL_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
    }
  return VCOLL_OK;
}

inline int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!need) return VCOLL_OK;
  if (!workspace || bytes < need)
    return fail(VCOLL_ERR_INVALID_ARG, "the workspace holds %zu bytes, %zu are needed",
                workspace ? bytes : (size_t)0, need);
  if ((uint64_t)workspace % 256)
    return fail(VCOLL_ERR_INVALID_ARG, "the workspace is not 256-byte aligned");
  return VCOLL_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace vcoll
