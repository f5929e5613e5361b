// qr_checks.h -- argument checks that the entry points of include/qr_layer.h and
// include/qr_f8.h share (host code).  Not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qr_internal.h"
#include "qr_layer.h"

#define QR_TRY(expr)              \
  do {                            \
    int rc_ = (expr);             \
    if (rc_ != QR_OK) return rc_; \
  } while (0)

namespace qr {
namespace checks {

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// a buffer of a call: rows of `cols` values of `elem` bytes, `ld` apart
struct Rows {
  const char* what;
  const void* p;
  size_t rows, cols, ld;
  unsigned elem, align;
  size_t bytes() const { return ((rows - 1) * ld + cols) * elem; }
};

// longest row stride: keeps every extent below 2^64 bytes, though not its end
constexpr size_t kMaxStride = (size_t)1 << 40;
constexpr size_t kMaxRows = (size_t)1 << 22;

inline int check(const Rows& r) {
  if (r.p == nullptr) return fail(QR_ERR_ARG, "%s is NULL", r.what);
  if (((uintptr_t)r.p & (r.align - 1)) != 0)
    return fail(QR_ERR_ALIGN, "%s is not %u-byte aligned", r.what, r.align);
  if (r.ld < r.cols || r.ld > kMaxStride)
    return fail(QR_ERR_ARG, "%s: row stride %zu for rows of %zu", r.what, r.ld, r.cols);
  return QR_OK;
}

// Extents that meet, but for rows of one stride in bytes that lie between one
// another (columns of one buffer).
inline bool overlap(const Rows& a, const Rows& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y ? x - y >= b.bytes() : y - x >= a.bytes()) return false;
  const size_t stride = a.ld * a.elem;
  if (stride != b.ld * b.elem) return true;
  const size_t at = y >= x ? (y - x) % stride : stride - 1 - (x - y - 1) % stride;
  return at < a.cols * a.elem || at + b.cols * b.elem > stride;
}

inline int check_apart(const Rows& a, const Rows& b) {
  if (overlap(a, b)) return fail(QR_ERR_ARG, "%s overlaps %s", a.what, b.what);
  return QR_OK;
}

inline int check_dtype(int dtype, bool cast) {
  if (dtype != QR_FP16 && dtype != QR_BF16 && !(cast && dtype == QR_BF16_VIA_FP16))
    return fail(QR_ERR_UNSUPPORTED, "unsupported dtype %d", dtype);
  return QR_OK;
}

inline int check_rows(size_t M, size_t d) {
  if (d == 0 || d > QR_MAX_ROW)
    return fail(QR_ERR_SIZE, "d = %zu outside 1..%zu", d, QR_MAX_ROW);
  if (M > kMaxRows) return fail(QR_ERR_SIZE, "M = %zu exceeds %zu", M, kMaxRows);
  return QR_OK;
}

}  // namespace checks
}  // namespace qr
