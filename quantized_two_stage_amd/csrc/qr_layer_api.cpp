// qr_layer_api.cpp -- the extern "C" entry points declared in
// include/qr_layer.h: argument checks, done before anything is launched, and
// the launches of qr_rows.hip and qr_gemm.hip.  No state is kept.
#include <math.h>
#include <stdint.h>

#include "qr_internal.h"
#include "qr_layer.h"
#include "qr_layer_internal.h"

namespace {

using qr::fail;
using qr::hip_status;
using qr::ok;

#define QR_TRY(expr)              \
  do {                            \
    int rc_ = (expr);             \
    if (rc_ != QR_OK) return rc_; \
  } while (0)

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// a buffer of a call: rows of `cols` values of `elem` bytes, `ld` apart
struct Rows {
  const char* what;
  const void* p;
  size_t rows, cols, ld;
  unsigned elem, align;
  size_t bytes() const { return ((rows - 1) * ld + cols) * elem; }
};

// longest row stride: keeps every extent far below 2^64 bytes
constexpr size_t kMaxStride = (size_t)1 << 40;
constexpr size_t kMaxRows = (size_t)1 << 22;

int check(const Rows& r) {
  if (r.p == nullptr) return fail(QR_ERR_ARG, "%s is NULL", r.what);
  if (((uintptr_t)r.p & (r.align - 1)) != 0)
    return fail(QR_ERR_ALIGN, "%s is not %u-byte aligned", r.what, r.align);
  if (r.ld < r.cols || r.ld > kMaxStride)
    return fail(QR_ERR_ARG, "%s: row stride %zu for rows of %zu", r.what, r.ld, r.cols);
  return QR_OK;
}

// Extents that meet, but for rows of one stride in bytes that lie between one
// another (columns of one buffer).
bool overlap(const Rows& a, const Rows& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y + b.bytes() || y >= x + a.bytes()) return false;
  const size_t stride = a.ld * a.elem;
  if (stride != b.ld * b.elem) return true;
  const size_t at = y >= x ? (y - x) % stride : stride - 1 - (x - y - 1) % stride;
  return at < a.cols * a.elem || at + b.cols * b.elem > stride;
}

int check_apart(const Rows& a, const Rows& b) {
  if (overlap(a, b)) return fail(QR_ERR_ARG, "%s overlaps %s", a.what, b.what);
  return QR_OK;
}

int check_dtype(int dtype, bool cast) {
  if (dtype != QR_FP16 && dtype != QR_BF16 && !(cast && dtype == QR_BF16_VIA_FP16))
    return fail(QR_ERR_UNSUPPORTED, "unsupported dtype %d", dtype);
  return QR_OK;
}

int check_rows(size_t M, size_t d) {
  if (d == 0 || d > QR_MAX_ROW)
    return fail(QR_ERR_SIZE, "d = %zu outside 1..%zu", d, QR_MAX_ROW);
  if (M > kMaxRows) return fail(QR_ERR_SIZE, "M = %zu exceeds %zu", M, kMaxRows);
  return QR_OK;
}

// the norm's arguments other than x
int check_norm(const Rows& x, const Rows& res, const Rows& w, float eps, const Rows& h,
               const Rows& q, const Rows& s) {
  if (!(eps > 0.0f) || isinf(eps)) return fail(QR_ERR_ARG, "eps must be positive and finite");
  QR_TRY(check(w));
  QR_TRY(check(q));
  QR_TRY(check(s));
  QR_TRY(check_apart(q, x));
  QR_TRY(check_apart(q, w));
  QR_TRY(check_apart(q, s));
  QR_TRY(check_apart(s, x));
  QR_TRY(check_apart(s, w));
  if (res.p != nullptr) {
    QR_TRY(check(res));
    QR_TRY(check_apart(q, res));
    QR_TRY(check_apart(s, res));
  }
  if (h.p != nullptr) {
    QR_TRY(check(h));
    QR_TRY(check_apart(h, x));
    QR_TRY(check_apart(h, w));
    QR_TRY(check_apart(h, q));
    QR_TRY(check_apart(h, s));
    if (res.p != nullptr && !(h.p == res.p && (h.ld == res.ld || h.rows == 1)))
      QR_TRY(check_apart(h, res));
  }
  return QR_OK;
}

}  // namespace

extern "C" {

int qr_add_rmsnorm_q8(qr_dtype dtype, const void* x, size_t ldx, const void* residual, size_t ldr,
                      const void* weight, float eps, size_t M, size_t d, void* h, size_t ldh,
                      int8_t* q, size_t ldq, float* scales, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_rows(M, d));
  if (M == 0) return ok();
  const Rows rx{"x", x, M, d, ldx, 2, 2}, rr{"residual", residual, M, d, ldr, 2, 2},
      rw{"weight", weight, 1, d, d, 2, 2}, rh{"h", h, M, d, ldh, 2, 2},
      rq{"q", q, M, d, ldq, 1, 1}, rs{"scales", scales, 1, M, M, 4, 4};
  QR_TRY(check(rx));
  if ((residual == nullptr) != (h == nullptr))
    return fail(QR_ERR_ARG, "residual and h come together");
  QR_TRY(check_norm(rx, rr, rw, eps, rh, rq, rs));
  const qr::NormArgs a{static_cast<const uint8_t*>(x), ldx, 0, 0,
                       static_cast<const uint8_t*>(residual), ldr,
                       static_cast<const uint8_t*>(weight), static_cast<uint8_t*>(h), ldh, eps};
  const qr::RowsOut o{q, ldq, scales, (uint32_t)M, (uint32_t)d};
  (void)hipGetLastError();
  return hip_status(qr::launch_norm(-1, dtype, a, o, as_stream(stream)), "norm launch");
}

int qr_gather_add_rmsnorm_q8(qr_codec codec, qr_dtype dtype, const void* wire,
                             const void* residual, size_t ldr, const void* weight, float eps,
                             size_t M, size_t d, void* h, size_t ldh, int8_t* q, size_t ldq,
                             float* scales, void* stream) {
  if (!qr::codec_valid(codec)) return fail(QR_ERR_UNSUPPORTED, "unsupported codec %d", codec);
  QR_TRY(check_dtype(dtype, true));
  QR_TRY(check_rows(M, d));
  if (d % 8 != 0) return fail(QR_ERR_SIZE, "d = %zu is not a multiple of 8", d);
  if (M == 0) return ok();
  if (M * d > QR_MAX_BYTES / 2)
    return fail(QR_ERR_SIZE, "M*d = %zu exceeds QR_MAX_BYTES", M * d);
  const qr::Layout L = qr::make_layout(codec, M * d);
  const Rows rx{"wire", wire, 1, L.total, L.total, 1, 16},
      rr{"residual", residual, M, d, ldr, 2, 2}, rw{"weight", weight, 1, d, d, 2, 2},
      rh{"h", h, M, d, ldh, 2, 2}, rq{"q", q, M, d, ldq, 1, 1},
      rs{"scales", scales, 1, M, M, 4, 4};
  QR_TRY(check(rx));
  if (h == nullptr) return fail(QR_ERR_ARG, "h is NULL");
  QR_TRY(check_norm(rx, rr, rw, eps, rh, rq, rs));
  const qr::NormArgs a{static_cast<const uint8_t*>(wire), 0, L.off_s, L.off_z,
                       static_cast<const uint8_t*>(residual), ldr,
                       static_cast<const uint8_t*>(weight), static_cast<uint8_t*>(h), ldh, eps};
  const qr::RowsOut o{q, ldq, scales, (uint32_t)M, (uint32_t)d};
  (void)hipGetLastError();
  return hip_status(qr::launch_norm(codec, dtype, a, o, as_stream(stream)), "norm launch");
}

int qr_silu_mul_q8(qr_dtype dtype, const void* gu, size_t ldg, size_t M, size_t d, int8_t* q,
                   size_t ldq, float* scales, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_rows(M, d));
  if (M == 0) return ok();
  const Rows rg{"gu", gu, M, 2 * d, ldg, 2, 2}, rq{"q", q, M, d, ldq, 1, 1},
      rs{"scales", scales, 1, M, M, 4, 4};
  QR_TRY(check(rg));
  QR_TRY(check(rq));
  QR_TRY(check(rs));
  QR_TRY(check_apart(rq, rg));
  QR_TRY(check_apart(rs, rg));
  QR_TRY(check_apart(rq, rs));
  const qr::RowsOut o{q, ldq, scales, (uint32_t)M, (uint32_t)d};
  (void)hipGetLastError();
  return hip_status(qr::launch_silu(dtype, static_cast<const uint8_t*>(gu), ldg, o,
                                    as_stream(stream)),
                    "activation launch");
}

// every size keeps its partial sums in LDS
size_t qr_gemm_i8_workspace_bytes(size_t, size_t, size_t) { return 0; }

int qr_gemm_i8(qr_dtype dtype, const int8_t* a, size_t lda, const float* sa, const int8_t* b,
               size_t ldb, const float* sb, const void* bias, size_t M, size_t N, size_t K,
               void* c, size_t ldc, void* /*workspace*/, size_t /*ws_bytes*/, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  if (K == 0 || K > QR_MAX_ROW)
    return fail(QR_ERR_SIZE, "K = %zu outside 1..%zu", K, QR_MAX_ROW);
  if (N == 0 || N > kMaxRows) return fail(QR_ERR_SIZE, "N = %zu outside 1..%zu", N, kMaxRows);
  if (M > kMaxRows) return fail(QR_ERR_SIZE, "M = %zu exceeds %zu", M, kMaxRows);
  if (M == 0) return ok();
  const Rows ra{"a", a, M, K, lda, 1, 16}, rb{"b", b, N, K, ldb, 1, 16},
      rsa{"sa", sa, 1, M, M, 4, 4}, rsb{"sb", sb, 1, N, N, 4, 4},
      rbias{"bias", bias, 1, N, N, 2, 2}, rc{"c", c, M, N, ldc, 2, 2};
  QR_TRY(check(ra));
  QR_TRY(check(rb));
  for (const Rows* r : {&ra, &rb}) {
    if (r->ld % 16 != 0)
      return fail(QR_ERR_ALIGN, "%s: row stride %zu is not a multiple of 16", r->what, r->ld);
    if (r->ld >= (size_t)1 << 23)
      return fail(QR_ERR_SIZE, "%s: row stride %zu is 2^23 or more", r->what, r->ld);
  }
  QR_TRY(check(rsa));
  QR_TRY(check(rsb));
  QR_TRY(check(rc));
  QR_TRY(check_apart(rc, ra));
  QR_TRY(check_apart(rc, rb));
  QR_TRY(check_apart(rc, rsa));
  QR_TRY(check_apart(rc, rsb));
  if (bias != nullptr) {
    QR_TRY(check(rbias));
    QR_TRY(check_apart(rc, rbias));
  }
  const qr::GemmArgs g{a, lda, sa, b, ldb, sb, static_cast<const uint8_t*>(bias),
                       static_cast<uint8_t*>(c), ldc, (uint32_t)M, (uint32_t)N, (uint32_t)K};
  (void)hipGetLastError();
  return hip_status(qr::launch_gemm(dtype, g, as_stream(stream)), "product launch");
}

}  // extern "C"
