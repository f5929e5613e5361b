// qr_f8_api.cpp -- the extern "C" entry points declared in include/qr_f8.h:
// argument checks, done before anything is launched, and the launches of
// qr_rows_f8.hip, qr_gemm_f8.hip and qr_experts.hip.  No state is kept.
#include <initializer_list>
#include <math.h>
#include <stdint.h>

#include "qr_checks.h"
#include "qr_f8.h"
#include "qr_f8_internal.h"
#include "qr_gemm_f8_tiles.h"

namespace {

using namespace qr::checks;
using qr::fail;
using qr::hip_status;
using qr::ok;

constexpr size_t blocks_of(size_t n) { return (n + qr::kF8Block - 1) / qr::kF8Block; }

// `out` apart from every one of `others` that is given
int check_apart_from(const Rows& out, std::initializer_list<const Rows*> others) {
  for (const Rows* o : others)
    if (o->p != nullptr) QR_TRY(check_apart(out, *o));
  return QR_OK;
}

// the arguments of a product whose a has `rows` rows and whose c has M
int check_product(const Rows& ra, const Rows& rsa, const Rows& rb, const Rows& rsb) {
  QR_TRY(check(ra));
  QR_TRY(check(rsa));
  QR_TRY(check(rb));
  QR_TRY(check(rsb));
  for (const Rows* r : {&ra, &rb}) {
    if (r->ld % 16 != 0)
      return fail(QR_ERR_ALIGN, "%s: row stride %zu is not a multiple of 16", r->what, r->ld);
    if (r->ld >= (size_t)1 << 23)
      return fail(QR_ERR_SIZE, "%s: row stride %zu is 2^23 or more", r->what, r->ld);
  }
  if (rsa.ld % 4 != 0)
    return fail(QR_ERR_ALIGN, "sa: row stride %zu is not a multiple of 4", rsa.ld);
  if (rsa.ld > (size_t)1 << 20)
    return fail(QR_ERR_SIZE, "sa: row stride %zu exceeds 2^20", rsa.ld);
  return QR_OK;
}

int check_product_sizes(size_t M, size_t N, size_t K) {
  if (K == 0 || K > QR_MAX_ROW)
    return fail(QR_ERR_SIZE, "K = %zu outside 1..%zu", K, QR_MAX_ROW);
  if (N == 0 || N > kMaxRows) return fail(QR_ERR_SIZE, "N = %zu outside 1..%zu", N, kMaxRows);
  if (M > kMaxRows) return fail(QR_ERR_SIZE, "M = %zu exceeds %zu", M, kMaxRows);
  return QR_OK;
}

int launch_product(int dtype, const qr::F8Args& g, void* stream) {
  const int tile = qr::choose_f8_tile(g.M, g.N, g.K, g.E);
  if (tile < 0)
    return fail(QR_ERR_SIZE, "M = %u, N = %u, E = %u: more tiles than a launch holds", g.M, g.N, g.E);
  (void)hipGetLastError();
  return hip_status(qr::launch_gemm_f8(tile, dtype, g, as_stream(stream)), "product launch");
}

int check_chosen(size_t T, size_t k) {
  if (k == 0 || k > QR_MAX_CHOSEN)
    return fail(QR_ERR_SIZE, "k = %zu outside 1..%zu", k, QR_MAX_CHOSEN);
  if (T > kMaxRows) return fail(QR_ERR_SIZE, "T = %zu exceeds %zu", T, kMaxRows);
  return QR_OK;
}

}  // namespace

extern "C" {

int qr_add_rmsnorm_f8(qr_dtype dtype, const void* x, size_t ldx, const void* residual, size_t ldr,
                      const void* weight, float eps, size_t M, size_t d, void* h, size_t ldh,
                      void* y, size_t ldy, uint8_t* q, size_t ldq, float* scales, size_t lds,
                      void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_rows(M, d));
  if (M == 0) return ok();
  const Rows rx{"x", x, M, d, ldx, 2, 2}, rr{"residual", residual, M, d, ldr, 2, 2},
      rw{"weight", weight, 1, d, d, 2, 2}, rh{"h", h, M, d, ldh, 2, 2}, ry{"y", y, M, d, ldy, 2, 2},
      rq{"q", q, M, d, ldq, 1, 1}, rs{"scales", scales, M, blocks_of(d), lds, 4, 4};
  QR_TRY(check(rx));
  if ((residual == nullptr) != (h == nullptr))
    return fail(QR_ERR_ARG, "residual and h come together");
  if (!(eps > 0.0f) || isinf(eps)) return fail(QR_ERR_ARG, "eps must be positive and finite");
  QR_TRY(check(rw));
  QR_TRY(check(rq));
  QR_TRY(check(rs));
  for (const Rows* r : {&rr, &rh, &ry})
    if (r->p != nullptr) QR_TRY(check(*r));
  QR_TRY(check_apart_from(rq, {&rx, &rr, &rw, &rh, &ry, &rs}));
  QR_TRY(check_apart_from(rs, {&rx, &rr, &rw, &rh, &ry}));
  if (y != nullptr) QR_TRY(check_apart_from(ry, {&rx, &rr, &rw, &rh}));
  if (h != nullptr) {
    QR_TRY(check_apart_from(rh, {&rx, &rw}));
    if (!(h == residual && (ldh == ldr || M == 1))) QR_TRY(check_apart(rh, rr));
  }
  const qr::NormArgs a{static_cast<const uint8_t*>(x), ldx, 0, 0,
                       static_cast<const uint8_t*>(residual), ldr,
                       static_cast<const uint8_t*>(weight), static_cast<uint8_t*>(h), ldh, eps};
  const qr::F8Out o{q, ldq, scales, lds, static_cast<uint8_t*>(y), ldy, (uint32_t)M, (uint32_t)d};
  (void)hipGetLastError();
  return hip_status(qr::launch_norm_f8(dtype, a, o, as_stream(stream)), "norm launch");
}

int qr_silu_mul_f8(qr_dtype dtype, const void* gu, size_t ldg, size_t M, size_t d, uint8_t* q,
                   size_t ldq, float* scales, size_t lds, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_rows(M, d));
  if (M == 0) return ok();
  const Rows rg{"gu", gu, M, 2 * d, ldg, 2, 2}, rq{"q", q, M, d, ldq, 1, 1},
      rs{"scales", scales, M, blocks_of(d), lds, 4, 4};
  QR_TRY(check(rg));
  QR_TRY(check(rq));
  QR_TRY(check(rs));
  QR_TRY(check_apart_from(rq, {&rg, &rs}));
  QR_TRY(check_apart(rs, rg));
  const qr::F8Out o{q, ldq, scales, lds, nullptr, 0, (uint32_t)M, (uint32_t)d};
  (void)hipGetLastError();
  return hip_status(qr::launch_silu_f8(dtype, static_cast<const uint8_t*>(gu), ldg, o,
                                       as_stream(stream)),
                    "activation launch");
}

int qr_gemm_f8(qr_dtype dtype, const uint8_t* a, size_t lda, const float* sa, size_t ldsa,
               const uint8_t* b, size_t ldb, const float* sb, size_t ldsb, const void* bias,
               size_t M, size_t N, size_t K, void* c, size_t ldc, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_product_sizes(M, N, K));
  if (M == 0) return ok();
  const size_t kb = blocks_of(K);
  const Rows ra{"a", a, M, K, lda, 1, 16}, rsa{"sa", sa, M, kb, ldsa, 4, 16},
      rb{"b", b, N, K, ldb, 1, 16}, rsb{"sb", sb, blocks_of(N), kb, ldsb, 4, 4},
      rbias{"bias", bias, 1, N, N, 2, 2}, rc{"c", c, M, N, ldc, 2, 2};
  QR_TRY(check_product(ra, rsa, rb, rsb));
  if (bias != nullptr) QR_TRY(check(rbias));
  QR_TRY(check(rc));
  QR_TRY(check_apart_from(rc, {&ra, &rsa, &rb, &rsb, &rbias}));
  const qr::F8Args g{a, lda, sa, ldsa, b, ldb, sb, ldsb, static_cast<const uint8_t*>(bias),
                     static_cast<uint8_t*>(c), ldc, (uint32_t)M, (uint32_t)N, (uint32_t)K,
                     0, (uint32_t)M, nullptr, nullptr, 0, 0, 0};
  return launch_product(dtype, g, stream);
}

int qr_gemm_f8_grouped(qr_dtype dtype, const uint8_t* a, size_t lda, const float* sa, size_t ldsa,
                       const int32_t* rows, size_t tokens, const uint8_t* b, size_t ldb, size_t gb,
                       const float* sb, size_t ldsb, size_t gsb, const void* bias, size_t ldbias,
                       const int32_t* offsets, size_t E, size_t M, size_t N, size_t K, void* c,
                       size_t ldc, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_product_sizes(M, N, K));
  if (E == 0 || E > QR_MAX_EXPERTS)
    return fail(QR_ERR_SIZE, "E = %zu outside 1..%zu", E, QR_MAX_EXPERTS);
  if (M == 0) return ok();
  if (rows == nullptr) tokens = M;
  if (tokens == 0 || tokens > kMaxRows)
    return fail(QR_ERR_SIZE, "tokens = %zu outside 1..%zu", tokens, kMaxRows);
  const size_t kb = blocks_of(K), nb = blocks_of(N);
  const Rows ra{"a", a, tokens, K, lda, 1, 16}, rsa{"sa", sa, tokens, kb, ldsa, 4, 16},
      rb{"b", b, N, K, ldb, 1, 16}, rsb{"sb", sb, nb, kb, ldsb, 4, 4};
  QR_TRY(check_product(ra, rsa, rb, rsb));
  if (gb % 16 != 0) return fail(QR_ERR_ALIGN, "gb = %zu is not a multiple of 16", gb);
  // the experts' matrices as rows that do not meet
  const Rows rbs{"b", b, E, rb.bytes(), E == 1 ? rb.bytes() : gb, 1, 16},
      rsbs{"sb", sb, E, rsb.bytes() / 4, E == 1 ? rsb.bytes() / 4 : gsb, 4, 4},
      rbias{"bias", bias, E, N, E == 1 ? N : ldbias, 2, 2},
      roff{"offsets", offsets, 1, E + 1, E + 1, 4, 4}, rrows{"rows", rows, 1, M, M, 4, 4},
      rc{"c", c, M, N, ldc, 2, 2};
  QR_TRY(check(rbs));
  QR_TRY(check(rsbs));
  QR_TRY(check(roff));
  if (bias != nullptr) QR_TRY(check(rbias));
  if (rows != nullptr) {
    QR_TRY(check(rrows));
    constexpr size_t kReach = ((size_t)1 << 32) - ((size_t)1 << 18);
    if (tokens * lda >= kReach || 4 * tokens * ldsa >= kReach)
      return fail(QR_ERR_SIZE, "tokens * lda = %zu or 4 * tokens * ldsa = %zu too large for rows",
                  tokens * lda, 4 * tokens * ldsa);
  }
  QR_TRY(check(rc));
  QR_TRY(check_apart_from(rc, {&ra, &rsa, &rbs, &rsbs, &rbias, &roff, &rrows}));
  const qr::F8Args g{a, lda, sa, ldsa, b, ldb, sb, ldsb, static_cast<const uint8_t*>(bias),
                     static_cast<uint8_t*>(c), ldc, (uint32_t)M, (uint32_t)N, (uint32_t)K,
                     (uint32_t)E, (uint32_t)tokens, offsets, rows, gb, gsb, ldbias};
  return launch_product(dtype, g, stream);
}

size_t qr_route_workspace_bytes(size_t T, size_t E, size_t k) {
  if (E == 0 || E > QR_MAX_EXPERTS || k == 0 || k > QR_MAX_CHOSEN || T > kMaxRows) return 0;
  return qr::route_workspace_bytes((uint32_t)T, (uint32_t)E);
}

int qr_route(int dtype, const void* logits, size_t ldl, size_t T, size_t E, size_t k,
             int renormalize, float* weights, int32_t* experts, int32_t* offsets, int32_t* rows,
             int32_t* place, void* workspace, size_t ws_bytes, void* stream) {
  if (dtype != QR_FP16 && dtype != QR_BF16 && dtype != QR_FP32)
    return fail(QR_ERR_UNSUPPORTED, "unsupported dtype %d", dtype);
  if (E == 0 || E > QR_MAX_EXPERTS)
    return fail(QR_ERR_SIZE, "E = %zu outside 1..%zu", E, QR_MAX_EXPERTS);
  QR_TRY(check_chosen(T, k));
  if (k > E) return fail(QR_ERR_SIZE, "k = %zu of E = %zu experts", k, E);
  if (T * k > kMaxRows) return fail(QR_ERR_SIZE, "T*k = %zu exceeds %zu", T * k, kMaxRows);
  const unsigned elem = dtype == QR_FP32 ? 4 : 2;
  const size_t need = qr_route_workspace_bytes(T, E, k), n = T * k;
  const Rows rl{"logits", logits, T, E, ldl, elem, elem}, rw{"weights", weights, 1, n, n, 4, 4},
      re{"experts", experts, 1, n, n, 4, 4}, ro{"offsets", offsets, 1, E + 1, E + 1, 4, 4},
      rr{"rows", rows, 1, n, n, 4, 4}, rp{"place", place, 1, n, n, 4, 4},
      rws{"workspace", workspace, 1, need, need, 1, 16};
  QR_TRY(check(ro));
  if (T != 0) {
    for (const Rows* r : {&rl, &rw, &re, &rr, &rp}) QR_TRY(check(*r));
    if (need != 0) {
      if (ws_bytes < need)
        return fail(QR_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
      QR_TRY(check(rws));
      QR_TRY(check_apart_from(rws, {&rl, &rw, &re, &ro, &rr, &rp}));
    }
    QR_TRY(check_apart_from(rw, {&rl, &re, &ro, &rr, &rp}));
    QR_TRY(check_apart_from(re, {&rl, &ro, &rr, &rp}));
    QR_TRY(check_apart_from(ro, {&rl, &rr, &rp}));
    QR_TRY(check_apart_from(rr, {&rl, &rp}));
    QR_TRY(check_apart(rp, rl));
  }
  const qr::RouteArgs a{static_cast<const uint8_t*>(logits), ldl, (uint32_t)T, (uint32_t)E,
                        (uint32_t)k, renormalize != 0, weights, experts, offsets, rows, place,
                        static_cast<uint16_t*>(workspace)};
  (void)hipGetLastError();
  return hip_status(qr::launch_route(dtype, a, as_stream(stream)), "route launch");
}

int qr_combine(qr_dtype dtype, const void* c, size_t ldc, size_t R, const int32_t* place,
               const float* weights, size_t T, size_t k, size_t d, const void* addend, size_t lda,
               void* y, size_t ldy, void* stream) {
  QR_TRY(check_dtype(dtype, false));
  QR_TRY(check_rows(T, d));
  QR_TRY(check_chosen(T, k));
  if (R > kMaxRows) return fail(QR_ERR_SIZE, "R = %zu exceeds %zu", R, kMaxRows);
  if (T == 0) return ok();
  if (R == 0) return fail(QR_ERR_SIZE, "R = 0 rows for T = %zu", T);
  const size_t n = T * k;
  const Rows rc{"c", c, R, d, ldc, 2, 2}, rp{"place", place, 1, n, n, 4, 4},
      rw{"weights", weights, 1, n, n, 4, 4}, ra{"addend", addend, T, d, lda, 2, 2},
      ry{"y", y, T, d, ldy, 2, 2};
  QR_TRY(check(rc));
  QR_TRY(check(rp));
  QR_TRY(check(rw));
  if (addend != nullptr) QR_TRY(check(ra));
  QR_TRY(check(ry));
  QR_TRY(check_apart_from(ry, {&rc, &rp, &rw}));
  if (addend != nullptr && !(y == addend && (ldy == lda || T == 1))) QR_TRY(check_apart(ry, ra));
  const qr::CombineArgs a{static_cast<const uint8_t*>(c), ldc, (uint32_t)R, place, weights,
                          (uint32_t)T, (uint32_t)k, (uint32_t)d,
                          static_cast<const uint8_t*>(addend), lda, static_cast<uint8_t*>(y), ldy};
  (void)hipGetLastError();
  return hip_status(qr::launch_combine(dtype, a, as_stream(stream)), "combine launch");
}

}  // extern "C"
