/*
 * qr_layer.h -- C ABI of the operators that run between two allreduces in a
 * tensor-parallel transformer layer, in 8-bit integers, for MI355X (gfx950).
 *
 * The allreduce of qr.h ends a row-parallel matrix product; what follows it
 * on every rank is
 *   qr_gather_add_rmsnorm_q8  the allreduce's reduced wire image dequantized
 *                             (stage 2), added to the residual, normalised by
 *                             its root mean square, in 8-bit codes;
 *   qr_add_rmsnorm_q8         the same from a 16-bit buffer;
 *   qr_gemm_i8                the next matrix product, on 8-bit codes;
 *   qr_silu_mul_q8            the gated activation between two products, in
 *                             8-bit codes.
 * All are for inference; none has a gradient.
 *
 * 8-bit rows.  A matrix of M rows ("tokens") of d values is held as M rows of
 * int8 codes and M binary32 scales; row m stands for code * scales[m].  The
 * codes of a row u (binary32 values) are
 *     a = max |u_i|;  code_i = round-half-even(127 * u_i / a)
 * of the exact quotient, so |code_i| <= 127 and the largest value has code
 * +-127.  A row with a < 2^-119 (where 127 / a would overflow; all zeros among
 * them) has codes 0 and scale 0.  A row that holds
 * a NaN or an infinity has codes 0 and scale NaN, so that every product with
 * it is NaN.
 *
 * Conventions, beside those of qr.h (caller-owned device memory, `stream`,
 * checks on the host before any launch, negative QR_ERR_* codes and
 * qr_last_error(), thread safety):
 *   - Matrices are row-major with a row stride ("ld...", in elements, at
 *     least the row's length); elements past a row's end are never written.
 *     Rows of 16-bit values may start at any element (2-byte alignment).
 *   - dtype is QR_FP16 or QR_BF16 (qr_gather_add_rmsnorm_q8 also takes
 *     QR_BF16_VIA_FP16) and is the type of every 16-bit buffer of a call.
 *   - M and N are at most 2^22 and row strides at most 2^40 elements (those of
 *     qr_gemm_i8's codes less, see there); QR_ERR_SIZE and QR_ERR_ARG above.
 *   - M == 0 is a batch without tokens: the call returns QR_OK and launches
 *     nothing (pointers may be NULL).
 *   - Outputs must not overlap inputs or each other, except where a function
 *     says so.  Matrices whose rows lie between one another may share a buffer
 *     if their strides are the same number of bytes (columns of one buffer).
 */
#ifndef QR_LAYER_H
#define QR_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "qr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* longest row of the row operators, and longest sum of qr_gemm_i8: up to
 * 2^17 - 1 products of two codes cannot overflow 32 bits. */
#define QR_MAX_ROW ((size_t)131071)

/* h = round_to_dtype(x + residual) (the sum in binary32), the residual stream
 * after this layer's addition; then codes and scales of
 *     h_i * weight_i * r,   r = 1 / sqrt(mean(h^2) + eps).
 * The codes are those of u_i = h_i * weight_i (exact in binary32), since r
 * is common to the row and cancels in them; scales[m] = a / 127 * r.  The
 * sum of squares is held in binary32; a row where it overflows counts as
 * holding an infinity.
 *   x         M x d, row stride ldx
 *   residual  M x d, row stride ldr; NULL (with h NULL): h = x, not written
 *   weight    d values
 *   eps       > 0, finite
 *   h         M x d, row stride ldh; may be `residual` itself (the same
 *             pointer and stride: updated in place), else apart from it
 *   q         M x d codes, row stride ldq
 *   scales    M values, 4-byte aligned
 * d in 1..QR_MAX_ROW. */
int qr_add_rmsnorm_q8(qr_dtype dtype, const void* x, size_t ldx, const void* residual,
                      size_t ldr, const void* weight, float eps, size_t M, size_t d,
                      void* h, size_t ldh, int8_t* q, size_t ldq, float* scales,
                      void* stream);

/* qr_add_rmsnorm_q8 with x = the values of a wire image of M*d elements (row
 * m holds elements [m*d, (m+1)*d)), as qr_dequantize would write them: the
 * same h, codes and scales bit for bit, without writing x.  d must be a
 * multiple of 8 and M*d at most QR_MAX_BYTES / 2; wire 16-byte aligned.
 * residual may be NULL (h = x); h is always written. */
int qr_gather_add_rmsnorm_q8(qr_codec codec, qr_dtype dtype, const void* wire,
                             const void* residual, size_t ldr, const void* weight,
                             float eps, size_t M, size_t d, void* h, size_t ldh, int8_t* q,
                             size_t ldq, float* scales, void* stream);

/* Codes and scales of v_i = g_i / (1 + exp(-g_i)) * u_i, where row m of gu (row
 * stride ldg >= 2d) holds the d gate values g and then the d up values u.  v is
 * held in binary32, within 16 * 2^-24 of its value for every finite g and u
 * (gates where exp(-g) passes the largest binary32 among them); a v that itself
 * passes it counts as an infinity.  d in 1..QR_MAX_ROW. */
int qr_silu_mul_q8(qr_dtype dtype, const void* gu, size_t ldg, size_t M, size_t d, int8_t* q,
                   size_t ldq, float* scales, void* stream);

/* c[m][n] = round_to_dtype(f32(sum_k a[m][k] * b[n][k]) * (sa[m] * sb[n]) + bias[n]):
 * the sum exact in 32-bit integers, the rest in binary32 in this order.
 *   a, sa     M x K codes, row stride lda, and M scales (the tokens)
 *   b, sb     N x K codes, row stride ldb, and N scales (the weights, a row
 *             for each output channel)
 *   bias      N values of dtype, or NULL
 *   c         M x N, row stride ldc
 * K in 1..QR_MAX_ROW, N >= 1.  Codes take all 256 values.  a and b must be
 * 16-byte aligned, lda and ldb multiples of 16 below 2^23: rows are read in
 * pieces of 16 bytes, so the bytes of a row up to the next multiple of 16
 * past K must be readable (the last row's too); what they hold does not
 * matter.  workspace: device memory of at least
 * qr_gemm_i8_workspace_bytes(M, N, K) bytes.  That is 0 for every size in this
 * version (partial sums stay on chip), so NULL will do and nothing is read
 * from or written to it. */
int qr_gemm_i8(qr_dtype dtype, const int8_t* a, size_t lda, const float* sa, const int8_t* b,
               size_t ldb, const float* sb, const void* bias, size_t M, size_t N, size_t K,
               void* c, size_t ldc, void* workspace, size_t ws_bytes, void* stream);

/* Workspace of qr_gemm_i8 for these sizes (0: none). */
size_t qr_gemm_i8_workspace_bytes(size_t M, size_t N, size_t K);

#ifdef __cplusplus
}
#endif

#endif /* QR_LAYER_H */
