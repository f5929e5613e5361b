// qr_rows.hip -- gfx950 kernels of the row operators of include/qr_layer.h:
// root-mean-square norm with the residual's addition (from 16-bit rows or
// from a wire image) and the gated activation, both to 8-bit codes with one
// scale a row.
//
// One pass over HBM.  A workgroup (or, for short rows, a wave) holds a whole
// row in registers: it loads its vectors of 8 values, writes h, keeps the
// values u that are to be coded, reduces the sum of squares and the largest
// magnitude across the row once, and codes from the registers.  That a single
// reduction is enough rests on the norm's factor r being common to the row:
// u_i*r*127/(a*r) = u_i*127/a, so the codes need the maximum a of u = h*weight
// alone, and r enters the scale only.
//
// HBM bounds long batches: 8192 rows of 8192 (norm, bf16) take 82 to 96 us, 4.9
// to 5.7 TB/s (a large copy reaches 5.2); 4096 rows of 8192 from asymmetric
// 4-bit wire codes 40 to 45 us, 4.2 to 4.7 TB/s (48 under the cast option); the
// activation of 8192 rows of 4096 30 to 32 us, 5.3 to 5.7 TB/s.  Single rows are bound by the latency of a launch, of
// one read and of the reduction: 3.6 us at 8192 values.
#include "qr_rows_device.h"

namespace qr {
namespace {

// 8 codes: round-half-even(127 * u / a) as u*f + 1.5*2^23, one rounding, f = 127/a
// rounded.  f's rounding moves u*f by at most 127 * 2^-24, so a value within 2^-17
// of a tie (one in 65000) is rounded from the quotient in 64 bits: that is
// off by less than 2^-44, and the exact one is a tie or at least 2^-33 away from
// one (u and a have 24 bits each), so rounded to multiples of 2^-36 it is a tie
// where the exact one is.  f = 0 marks a row without codes.
__device__ __forceinline__ u32x2 code8(const float (&u)[8], float f, float a) {
  u32x2 w = {0u, 0u};
  if (f != 0.0f) {
    constexpr float kMagic = 0x1.8p23f, kNear = 0.5f - 0x1p-17f;
    float m[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      m[i] = __builtin_fmaf(u[i], f, kMagic);
      far = max_abs(far, __builtin_fmaf(u[i], f, -(m[i] - kMagic)));
    }
    if (far > kNear) {
      constexpr double kGrid = 0x1.8p16;
      const double exact_f = 127.0 / (double)a;
#pragma unroll
      for (int i = 0; i < 8; i++)
        m[i] = (float)__builtin_rint((double)u[i] * exact_f + kGrid - kGrid) + kMagic;
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const auto bits = [&](int i) { return __builtin_bit_cast(uint32_t, m[4 * k + i]); };
      w[k] = __builtin_amdgcn_perm(bits(1), bits(0), 0x0c0c0400u) |
             __builtin_amdgcn_perm(bits(3), bits(2), 0x04000c0cu);
    }
  }
  return w;
}

// f = 127 / a (0: the row has no codes) and the row's scale
template <class Op>
__device__ __forceinline__ float row_scale(const Op& op, float ss, float a, uint32_t d,
                                           float& scale) {
  constexpr float kTiny = 0x1p-119f, kInf = __builtin_inff();
  const float r = op.factor(ss, d);
  const bool fine = a < kInf && (!Op::kNorm || ss < kInf);    // false for NaN
  const bool use = fine && a >= kTiny;
  scale = use ? a / 127.0f * r : fine ? 0.0f : __builtin_nanf("");      // a * r may overflow
  return use ? 127.0f / a : 0.0f;
}

constexpr uint32_t kRowsOfAGroup = 4;              // where a row has one wave

// A row of at most 8*V values a lane, held in registers.  Wave: a wave to a
// row, kRowsOfAGroup of them to a workgroup; else the workgroup's lanes to a row.
template <class Op, bool Wave, int V, int E>
__global__ __launch_bounds__(Wave ? 64 * kRowsOfAGroup : 1024) void k_rows(Op op, RowsOut o) {
  __shared__ Joined lds;
  const uint32_t R = Wave ? kRowsOfAGroup : 1, T = Wave ? 64 : blockDim.x;
  const uint32_t t = Wave ? threadIdx.x % 64 : threadIdx.x;
  if (!Wave) clear(lds);
  for (uint32_t m = blockIdx.x * R + (Wave ? threadIdx.x / 64 : 0); m < o.M; m += gridDim.x * R) {
    const auto row = op.row(m, o.d);
    constexpr int B = V < 2 ? V : 2;       // vectors on their way at a time
    float u[V][8];
    float ss = 0.0f, a = 0.0f;
#pragma unroll
    for (int j0 = 0; j0 < V; j0 += B) {
      typename Op::Raw raw[B];
#pragma unroll
      for (int j = 0; j < B; j++) {
        const uint32_t vec = t + T * (j0 + j), i0 = 8 * vec;
        if (i0 < o.d) op.template load<E>(row, vec, o.d - i0 < 8 ? o.d - i0 : 8, raw[j]);
      }
#pragma unroll
      for (int j = 0; j < B; j++) {
        const uint32_t vec = t + T * (j0 + j), i0 = 8 * vec;
        if (i0 < o.d) {
          op.template values<E>(row, vec, o.d - i0 < 8 ? o.d - i0 : 8, raw[j], u[j0 + j], ss);
#pragma unroll
          for (int i = 0; i < 8; i++) a = max_abs(a, u[j0 + j][i]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (Op::kNorm) ss = wave_sum(ss);
    a = wave_max(a);
    if (!Wave) waves_reduce<Op::kNorm>(ss, a, lds);
    float scale;
    const float f = row_scale(op, ss, a, o.d, scale);
    int8_t* q = o.q + (size_t)m * o.ldq;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const uint32_t i0 = 8 * (t + T * j);
      if (i0 < o.d) store_codes<E>(q + i0, code8(u[j], f, a), o.d - i0 < 8 ? o.d - i0 : 8);
    }
    if (t == 0) o.scales[m] = scale;
    if (!Wave && m + gridDim.x < o.M) __syncthreads();         // lds is used again
  }
}

// rows of any length: a second pass reads the row again to code it (each lane
// what it has itself written or read)
template <class Op, int T>
__global__ __launch_bounds__(T) void k_rows_long(Op op, RowsOut o) {
  __shared__ Joined lds;
  clear(lds);
  for (uint32_t m = blockIdx.x; m < o.M; m += gridDim.x) {
    const auto row = op.row(m, o.d);
    float ss = 0.0f, a = 0.0f;
    for (uint32_t vec = threadIdx.x; 8 * vec < o.d; vec += T) {
      const uint32_t n = o.d - 8 * vec < 8 ? o.d - 8 * vec : 8;
      typename Op::Raw raw;
      float u[8];
      op.template load<kAny>(row, vec, n, raw);
      op.template values<kAny>(row, vec, n, raw, u, ss);
#pragma unroll
      for (int i = 0; i < 8; i++) a = max_abs(a, u[i]);
    }
    if (Op::kNorm) ss = wave_sum(ss);
    a = wave_max(a);
    waves_reduce<Op::kNorm>(ss, a, lds);
    float scale;
    const float f = row_scale(op, ss, a, o.d, scale);
    int8_t* q = o.q + (size_t)m * o.ldq;
    for (uint32_t vec = threadIdx.x; 8 * vec < o.d; vec += T) {
      const uint32_t n = o.d - 8 * vec < 8 ? o.d - 8 * vec : 8;
      float u[8];
      op.template again<kAny>(row, vec, n, u);
      store_codes<kAny>(q + 8 * vec, code8(u, f, a), n);
    }
    if (threadIdx.x == 0) o.scales[m] = scale;
    if (m + gridDim.x < o.M) __syncthreads();
  }
}

constexpr uint32_t kMaxGroups = 1u << 21;         // times 1024 lanes: below 2^32

template <class Op, bool Wave, int V, int E>
hipError_t rows_in_registers(const Op& op, const RowsOut& o, hipStream_t st) {
  constexpr uint32_t R = Wave ? kRowsOfAGroup : 1;
  const uint32_t g = (o.M + R - 1) / R, lanes = (o.d + 8 * V - 1) / (8 * V);
  k_rows<Op, Wave, V, E><<<g < kMaxGroups ? g : kMaxGroups, Wave ? 64 * R : (lanes + 63) / 64 * 64,
                           0, st>>>(op, o);
  return hipGetLastError();
}
template <class Op, int T>
hipError_t rows_twice(const Op& op, const RowsOut& o, hipStream_t st) {
  k_rows_long<Op, T><<<o.M < kMaxGroups ? o.M : kMaxGroups, T, 0, st>>>(op, o);
  return hipGetLastError();
}

// One vector to a lane wherever a workgroup has the lanes, and no more waves
// than the row needs: the loads of a row are all on their way at once, few
// registers are held, and many waves share a CU.  The norm from 16-bit rows,
// us, when this was chosen: 8192 rows of 8192 with 1024 lanes x 1 vector 89,
// 512 x 2 88, 256 x 4 98, 128 x 8 117; of 4096 with 512 x 1 45, 256 x 2 48,
// 1024 x 1 56; one row of 8192 3.4, 3.4, 4.2, 5.9; 1024 rows of 5003 with 640
// lanes 14.4, with 1024 lanes 19.9 (exact codes have added 0.3 to 3 us since).
// Rows that are whole vectors apart from the others: the former with the
// latter's loads take 113 instead of 98 (256 x 4).  Lengths of 16385 to 32768 hold
// four vectors a lane, in the 128 registers that 1024 lanes have: 500 rows of
// 20000 take 22.7, of 20003 25.6, of 30000 29.9, of 30001 33.4.
template <class Op, int E>
hipError_t rows_by_length(const Op& op, const RowsOut& o, hipStream_t st) {
  if (o.d <= 512) return rows_in_registers<Op, true, 1, E>(op, o, st);
  if (o.d <= 8192) return rows_in_registers<Op, false, 1, E>(op, o, st);
  if (o.d <= 16384) return rows_in_registers<Op, false, 2, E>(op, o, st);
  if (o.d <= 32768) return rows_in_registers<Op, false, 4, E>(op, o, st);
  return rows_twice<Op, 1024>(op, o, st);
}
template <class Op>
hipError_t launch_rows(const Op& op, const RowsOut& o, hipStream_t st) {
  if constexpr (!Op::kWire) {            // a wire image's rows are whole vectors
    if (o.d < 8) return rows_twice<Op, 64>(op, o, st);
    if (o.d % 8 != 0) return rows_by_length<Op, kShort>(op, o, st);
  }
  return rows_by_length<Op, kWhole>(op, o, st);
}

template <int D>
hipError_t launch_wire(int codec, const NormArgs& a, const RowsOut& o, hipStream_t st) {
  switch (codec) {
    case kFP: return launch_rows(Norm<D, kFP>{a}, o, st);
    case kQ8: return launch_rows(Norm<D, kQ8>{a}, o, st);
    case kQ6: return launch_rows(Norm<D, kQ6>{a}, o, st);
    case kQ4: return launch_rows(Norm<D, kQ4>{a}, o, st);
    case kFP8: return launch_rows(Norm<D, kFP8>{a}, o, st);
    case kQ8A: return launch_rows(Norm<D, kQ8A>{a}, o, st);
    case kQ6A: return launch_rows(Norm<D, kQ6A>{a}, o, st);
    default: return launch_rows(Norm<D, kQ4A>{a}, o, st);
  }
}

}  // namespace

hipError_t launch_norm(int codec, int dtype, const NormArgs& a, const RowsOut& o,
                       hipStream_t st) {
  if (codec < 0)
    return dtype == kF16 ? launch_rows(Norm<kF16, -1>{a}, o, st)
                         : launch_rows(Norm<kBF16, -1>{a}, o, st);
  switch (dtype) {
    case kF16: return launch_wire<kF16>(codec, a, o, st);
    case kBF16: return launch_wire<kBF16>(codec, a, o, st);
    default: return launch_wire<kBF16H>(codec, a, o, st);
  }
}

hipError_t launch_silu(int dtype, const uint8_t* gu, size_t ldg, const RowsOut& o,
                       hipStream_t st) {
  return dtype == kF16 ? launch_rows(Silu<kF16>{gu, ldg}, o, st)
                       : launch_rows(Silu<kBF16>{gu, ldg}, o, st);
}

}  // namespace qr
