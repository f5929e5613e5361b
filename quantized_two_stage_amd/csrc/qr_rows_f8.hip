// qr_rows_f8.hip -- gfx950 kernels of the row operators of include/qr_f8.h: the
// root-mean-square norm with the residual's addition and the gated activation,
// both to E4M3FN codes with a scale for each block of 128 values.
//
// A lane holds a vector of 8 values, so a block is 16 lanes: its largest
// magnitude is four exchanges inside a row of 16 lanes, and its codes leave at
// once.  The norm's factor r is common to the row and enters the scales (and y)
// alone, so nothing but them waits for the row's sum of squares.
//
// All values are held in binary32; they are rounded once, to h (which enters the
// sum of squares as rounded: it is what the next layer adds to), y and the codes.
//
// Bound by HBM, short calls by the launch and one read's latency.  Measured (cold
// inputs; a copy reaches 5.2 TB/s):
//   norm, 8192 x 8192 bf16 with h and y   112 us, 5.4 TB/s; without y 91, 5.2 TB/s
//   norm, 1 x 8192                        3.9 us (an empty launch with one read 2.2)
//   norm, 3000 x 5003 fp16                31.5 us, 3.35 TB/s (3000 x 5000 27.5): rows that
//                                         start at any even byte are read across lines
//   activation, 8192 x 4096 bf16          34.7 us, 4.9 TB/s
//   activation, 32768 x 1024 bf16         36.4 us, 4.6 TB/s; 333 x 1000 3.3 us
#include "qr_f8.h"
#include "qr_f8_internal.h"
#include "qr_rows_device.h"

namespace qr {
namespace {

// the largest of 16 lanes' v, NaN if there is one
__device__ __forceinline__ float block_max(float v) {
  const auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf,
                                        0xf, true));
  };
  v = __builtin_elementwise_maximum(v, dpp(v, std::integral_constant<int, 0xb1>{}));   // lane ^ 1
  v = __builtin_elementwise_maximum(v, dpp(v, std::integral_constant<int, 0x4e>{}));   // lane ^ 2
  v = __builtin_elementwise_maximum(v, dpp(v, std::integral_constant<int, 0x141>{}));  // 4 of 8
  return __builtin_elementwise_maximum(v, dpp(v, std::integral_constant<int, 0x140>{}));
}

// f = 448 / a (0: the block has no codes) and the block's scale a / 448
__device__ __forceinline__ float block_scale(float a, float& scale) {
  constexpr float kTiny = 0x1p-119f, kInf = __builtin_inff();
  const bool fine = a < kInf, use = fine && a >= kTiny;       // false for NaN
  scale = use ? a / 448.0f : fine ? 0.0f : __builtin_nanf("");
  return use ? 448.0f / a : 0.0f;
}

// The code of value i where the quotient 448*u/a lies between the neighbouring
// codes lo and hi, or on one of them: 448*u and the codes' middle times a are
// exact in 64 bits (27 and 29 bits), so this is the exact quotient's.
template <int I>
__device__ __forceinline__ uint32_t nearer(float u, float a, uint32_t lo, uint32_t hi) {
  const float x = e4m3_dec<I % 4>(lo), y = e4m3_dec<I % 4>(hi);
  const double mid = 0.5 * (double)(__builtin_fabsf(x) + __builtin_fabsf(y)) * (double)a;
  const double v = 448.0 * (double)__builtin_fabsf(u);
  const uint32_t cl = lo >> (8 * (I % 4)) & 0xffu, ch = hi >> (8 * (I % 4)) & 0xffu;
  return v > mid || (v == mid && (ch & 1u) == 0u) ? ch : cl;
}

// 8 codes.  The quotient is u*f but for three roundings, so it lies between u*f
// less and plus 2^-21 of it: where both round to the same code that is the
// quotient's, elsewhere (about one value in 100000) the exact products decide.
__device__ __forceinline__ u32x2 code_f8(const float (&u)[8], float f, float a) {
  u32x2 w = {0u, 0u};
  if (f != 0.0f) {
    const float fl = f * (1.0f - 0x1p-21f), fh = f * (1.0f + 0x1p-21f);
    u32x2 h;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const float* v = u + 4 * k;
      w[k] = e4m3_pack2(v[2] * fl, v[3] * fl, e4m3_pack2(v[0] * fl, v[1] * fl, 0u, false), true);
      h[k] = e4m3_pack2(v[2] * fh, v[3] * fh, e4m3_pack2(v[0] * fh, v[1] * fh, 0u, false), true);
    }
    if (w.x != h.x || w.y != h.y) {
      const auto both = [&](auto i) {
        constexpr int I = decltype(i)::value;
        return nearer<I>(u[I], a, w[I / 4], h[I / 4]) << (8 * (I % 4));
      };
      const uint32_t x = both(std::integral_constant<int, 0>{}) | both(std::integral_constant<int, 1>{}) |
                         both(std::integral_constant<int, 2>{}) | both(std::integral_constant<int, 3>{});
      w.y = both(std::integral_constant<int, 4>{}) | both(std::integral_constant<int, 5>{}) |
            both(std::integral_constant<int, 6>{}) | both(std::integral_constant<int, 7>{});
      w.x = x;
    }
  }
  return w;
}

__device__ __forceinline__ float largest(const float (&u)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) a = max_abs(a, u[i]);
  return a;
}
template <int E>
__device__ __forceinline__ void store_f8(uint8_t* p, u32x2 w, uint32_t n) {
  store_codes<E>(reinterpret_cast<int8_t*>(p), w, n);
}
// 8 values times r in 16 bits
template <int D, int E>
__device__ __forceinline__ void store_values(uint8_t* p, const float (&u)[8], float r, uint32_t n) {
  u32x4 v;
#pragma unroll
  for (int k = 0; k < 4; k++) v[k] = st16x2<D>(u[2 * k] * r, u[2 * k + 1] * r);
  store_vec<E>(p, v, n);
}

// the sum over a workgroup's waves, at most 16; entries of waves that are not
// there hold 0
__device__ __forceinline__ float waves_sum(float ss, float (&lds)[16]) {
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = ss;
  __syncthreads();
  ss = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; w++) ss += lds[w];
  return ss;
}
__device__ __forceinline__ void clear(float (&lds)[16]) {
  if (threadIdx.x >= blockDim.x / 64 && threadIdx.x < 16) lds[threadIdx.x] = 0.0f;
}

constexpr uint32_t kRowsOfAGroup = 4;              // where a row has one wave

template <class Op>
__device__ __forceinline__ float row_factor(const Op& op, float ss, uint32_t d) {
  return ss < __builtin_inff() ? op.factor(ss, d) : __builtin_nanf("");
}

// The norm of a row of at most 8*V values a lane, held in registers.  Wave: a
// wave to a row, kRowsOfAGroup of them to a workgroup; else the workgroup's
// lanes (whole waves) to a row.
template <int D, bool Wave, int V, int E>
__global__ __launch_bounds__(Wave ? 64 * kRowsOfAGroup : 1024) void k_norm_f8(Norm<D, -1> op,
                                                                              F8Out o) {
  __shared__ float lds[16];
  const uint32_t R = Wave ? kRowsOfAGroup : 1, T = Wave ? 64 : blockDim.x;
  const uint32_t t = Wave ? threadIdx.x % 64 : threadIdx.x;
  if (!Wave) clear(lds);
  for (uint32_t m = blockIdx.x * R + (Wave ? threadIdx.x / 64 : 0); m < o.M; m += gridDim.x * R) {
    const auto row = op.row(m, o.d);
    uint8_t* const q = o.q + (size_t)m * o.ldq;
    constexpr int B = V < 2 ? V : 2;       // vectors on their way at a time
    float u[V][8], scale[V];
    float ss = 0.0f;
#pragma unroll
    for (int j0 = 0; j0 < V; j0 += B) {
      typename Norm<D, -1>::Raw raw[B];
#pragma unroll
      for (int j = 0; j < B; j++) {
        const uint32_t vec = t + T * (j0 + j), i0 = 8 * vec;
        if (i0 < o.d) op.template load<E>(row, vec, o.d - i0 < 8 ? o.d - i0 : 8, raw[j]);
      }
#pragma unroll
      for (int j = 0; j < B; j++) {
        const uint32_t vec = t + T * (j0 + j), i0 = 8 * vec, n = o.d - i0 < 8 ? o.d - i0 : 8;
        float(&v)[8] = u[j0 + j];
        float a = 0.0f;
        if (i0 < o.d) {
          op.template values<E>(row, vec, n, raw[j], v, ss);
          a = largest(v);
        }
        a = block_max(a);
        const float f = block_scale(a, scale[j0 + j]);
        if (i0 < o.d) store_f8<E>(q + i0, code_f8(v, f, a), n);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    ss = wave_sum(ss);
    if (!Wave) ss = waves_sum(ss, lds);
    const float r = row_factor(op, ss, o.d);
    float* const s = o.scales + (size_t)m * o.lds;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const uint32_t vec = t + T * j, i0 = 8 * vec;
      if (i0 < o.d && vec % 16 == 0) s[vec / 16] = scale[j] * r;
      if (o.y && i0 < o.d)
        store_values<D, E>(o.y + 2 * ((size_t)m * o.ldy + i0), u[j], r,
                           o.d - i0 < 8 ? o.d - i0 : 8);
    }
    if (!Wave && m + gridDim.x < o.M) __syncthreads();         // lds is used again
  }
}

// Rows of any length: a second pass multiplies the scales by r, each lane those
// that it has written, and reads the row again for y.
template <int D, int T>
__global__ __launch_bounds__(T) void k_norm_f8_long(Norm<D, -1> op, F8Out o) {
  __shared__ float lds[16];
  clear(lds);
  for (uint32_t m = blockIdx.x; m < o.M; m += gridDim.x) {
    const auto row = op.row(m, o.d);
    uint8_t* const q = o.q + (size_t)m * o.ldq;
    float* const s = o.scales + (size_t)m * o.lds;
    float ss = 0.0f;
    for (uint32_t v0 = 0; 8 * v0 < o.d; v0 += T) {
      const uint32_t vec = v0 + threadIdx.x, i0 = 8 * vec, n = o.d - i0 < 8 ? o.d - i0 : 8;
      float u[8], a = 0.0f, scale;
      if (i0 < o.d) {
        typename Norm<D, -1>::Raw raw;
        op.template load<kAny>(row, vec, n, raw);
        op.template values<kAny>(row, vec, n, raw, u, ss);
        a = largest(u);
      }
      a = block_max(a);
      const float f = block_scale(a, scale);
      if (i0 < o.d) store_f8<kAny>(q + i0, code_f8(u, f, a), n);
      if (i0 < o.d && vec % 16 == 0) s[vec / 16] = scale;
    }
    ss = waves_sum(wave_sum(ss), lds);
    const float r = row_factor(op, ss, o.d);
    for (uint32_t vec = threadIdx.x; 8 * vec < o.d; vec += T) {
      const uint32_t i0 = 8 * vec, n = o.d - i0 < 8 ? o.d - i0 : 8;
      if (vec % 16 == 0) s[vec / 16] *= r;
      if (o.y) {
        float u[8];
        op.template again<kAny>(row, vec, n, u);
        store_values<D, kAny>(o.y + 2 * ((size_t)m * o.ldy + i0), u, r, n);
      }
    }
    if (m + gridDim.x < o.M) __syncthreads();
  }
}

// The activation: no step crosses a block, so rows and workgroups do not belong
// together: lane l of the grid takes vector l mod `lanes` of row l / lanes, with
// `lanes` the row's vectors filled up to whole blocks.
template <int D, int E>
__global__ __launch_bounds__(256) void k_silu_f8(Silu<D> op, F8Out o, uint32_t lanes) {
  const uint32_t l = blockIdx.x * 256 + threadIdx.x, m = l / lanes, vec = l - m * lanes;
  const uint32_t i0 = 8 * vec, n = o.d - i0 < 8 ? o.d - i0 : 8;
  const bool in = m < o.M && i0 < o.d;
  float u[8], a = 0.0f, unused = 0.0f;
  if (in) {
    const auto row = op.row(m, o.d);
    typename Silu<D>::Raw raw;
    op.template load<E>(row, vec, n, raw);
    op.template values<E>(row, vec, n, raw, u, unused);
    a = largest(u);
  }
  a = block_max(a);
  float scale;
  const float f = block_scale(a, scale);
  if (in) {
    store_f8<E>(o.q + (size_t)m * o.ldq + i0, code_f8(u, f, a), n);
    if (vec % 16 == 0) o.scales[(size_t)m * o.lds + vec / 16] = scale;
  }
}

constexpr uint32_t kMaxGroups = 1u << 21;         // times 1024 lanes: below 2^32

template <int D, bool Wave, int V, int E>
hipError_t norm_in_registers(const Norm<D, -1>& op, const F8Out& o, hipStream_t st) {
  constexpr uint32_t R = Wave ? kRowsOfAGroup : 1;
  const uint32_t g = (o.M + R - 1) / R, lanes = (o.d + 8 * V - 1) / (8 * V);
  k_norm_f8<D, Wave, V, E><<<g < kMaxGroups ? g : kMaxGroups,
                             Wave ? 64 * R : (lanes + 63) / 64 * 64, 0, st>>>(op, o);
  return hipGetLastError();
}
template <int D, int T>
hipError_t norm_twice(const Norm<D, -1>& op, const F8Out& o, hipStream_t st) {
  k_norm_f8_long<D, T><<<o.M < kMaxGroups ? o.M : kMaxGroups, T, 0, st>>>(op, o);
  return hipGetLastError();
}
// lanes to a row as for the norm in 8-bit integers
template <int D, int E>
hipError_t norm_by_length(const Norm<D, -1>& op, const F8Out& o, hipStream_t st) {
  if (o.d <= 512) return norm_in_registers<D, true, 1, E>(op, o, st);
  if (o.d <= 8192) return norm_in_registers<D, false, 1, E>(op, o, st);
  if (o.d <= 16384) return norm_in_registers<D, false, 2, E>(op, o, st);
  return norm_twice<D, 1024>(op, o, st);
}
template <int D>
hipError_t norm_f8(const NormArgs& a, const F8Out& o, hipStream_t st) {
  const Norm<D, -1> op{a};
  if (o.d < 8) return norm_twice<D, 64>(op, o, st);
  return o.d % 8 != 0 ? norm_by_length<D, kShort>(op, o, st) : norm_by_length<D, kWhole>(op, o, st);
}

template <int D>
hipError_t silu_f8(const uint8_t* gu, size_t ldg, const F8Out& all, hipStream_t st) {
  const uint32_t lanes = (all.d + kF8Block - 1) / kF8Block * 16;
  const uint32_t most = (1u << 31) / lanes;       // rows of a launch: lanes are counted in 32 bits
  for (uint32_t m = 0; m < all.M; m += most) {
    F8Out o = all;
    o.M = all.M - m < most ? all.M - m : most;
    o.q += (size_t)m * o.ldq;
    o.scales += (size_t)m * o.lds;
    const Silu<D> op{gu + 2 * (size_t)m * ldg, ldg};
    const uint32_t groups = (uint32_t)(((uint64_t)o.M * lanes + 255) / 256);
    if (o.d < 8) k_silu_f8<D, kAny><<<groups, 256, 0, st>>>(op, o, lanes);
    else if (o.d % 8 != 0) k_silu_f8<D, kShort><<<groups, 256, 0, st>>>(op, o, lanes);
    else k_silu_f8<D, kWhole><<<groups, 256, 0, st>>>(op, o, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_norm_f8(int dtype, const NormArgs& a, const F8Out& o, hipStream_t st) {
  return dtype == kF16 ? norm_f8<kF16>(a, o, st) : norm_f8<kBF16>(a, o, st);
}

hipError_t launch_silu_f8(int dtype, const uint8_t* gu, size_t ldg, const F8Out& o,
                          hipStream_t st) {
  return dtype == kF16 ? silu_f8<kF16>(gu, ldg, o, st) : silu_f8<kBF16>(gu, ldg, o, st);
}

}  // namespace qr
