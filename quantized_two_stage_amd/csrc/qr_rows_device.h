// qr_rows_device.h -- what the row kernels share (qr_rows.hip, qr_rows_f8.hip):
// vectors of 8 values at any address, the norm's and the activation's values,
// and reductions over a wave and a workgroup.  Not part of the ABI.
#pragma once

#include <type_traits>

#include "qr.h"
#include "qr_device.h"
#include "qr_layer_internal.h"

namespace qr {
namespace {

// A vector is 8 values, 16 bytes, at any 2-byte address (rows of odd length
// or stride): gfx950 runs with unaligned access enabled, and a memcpy of
// known size becomes one global_load_dwordx4 whatever the alignment.
__device__ __forceinline__ u32x4 load8(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store8(uint8_t* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// The first n values of the vector at p, zeros after them.  Rows of 8 values or
// more: a row's last, short vector is read as the 16 bytes that end where the
// row ends (load_ending) and shifted down (shifted), one load whatever n is.  All
// of a lane's loads come before the first shift: a shift between them waits for
// the load before it (the norm of 3000 x 5003 took 37 us so, now 31.5).
__device__ __forceinline__ u32x4 load_ending(const uint8_t* p, uint32_t n) {
  return load8(p - 2 * (8 - n));
}
__device__ __forceinline__ u32x4 shifted(u32x4 v, uint32_t n) {
  const uint32_t miss = 8 - n;
  if (miss != 0) {
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    if (miss >= 4) {
      lo = hi;
      hi = 0;
    }
    const uint32_t sh = 16 * (miss & 3);
    lo = lo >> sh | (hi << 1) << (63 - sh);
    hi >>= sh;
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  return v;
}
__device__ __forceinline__ u32x4 load_n(const uint8_t* p, uint32_t n) {
  return shifted(load_ending(p, n), n);
}
// the same, value by value, for rows of any length
__device__ __forceinline__ u32x4 load_each(const uint8_t* p, uint32_t n) {
  if (n == 8) return load8(p);
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (uint32_t i = 0; i < n; i++) {
    const uint64_t v = reinterpret_cast<const uint16_t*>(p)[i];
    if (i < 4) lo |= v << (16 * i);
    else hi |= v << (16 * (i - 4));
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
// rows that are whole vectors; rows whose last vector may be short; the same,
// of any length
enum Ends { kWhole, kShort, kAny };
template <int E>
__device__ __forceinline__ u32x4 load_vec(const uint8_t* p, uint32_t n) {
  return E == kWhole ? load8(p) : E == kShort ? load_n(p, n) : load_each(p, n);
}
// the same in two steps
template <int E>
__device__ __forceinline__ u32x4 load_raw(const uint8_t* p, uint32_t n) {
  return E == kWhole ? load8(p) : E == kShort ? load_ending(p, n) : load_each(p, n);
}
template <int E>
__device__ __forceinline__ u32x4 from_raw(u32x4 v, uint32_t n) {
  return E == kShort ? shifted(v, n) : v;
}
template <int E>
__device__ __forceinline__ void store_vec(uint8_t* p, u32x4 v, uint32_t n) {
  if (E == kWhole || n == 8) {
    store8(p, v);
    return;
  }
  uint64_t lo = v.x | (uint64_t)v.y << 32;
  if (n & 4) {
    __builtin_memcpy(p, &lo, 8);
    p += 8;
    lo = v.z | (uint64_t)v.w << 32;
  }
  if (n & 2) {
    const uint32_t two = (uint32_t)lo;
    __builtin_memcpy(p, &two, 4);
    p += 4;
    lo >>= 32;
  }
  if (n & 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)lo;
}

template <int D>
__device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    f[2 * k] = ld16<D>(v[k] & 0xffffu);
    f[2 * k + 1] = ld16<D>(v[k] >> 16);
  }
}

// max(a, |v|) that keeps a NaN (v_maximum3_f32)
__device__ __forceinline__ float max_abs(float a, float v) {
  return __builtin_elementwise_maximum(a, __builtin_fabsf(v));
}

// Words of quarter j (0..3) of a block's codes in a planar wire image: 8 codes
// = 8*b bits starting at bit 8*b*j of the block's bitstring, the first code at
// bit 0 (6-bit quarters 1 and 3 start in the middle of a word).
template <int C>
__device__ __forceinline__ void quarter_words(const uint8_t* blk, int j, u32x4& w) {
  constexpr int b = CodecT<C>::bits;
  if constexpr (b == 4) {
    w[0] = reinterpret_cast<const uint32_t*>(blk)[j];
  } else if constexpr (b == 8) {
    const u32x2 q = reinterpret_cast<const u32x2*>(blk)[j];
    w[0] = q.x;
    w[1] = q.y;
  } else {                                           // bits [48j, 48j+48)
    const uint32_t* p = reinterpret_cast<const uint32_t*>(blk) + ((3 * j) >> 1);
    const uint32_t lo = p[0], hi = p[1];
    const int sh = (j & 1) * 16;
    w[0] = __builtin_amdgcn_alignbit(hi, lo, sh);
    w[1] = hi >> sh;
  }
}

// type of the 16-bit buffers under the wire's type: with the cast option the
// wire holds binary16 and the buffers bfloat16
template <int D>
constexpr int kBufType = D == kBF16H ? (int)kBF16 : D;

// ---------------------------------------------------------------------------
// operators: what a row's vector is read from, and the values to be coded

// C < 0: x from 16-bit rows; else from the planar wire image of codec C.
template <int D, int C>
struct Norm {
  static constexpr bool kNorm = true, kWire = C >= 0;
  static constexpr int B = kBufType<D>;
  NormArgs a;

  struct Raw {
    u32x4 x;               // 16-bit values; for a wire its code words (x, y)
    uint32_t s, z;         // the wire block's scale and zero
    u32x4 res, w;
  };
  struct Row {
    const uint8_t *x, *res;
    uint8_t* h;
    uint32_t vec0;         // the row's first vector in the wire image
  };

  __device__ __forceinline__ Row row(uint32_t m, uint32_t d) const {
    Row r;
    r.x = C < 0 ? a.x + 2 * (size_t)m * a.ldx : a.x;
    r.res = a.residual ? a.residual + 2 * (size_t)m * a.ldr : nullptr;
    r.h = a.h ? a.h + 2 * (size_t)m * a.ldh : nullptr;
    r.vec0 = C < 0 ? 0u : m * (d / 8);
    return r;
  }
  template <int E>
  __device__ __forceinline__ void load(const Row& r, uint32_t vec, uint32_t n, Raw& v) const {
    if constexpr (C < 0) {
      v.x = load_raw<E>(r.x + 16 * (size_t)vec, n);
    } else if constexpr (C == kFP) {
      v.x = load8(r.x + 16 * (size_t)(r.vec0 + vec));
    } else {
      const uint32_t q = r.vec0 + vec;
      quarter_words<C>(r.x + (size_t)(q >> 2) * CodecT<C>::block_bytes, q & 3, v.x);
      v.s = reinterpret_cast<const uint16_t*>(r.x + a.off_s)[q >> 2];
      if constexpr (CodecT<C>::asym)
        v.z = reinterpret_cast<const uint16_t*>(r.x + a.off_z)[q >> 2];
    }
    if (r.res) v.res = load_raw<E>(r.res + 16 * (size_t)vec, n);
    v.w = load_raw<E>(a.weight + 16 * (size_t)vec, n);
  }
  // u and the sum of squares, and h written
  template <int E>
  __device__ __forceinline__ void values(const Row& r, uint32_t vec, uint32_t n, const Raw& v,
                                         float (&u)[8], float& ss) const {
    u32x4 h;
    if constexpr (C < 0) {
      h = from_raw<E>(v.x, n);
    } else if constexpr (C == kFP) {
      h = v.x;
      if constexpr (D == kBF16H)
#pragma unroll
        for (int k = 0; k < 4; k++)
          h[k] = st16x2<kBF16>(h2f(v.x[k] & 0xffffu), h2f(v.x[k] >> 16));
    } else {
      using T = CodecT<C>;
      uint32_t w[2] = {v.x[0], T::bits > 4 ? v.x[1] : 0u};
      float cv[8];
      code_values<C, 8>(w, cv);
      const float s = h2f(v.s) * T::unpack_scale;
      const float z = T::asym ? h2f(v.z) : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i++) cv[i] = T::asym ? __builtin_fmaf(cv[i], s, z) : cv[i] * s;
#pragma unroll
      for (int k = 0; k < 4; k++) h[k] = st16x2<D>(cv[2 * k], cv[2 * k + 1]);
    }
    float hv[8];
    widen<B>(h, hv);
    if (r.res) {
      float rv[8];
      widen<B>(from_raw<E>(v.res, n), rv);
#pragma unroll
      for (int k = 0; k < 4; k++)
        h[k] = st16x2<B>(hv[2 * k] + rv[2 * k], hv[2 * k + 1] + rv[2 * k + 1]);
      widen<B>(h, hv);
    }
    if (r.h) store_vec<E>(r.h + 16 * (size_t)vec, h, n);
    weigh(hv, from_raw<E>(v.w, n), u, ss);
  }
  __device__ __forceinline__ void weigh(const float (&hv)[8], u32x4 w, float (&u)[8],
                                        float& ss) const {
    float wv[8];
    widen<B>(w, wv);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      ss = __builtin_fmaf(hv[i], hv[i], ss);
      u[i] = hv[i] * wv[i];
    }
  }
  // u of a vector whose h this lane has written (or x, where h is not)
  template <int E>
  __device__ __forceinline__ void again(const Row& r, uint32_t vec, uint32_t n,
                                        float (&u)[8]) const {
    const uint8_t* p = (r.h ? r.h : r.x) + 16 * (size_t)vec;
    float hv[8], unused = 0.0f;
    widen<B>(load_vec<E>(p, n), hv);
    weigh(hv, load_vec<E>(a.weight + 16 * (size_t)vec, n), u, unused);
  }
  __device__ __forceinline__ float factor(float ss, uint32_t d) const {
    return 1.0f / __builtin_sqrtf(ss / (float)d + a.eps);
  }
};

template <int D>
struct Silu {
  static constexpr bool kNorm = false, kWire = false;
  const uint8_t* gu;
  size_t ldg;

  struct Raw {
    u32x4 g, u;
  };
  struct Row {
    const uint8_t *g, *u;
  };
  __device__ __forceinline__ Row row(uint32_t m, uint32_t d) const {
    const uint8_t* p = gu + 2 * (size_t)m * ldg;
    return Row{p, p + 2 * (size_t)d};
  }
  template <int E>
  __device__ __forceinline__ void load(const Row& r, uint32_t vec, uint32_t n, Raw& v) const {
    v.g = load_raw<E>(r.g + 16 * (size_t)vec, n);
    v.u = load_raw<E>(r.u + 16 * (size_t)vec, n);
  }
  // exp(-x) for 0 <= x <= 500: v_exp_f32 (2^hi, within one unit) of the rounded
  // hi = -x*log2(e), times 1 + rest, rest = -x - hi*ln 2.  A rounded exponent
  // alone would cost x half units, which moves codes near a tie.  hi and rest
  // are finite, so nothing here is infinite; below 2^-126 the result is 0.
  static __device__ __forceinline__ float exp_minus(float x) {
    constexpr float kLn2 = 0.69314718055994530942f;
    constexpr float kLn2Rest = (float)(0.69314718055994530942 - (double)kLn2);
    const float hi = x * -1.44269504088896341f;
    const float rest = __builtin_fmaf(-kLn2Rest, hi, __builtin_fmaf(-kLn2, hi, -x));
    const float e = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(e, rest, e);
  }
  // g / (1 + exp(-g)) * u, as g*e / (1 + e) * u with e = exp(-|g|) where g is
  // negative and with g in place of g*e elsewhere, so that nothing overflows on
  // the way to a small value: within 16 * 2^-24 of the value whatever the gate.
  // The quotient is v_rcp_f32's with one correction (1 <= 1 + e <= 2).  This is
  // done for |g| <= 64, where e is a normal number that no instruction flushes.
  // A gate beyond becomes +-64 and leaves the rest to u: |g|/64 (exact), and
  // exp(g + 64) if it is negative, in two factors of half the exponent, of
  // which one that is flushed to 0 stands for a value below any binary32; 1 + e
  // rounds to 1 all the same.  An infinity or NaN in g or u comes out as one
  // (inf * 0 among them).  8192 rows of 4096, bf16: 31.4 us, and 32.5 where
  // every wave has a gate beyond.
  template <int E>
  __device__ __forceinline__ void values(const Row&, uint32_t, uint32_t n, const Raw& v,
                                         float (&u)[8], float&) const {
    constexpr float kFar = 64.0f;
    float g[8];
    widen<D>(from_raw<E>(v.g, n), g);
    widen<D>(from_raw<E>(v.u, n), u);
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) most = max_abs(most, g[i]);
    if (!(most <= kFar)) {                                   // rare; a NaN hides no gate
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float x = __builtin_fabsf(g[i]);
        const float half = exp_minus(__builtin_elementwise_minimum(0.5f * (x - kFar), 500.0f));
        if (x > kFar) {
          u[i] = (g[i] < 0.0f ? u[i] * half * half : u[i]) * (x / kFar);
          g[i] = __builtin_copysignf(kFar, g[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float e = exp_minus(__builtin_fabsf(g[i]));
      const float t = 1.0f + e, r = __builtin_amdgcn_rcpf(t);
      const float top = g[i] < 0.0f ? g[i] * e : g[i], q = top * r;
      u[i] *= __builtin_fmaf(__builtin_fmaf(-t, q, top), r, q);
    }
  }
  template <int E>
  __device__ __forceinline__ void again(const Row& r, uint32_t vec, uint32_t n,
                                        float (&u)[8]) const {
    Raw v;
    float unused;
    load<E>(r, vec, n, v);
    values<E>(r, vec, n, v, u, unused);
  }
  __device__ __forceinline__ float factor(float, uint32_t) const { return 1.0f; }
};

// ---------------------------------------------------------------------------

// v joined over the wave by `join`, the same bits in every lane: exchanges
// inside a row of 16 lanes, then of rows and of halves
template <class Join>
__device__ __forceinline__ float wave_join(float v, Join join) {
  const auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf,
                                        0xf, true));
  };
  v = join(v, dpp(v, std::integral_constant<int, 0xb1>{}));      // lane ^ 1
  v = join(v, dpp(v, std::integral_constant<int, 0x4e>{}));      // lane ^ 2
  v = join(v, dpp(v, std::integral_constant<int, 0x141>{}));     // the other four of 8
  v = join(v, dpp(v, std::integral_constant<int, 0x140>{}));     // the other eight of 16
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto rows = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  v = join(__builtin_bit_cast(float, (uint32_t)rows[0]), __builtin_bit_cast(float, (uint32_t)rows[1]));
  const uint32_t y = __builtin_bit_cast(uint32_t, v);
  const auto halves = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return join(__builtin_bit_cast(float, (uint32_t)halves[0]),
              __builtin_bit_cast(float, (uint32_t)halves[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_join(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_join(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}

// over the row's waves, at most 16, through LDS: every lane gets the result.
// Entries of waves that are not there hold 0, which changes neither (magnitudes
// are not negative).
struct Joined {
  float ss[16], a[16];
};
template <bool Sum>
__device__ __forceinline__ void waves_reduce(float& ss, float& a, Joined& lds) {
  const uint32_t t = threadIdx.x;
  if (t % 64 == 0) {
    if (Sum) lds.ss[t / 64] = ss;
    lds.a[t / 64] = a;
  }
  __syncthreads();
  ss = 0.0f;
  a = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; w++) {
    if (Sum) ss += lds.ss[w];
    a = __builtin_elementwise_maximum(a, lds.a[w]);
  }
}
__device__ __forceinline__ void clear(Joined& lds) {
  const uint32_t t = threadIdx.x, waves = blockDim.x / 64;
  if (t >= waves && t < 16) lds.ss[t] = lds.a[t] = 0.0f;
}

template <int E>
__device__ __forceinline__ void store_codes(int8_t* p, u32x2 w, uint32_t n) {
  if (E == kWhole || n == 8) {
    __builtin_memcpy(p, &w, 8);
  } else {
    uint32_t v = w.x;
    if (n & 4) {
      __builtin_memcpy(p, &v, 4);
      p += 4;
      v = w.y;
    }
    if (n & 2) {
      const uint16_t two = (uint16_t)v;
      __builtin_memcpy(p, &two, 2);
      p += 2;
      v >>= 16;
    }
    if (n & 1) *p = (int8_t)v;
  }
}

}  // namespace
}  // namespace qr
