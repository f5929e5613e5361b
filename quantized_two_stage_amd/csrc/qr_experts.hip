// qr_experts.hip -- gfx950 kernels around the products of a mixture of experts
// (include/qr_f8.h): the choice of every token's experts with the rows sorted by
// expert, and the weighted sum of a token's rows.
#include "qr_f8.h"
#include "qr_f8_internal.h"
#include "qr_rows_device.h"

namespace qr {
namespace {

// ---------------------------------------------------------------------------
// the router
//
// Tokens are taken 64 at a time: one bit of a 64-bit word for each, a word for
// each expert, so the rows that an expert gets from them, and how many of those
// lie before a token's, are population counts, whatever the order in which the
// waves set the bits.  Up to 64 tokens one workgroup does everything.  Above, a
// launch chooses and counts (k_choose, a workgroup for `turns` times 64 tokens),
// and a second one adds up the counts before its tokens' and places the rows
// (k_place); there are at most kMaxChunks counts of an expert to add.
//
// A token's k experts are k times the largest of its logits, held as ordered keys
// in the registers of a few lanes; weights are exponentials of differences to the
// largest logit, so nothing overflows, summed in binary32.
//
// Bound by the chain of k reductions over a group's lanes and, above 64 tokens, by
// adding up the counts in k_place (its LDS atomics conflict in 74% of the cycles that
// LDS is active in); short calls by the launch.
// Measured, k = 8: 16384 tokens over 256 experts, bf16: 18.7 us (k_choose 11, k_place
// 7.5), binary32: 23.6; 4096 over 512: 18 to 22 and 53; 4096 over 64: 9.4 and 11.5; 64
// over 512: 17 and 45; the bytes alone would take 2 to 4 at most.  16 over 32, k = 4: 4.0.
// Binary32 logits are read one by one and need a second reduction for the expert's
// number; over 257 to 512 experts (more than 16 tokens) 16 lanes hold 32 each, which
// passes the 128 registers that 1024 lanes have: 135 registers a lane are spilled, 147 up
// to 64 tokens (16-bit logits: 3 up to 64 tokens, none above).
// Placing the rows in a second launch costs about 2.5 us, but its workgroups need
// all the counts, and no workgroup may wait for another.

constexpr uint32_t kTokens = 64;           // of a turn
constexpr uint32_t kMaxChunks = 256;
constexpr uint32_t kLanes = 1024;

// The workspace: of every workgroup of k_choose a row of its experts' rows, at
// most 64 * 256 each.
__host__ __device__ constexpr uint32_t row_of_counts(uint32_t E) { return (E + 7) / 8 * 8; }

struct Masks {
  unsigned long long bits[QR_MAX_EXPERTS];
};

// v joined over groups of G lanes (8, 16 or 64), the same bits in every lane of a
// group
template <int G, class Join>
__device__ __forceinline__ uint32_t group_join(uint32_t v, Join join) {
  const auto dpp = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, decltype(ctrl)::value, 0xf, 0xf, true);
  };
  v = join(v, dpp(v, std::integral_constant<int, 0xb1>{}));      // lane ^ 1
  v = join(v, dpp(v, std::integral_constant<int, 0x4e>{}));      // lane ^ 2
  v = join(v, dpp(v, std::integral_constant<int, 0x141>{}));     // the other four of 8
  if constexpr (G >= 16) v = join(v, dpp(v, std::integral_constant<int, 0x140>{}));
  if constexpr (G == 64) {
    const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = join((uint32_t)rows[0], (uint32_t)rows[1]);
    const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = join((uint32_t)halves[0], (uint32_t)halves[1]);
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_join<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return __builtin_bit_cast(
      float, group_join<G>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(
            uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
      }));
}
// the sum of v over the lanes up to this one
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const uint32_t lane = threadIdx.x % 64;
#pragma unroll
  for (uint32_t d = 1; d < 64; d *= 2) {
    const uint32_t w = (uint32_t)__shfl_up((int)v, d);
    if (lane >= d) v += w;
  }
  return v;
}
// The sum of v over the lanes of the workgroup before this one.
template <int Waves>
__device__ __forceinline__ uint32_t before(uint32_t v, uint32_t (&lds)[Waves]) {
  const uint32_t up_to = wave_scan(v);
  if (threadIdx.x % 64 == 63) lds[threadIdx.x / 64] = up_to;
  __syncthreads();
  uint32_t sum = up_to - v;
#pragma unroll
  for (uint32_t w = 0; w < Waves; w++) sum += w < threadIdx.x / 64 ? lds[w] : 0u;
  return sum;
}

// A logit as a number that orders as the logits do: -0 as +0, NaN below
// -infinity, 0 for what cannot be chosen.  Of 16 bits: the upper half, with the
// expert's number, the lowest highest, in the lower half, so that no two are equal.
template <int D>
__device__ __forceinline__ uint32_t key_of(float x, uint32_t e) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  if constexpr (D == kF32) {
    return x != x ? 1u : (int)b < 0 ? ~b : b | 0x80000000u;
  } else {
    const uint32_t h = st16<D>(x + 0.0f);        // the logit's own bits
    const uint32_t k = x != x ? 1u : h & 0x8000u ? ~h & 0xffffu : h | 0x8000u;
    return k << 16 | (0xffffu - e);
  }
}
template <int D>
__device__ __forceinline__ float logit_of(uint32_t key) {
  if constexpr (D == kF32) {
    return key == 1u ? __builtin_nanf("")
                     : __builtin_bit_cast(float, (int)key < 0 ? key & 0x7fffffffu : ~key);
  } else {
    const uint32_t k = key >> 16;
    return k == 1u ? __builtin_nanf("") : ld16<D>(k & 0x8000u ? k & 0x7fffu : ~k & 0xffffu);
  }
}
// exp(x - top) for x <= top; 0 for x = -infinity whatever top is
__device__ __forceinline__ float exp_below(float x, float top) {
  const float d = top - x;
  const float e = Silu<kF16>::exp_minus(d > 500.0f ? 500.0f : d);
  return x == -__builtin_inff() ? 0.0f : e;
}

// The k experts of one token, by G lanes that hold V logits each: k times the
// largest key left, the lowest expert that has it.  Lane l of the group returns
// experts and weights l, l + G, ...
template <int D, int G, int V>
__device__ __forceinline__ void choose(const RouteArgs& a, uint32_t token,
                                       uint32_t (&expert)[QR_MAX_CHOSEN / G + 1],
                                       float (&weight)[QR_MAX_CHOSEN / G + 1]) {
  constexpr uint32_t kEach = (QR_MAX_CHOSEN + G - 1) / G;
  const uint32_t lane = threadIdx.x % G;
  const uint8_t* const p = a.logits + (size_t)token * a.ldl * (D == kF32 ? 4 : 2);
  uint32_t key[V];
  // vectors of 8 logits, a group's side by side
  const auto expert_of = [&](int v) { return (v / 8 * G + lane) * 8 + v % 8; };
#pragma unroll
  for (int v = 0; v < V; v += 8) {
    const uint32_t e = expert_of(v), n = e >= a.E ? 0u : a.E - e < 8 ? a.E - e : 8;
    float x[8];
    if constexpr (D == kF32) {
#pragma unroll
      for (uint32_t i = 0; i < 8; i++)
        x[i] = reinterpret_cast<const float*>(p)[i < n ? e + i : 0];
    } else {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (n != 0) w = a.E >= 8 ? load_n(p + 2 * e, n) : load_each(p + 2 * e, n);
      widen<D>(w, x);
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; i++) key[v + i] = i < n ? key_of<D>(x[i], e + i) : 0u;
  }
  const auto largest_key = [&] {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; v++) m = key[v] > m ? key[v] : m;
    return group_max<G>(m);
  };
  uint32_t m = largest_key();
  const float top = logit_of<D>(m);
  float all = 0.0f;
  if (!a.renormalize) {
#pragma unroll
    for (int v = 0; v < V; v++)
      all += key[v] == 0u ? 0.0f : exp_below(logit_of<D>(key[v]), top);
    all = group_sum<G>(all);
  }
  float chosen = 0.0f;
#pragma unroll
  for (uint32_t r = 0; r < kEach; r++) {
    uint32_t mine = 0u;
    expert[r] = 0u;
    for (uint32_t j = r * G; j < a.k && j < (r + 1) * G; j++) {
      uint32_t e;
      if constexpr (D == kF32) {
        uint32_t first = 0u;               // its complement
#pragma unroll
        for (int v = V - 1; v >= 0; v--) first = key[v] == m ? ~expert_of(v) : first;
        e = ~group_max<G>(first);
      } else {
        e = 0xffffu - (m & 0xffffu);
      }
      if (lane == j - r * G) {
        mine = m;
        expert[r] = e;
      }
#pragma unroll
      for (int v = 0; v < V; v++)
        key[v] = (D == kF32 ? expert_of(v) == e : key[v] == m) ? 0u : key[v];
      m = largest_key();
    }
    weight[r] = r * G + lane < a.k ? exp_below(logit_of<D>(mine), top) : 0.0f;
    chosen += weight[r];
  }
  if (a.renormalize) all = group_sum<G>(chosen);
#pragma unroll
  for (uint32_t r = 0; r < kEach; r++) weight[r] = all == 0.0f ? 0.0f : weight[r] / all;
}

// The places of the rows of one turn (64 tokens from t0 on): `base` holds where
// each expert's next row goes.
__device__ __forceinline__ void place_turn(const RouteArgs& a, uint32_t t0, uint32_t tokens,
                                           const Masks& masks, const uint16_t (&chosen)[kTokens][QR_MAX_CHOSEN],
                                           const uint32_t* base) {
  for (uint32_t x = threadIdx.x; x < tokens * a.k; x += blockDim.x) {
    const uint32_t t = x / a.k, j = x - t * a.k, e = chosen[t][j];
    const uint32_t row = base[e] + (uint32_t)__popcll(masks.bits[e] & ((1ull << t) - 1));
    a.place[(size_t)t0 * a.k + x] = (int32_t)row;
    // always so, unless another call has written the workspace meanwhile
    if (row < a.T * a.k) a.rows[row] = (int32_t)(t0 + t);
  }
}

// All: the only workgroup, which also places the rows.  At least E lanes.
template <int D, int G, int V, int Lanes, bool All>
__global__ __launch_bounds__(Lanes) void k_choose(RouteArgs a, uint32_t turns) {
  __shared__ Masks masks;
  __shared__ uint16_t chosen[kTokens][QR_MAX_CHOSEN];
  __shared__ uint32_t base[All ? QR_MAX_EXPERTS : 1], sums[Lanes / 64];
  const uint32_t lane = threadIdx.x % G, group = threadIdx.x / G;
  uint32_t count = 0;                      // of expert threadIdx.x
  for (uint32_t i = 0; i < turns; i++) {
    const uint32_t t0 = (blockIdx.x * turns + i) * kTokens;
    const uint32_t tokens = t0 >= a.T ? 0u : a.T - t0 < kTokens ? a.T - t0 : kTokens;
    if (threadIdx.x < a.E) masks.bits[threadIdx.x] = 0ull;
    __syncthreads();
    // whole waves take part as long as one of their groups has a token
    for (uint32_t t = group; t - group % (64 / G) < tokens; t += Lanes / G) {
      uint32_t expert[QR_MAX_CHOSEN / G + 1];
      float weight[QR_MAX_CHOSEN / G + 1];
      choose<D, G, V>(a, t0 + (t < tokens ? t : tokens - 1), expert, weight);
#pragma unroll
      for (uint32_t r = 0; r * G < QR_MAX_CHOSEN; r++) {
        const uint32_t j = r * G + lane;
        if (t < tokens && j < a.k) {
          const size_t at = (size_t)(t0 + t) * a.k + j;
          a.experts[at] = (int32_t)expert[r];
          a.weights[at] = weight[r];
          atomicOr(&masks.bits[expert[r]], 1ull << t);
          if (All) chosen[t][j] = (uint16_t)expert[r];
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < a.E) count += (uint32_t)__popcll(masks.bits[threadIdx.x]);
    if (All) {
      const uint32_t from = before(count, sums);
      if (threadIdx.x < a.E) {
        base[threadIdx.x] = from;
        a.offsets[threadIdx.x] = (int32_t)from;
        if (threadIdx.x == a.E - 1) a.offsets[a.E] = (int32_t)(from + count);
      }
      __syncthreads();
      place_turn(a, t0, tokens, masks, chosen, base);
    } else {
      __syncthreads();                     // the masks are cleared again
    }
  }
  // rows of whole vectors of 8: lanes past E hold 0
  if (!All && threadIdx.x < row_of_counts(a.E))
    a.counts[(size_t)blockIdx.x * row_of_counts(a.E) + threadIdx.x] = (uint16_t)count;
}

__global__ __launch_bounds__(kLanes) void k_place(RouteArgs a, uint32_t turns) {
  __shared__ Masks masks;
  __shared__ uint16_t chosen[kTokens][QR_MAX_CHOSEN];
  __shared__ uint32_t base[QR_MAX_EXPERTS], total[QR_MAX_EXPERTS], sums[kLanes / 64];
  const uint32_t t = threadIdx.x;
  if (t < a.E) base[t] = total[t] = 0u;
  __syncthreads();
  // vectors of 8 experts' counts, every G-th workgroup's; 8 loads at a time, and no
  // more lanes than they keep busy (16384 tokens over 8 experts: 8 us; with all
  // lanes, which meet on the same words of LDS, 20)
  const uint32_t row = row_of_counts(a.E), per = row / 8, most = (gridDim.x + 7) / 8;
  const uint32_t G = kLanes / per < most ? kLanes / per : most;
  if (t < G * per) {
    const uint32_t e0 = t % per * 8;
    uint32_t all[8] = {}, earlier[8] = {};
    for (uint32_t c = t / per; c < gridDim.x; c += 8 * G) {
      u32x4 v[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; i++) {
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (c + i * G < gridDim.x)
          __builtin_memcpy(&v[i], a.counts + (size_t)(c + i * G) * row + e0, 16);
      }
#pragma unroll
      for (uint32_t i = 0; i < 8; i++)
#pragma unroll
        for (uint32_t e = 0; e < 8; e++) {
          const uint32_t n = v[i][e / 2] >> (16 * (e % 2)) & 0xffffu;
          all[e] += n;
          earlier[e] += c + i * G < blockIdx.x ? n : 0u;
        }
    }
#pragma unroll
    for (uint32_t e = 0; e < 8; e++)
      if (e0 + e < a.E) {
        atomicAdd(&total[e0 + e], all[e]);
        atomicAdd(&base[e0 + e], earlier[e]);
      }
  }
  __syncthreads();
  const uint32_t mine = t < a.E ? total[t] : 0u, from = before(mine, sums);
  if (t < a.E) {
    base[t] += from;
    if (blockIdx.x == 0) {
      a.offsets[t] = (int32_t)from;
      if (t == a.E - 1) a.offsets[a.E] = (int32_t)(from + mine);
    }
  }
  for (uint32_t i = 0; i < turns; i++) {
    const uint32_t t0 = (blockIdx.x * turns + i) * kTokens;
    const uint32_t tokens = t0 >= a.T ? 0u : a.T - t0 < kTokens ? a.T - t0 : kTokens;
    if (t < a.E) masks.bits[t] = 0ull;
    __syncthreads();
    for (uint32_t x = t; x < tokens * a.k; x += kLanes) {
      const uint32_t tt = x / a.k, j = x - tt * a.k;
      const uint32_t e = (uint32_t)a.experts[(size_t)t0 * a.k + x];
      chosen[tt][j] = (uint16_t)e;
      atomicOr(&masks.bits[e], 1ull << tt);
    }
    __syncthreads();
    place_turn(a, t0, tokens, masks, chosen, base);
    __syncthreads();
    if (t < a.E) base[t] += (uint32_t)__popcll(masks.bits[t]);
  }
}

struct Chunks {
  uint32_t turns, count;                   // turns of a workgroup, workgroups
};
Chunks chunks_of(uint32_t T) {
  const uint32_t all = (T + kTokens - 1) / kTokens;
  const uint32_t turns = (all + kMaxChunks - 1) / kMaxChunks;
  return Chunks{turns, turns ? (all + turns - 1) / turns : 0u};
}

// G lanes to a token, V logits to a lane: at most G * V experts.
template <int D, int G, int V>
hipError_t route_at_once(const RouteArgs& a, hipStream_t st) {
  if constexpr (G * V <= 256)              // a lane to an expert
    if (a.T * G <= 256) {                  // a launch of few waves starts sooner
      k_choose<D, G, V, 256, true><<<1, 256, 0, st>>>(a, 1);
      return hipGetLastError();
    }
  k_choose<D, G, V, kLanes, true><<<1, kLanes, 0, st>>>(a, 1);
  return hipGetLastError();
}
template <int D, int G, int V>
hipError_t route(const RouteArgs& a, hipStream_t st) {
  if (a.T <= kTokens) return route_at_once<D, G, V>(a, st);
  const Chunks c = chunks_of(a.T);
  k_choose<D, G, V, kLanes, false><<<c.count, kLanes, 0, st>>>(a, c.turns);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_place<<<c.count, kLanes, 0, st>>>(a, c.turns);
  return hipGetLastError();
}
template <int D>
hipError_t route_by_experts(const RouteArgs& a, hipStream_t st) {
  // few lanes to a token where there are tokens enough: fewer exchanges, and as
  // many tokens side by side (4096 tokens over 512 experts: 18 us, with 64 lanes 22)
  if (a.E <= 64) return route<D, 8, 8>(a, st);
  if (a.E <= 128) return route<D, 16, 8>(a, st);
  if (a.E <= 256) return route<D, 16, 16>(a, st);
  if (a.E <= 512) return a.T <= 16 ? route_at_once<D, 64, 8>(a, st) : route<D, 16, 32>(a, st);
  return route<D, 64, 16>(a, st);
}

// ---------------------------------------------------------------------------
// the weighted sum

constexpr uint32_t kSumWaves = 4;          // of a workgroup
constexpr uint32_t kAtOnce = 8;            // rows on their way at a time

// y = sum_j weights[j] * c[place[j]] + addend in binary32, rounded once.  A wave
// takes 64 vectors of 8 values of one token's row (`pieces` waves to a token), and
// has up to 8 rows' vectors on their way.  Bound by HBM: 4096 tokens, k = 8, 8192
// bf16 122 us, 4.95 TB/s (a copy 5.2); k = 2 51 us, 5.3 TB/s; 17 x 5003 4.0 us, a
// launch with two dependent reads.
template <int D, int E>
__global__ __launch_bounds__(64 * kSumWaves) void k_combine(CombineArgs a, uint32_t pieces,
                                                           uint32_t waves) {
  const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(blockIdx.x * kSumWaves + threadIdx.x / 64));
  if (w >= waves) return;
  const uint32_t t = w / pieces, vec = (w - t * pieces) * 64 + threadIdx.x % 64, i0 = 8 * vec;
  if (i0 >= a.d) return;
  const uint32_t n = a.d - i0 < 8 ? a.d - i0 : 8;
  const int32_t* const place = a.place + (size_t)t * a.k;
  const float* const weights = a.weights + (size_t)t * a.k;
  u32x4 add = {0u, 0u, 0u, 0u};
  if (a.addend) add = load_raw<E>(a.addend + 2 * ((size_t)t * a.lda + i0), n);
  float y[8] = {};
  for (uint32_t j0 = 0; j0 < a.k; j0 += kAtOnce) {
    u32x4 v[kAtOnce];
    uint32_t row[kAtOnce];
#pragma unroll
    for (uint32_t j = 0; j < kAtOnce; j++) {
      row[j] = j0 + j < a.k ? (uint32_t)place[j0 + j] : ~0u;
      if (row[j] < a.R) v[j] = load_raw<E>(a.c + 2 * ((size_t)row[j] * a.ldc + i0), n);
    }
#pragma unroll
    for (uint32_t j = 0; j < kAtOnce; j++)
      if (row[j] < a.R) {
        const float s = weights[j0 + j];
        float f[8];
        widen<D>(from_raw<E>(v[j], n), f);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_fmaf(s, f[i], y[i]);
      }
  }
  if (a.addend) {
    float f[8];
    widen<D>(from_raw<E>(add, n), f);
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] += f[i];
  }
  u32x4 out;
#pragma unroll
  for (int k = 0; k < 4; k++) out[k] = st16x2<D>(y[2 * k], y[2 * k + 1]);
  store_vec<E>(a.y + 2 * ((size_t)t * a.ldy + i0), out, n);
}

template <int D>
hipError_t combine(const CombineArgs& all, hipStream_t st) {
  const uint32_t pieces = (all.d + 511) / 512;
  const uint32_t most = (1u << 25) / pieces;      // tokens of a launch: lanes are counted in 32 bits
  for (uint32_t t = 0; t < all.T; t += most) {
    CombineArgs a = all;
    a.T = all.T - t < most ? all.T - t : most;
    a.place += (size_t)t * a.k;
    a.weights += (size_t)t * a.k;
    if (a.addend) a.addend += 2 * (size_t)t * a.lda;
    a.y += 2 * (size_t)t * a.ldy;
    const uint32_t waves = a.T * pieces, groups = (waves + kSumWaves - 1) / kSumWaves;
    if (a.d < 8) k_combine<D, kAny><<<groups, 64 * kSumWaves, 0, st>>>(a, pieces, waves);
    else if (a.d % 8 != 0) k_combine<D, kShort><<<groups, 64 * kSumWaves, 0, st>>>(a, pieces, waves);
    else k_combine<D, kWhole><<<groups, 64 * kSumWaves, 0, st>>>(a, pieces, waves);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t route_workspace_bytes(uint32_t T, uint32_t E) {
  return T <= kTokens ? 0 : (size_t)chunks_of(T).count * row_of_counts(E) * 2;
}

hipError_t launch_route(int dtype, const RouteArgs& a, hipStream_t st) {
  switch (dtype) {
    case kF16: return route_by_experts<kF16>(a, st);
    case kBF16: return route_by_experts<kBF16>(a, st);
    default: return route_by_experts<kF32>(a, st);
  }
}

hipError_t launch_combine(int dtype, const CombineArgs& a, hipStream_t st) {
  return dtype == kF16 ? combine<kF16>(a, st) : combine<kBF16>(a, st);
}

}  // namespace qr
