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

constexpr uint32_t kTokens = 64;           // of a turn
constexpr uint32_t kMaxChunks = 256;
constexpr uint32_t kLanes = 1024;
constexpr uint32_t kWaves = kLanes / 64;

struct Masks {
  unsigned long long bits[QR_MAX_EXPERTS];
};

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  const auto word = [](float f) { return __builtin_bit_cast(uint32_t, f); };
  return word(wave_join(__builtin_bit_cast(float, v), [&](float a, float b) {
    return __builtin_bit_cast(float, word(a) > word(b) ? word(a) : word(b));
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
// The sum of v over the lanes before this one, of kLanes.
__device__ __forceinline__ uint32_t before(uint32_t v, uint32_t (&lds)[kWaves]) {
  const uint32_t up_to = wave_scan(v);
  if (threadIdx.x % 64 == 63) lds[threadIdx.x / 64] = up_to;
  __syncthreads();
  uint32_t sum = up_to - v;
  for (uint32_t w = 0; w < threadIdx.x / 64; w++) sum += lds[w];
  return sum;
}

// A logit as a number that orders as the logits do: -0 as +0, NaN below
// -infinity, 0 for what cannot be chosen.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x != x ? 1u : (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return key == 1u ? __builtin_nanf("")
                   : __builtin_bit_cast(float, (int)key < 0 ? key & 0x7fffffffu : ~key);
}
// exp(x - top) for x <= top; 0 for x = -infinity whatever top is
__device__ __forceinline__ float exp_below(float x, float top) {
  const float d = top - x;
  const float e = Silu<kF16>::exp_minus(d > 500.0f ? 500.0f : d);
  return x == -__builtin_inff() ? 0.0f : e;
}

// The k experts of one token, by one wave: k times the largest key left, the
// lowest expert that has it.  Lane j returns the j-th expert and its weight.
template <int D, int V>
__device__ __forceinline__ void choose(const RouteArgs& a, uint32_t token, uint32_t& expert,
                                       float& weight) {
  const uint32_t lane = threadIdx.x % 64;
  const uint8_t* const p = a.logits + (size_t)token * a.ldl * (D == kF32 ? 4 : 2);
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const uint32_t e = v * 64 + lane, at = e < a.E ? e : a.E - 1;
    float x;
    if constexpr (D == kF32) x = reinterpret_cast<const float*>(p)[at];
    else x = ld16<D>(reinterpret_cast<const uint16_t*>(p)[at]);
    key[v] = e < a.E ? key_of(x) : 0u;
  }
  float all = 0.0f, top = 0.0f;
  if (!a.renormalize) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; v++) m = key[v] > m ? key[v] : m;
    top = logit_of(wave_max_u32(m));
#pragma unroll
    for (int v = 0; v < V; v++)
      all += key[v] == 0u ? 0.0f : exp_below(logit_of(key[v]), top);
    all = wave_sum(all);
  }
  uint32_t mine = 0u;
  expert = 0u;
  for (uint32_t j = 0; j < a.k; j++) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; v++) m = key[v] > m ? key[v] : m;
    m = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_max_u32(m));
    uint32_t e = 0;
    bool found = false;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const uint64_t have = __ballot(key[v] == m);
      if (!found && have != 0) {
        e = v * 64 + (uint32_t)__builtin_ctzll(have);
        found = true;
        if (v * 64 + lane == e) key[v] = 0u;
      }
    }
    if (j == 0) top = logit_of(m);
    if (lane == j) {
      mine = m;
      expert = e;
    }
  }
  const float x = lane < a.k ? exp_below(logit_of(mine), top) : 0.0f;
  if (a.renormalize) all = wave_sum(x);
  weight = all == 0.0f ? 0.0f : x / all;
}

// The places of the rows of one turn (64 tokens from t0 on): `base` holds where
// each expert's next row goes.
__device__ __forceinline__ void place_turn(const RouteArgs& a, uint32_t t0, uint32_t tokens,
                                           const Masks& masks, const uint16_t (&chosen)[kTokens][QR_MAX_CHOSEN],
                                           const uint32_t* base) {
  for (uint32_t x = threadIdx.x; x < tokens * a.k; x += kLanes) {
    const uint32_t t = x / a.k, j = x - t * a.k, e = chosen[t][j];
    const uint32_t row = base[e] + (uint32_t)__popcll(masks.bits[e] & ((1ull << t) - 1));
    a.place[(size_t)t0 * a.k + x] = (int32_t)row;
    // always so, unless another call has written the workspace meanwhile
    if (row < a.T * a.k) a.rows[row] = (int32_t)(t0 + t);
  }
}

// All: the only workgroup, which also places the rows.
template <int D, int V, bool All>
__global__ __launch_bounds__(kLanes) void k_choose(RouteArgs a, uint32_t turns) {
  __shared__ Masks masks;
  __shared__ uint16_t chosen[kTokens][QR_MAX_CHOSEN];
  __shared__ uint32_t base[All ? QR_MAX_EXPERTS : 1], sums[kWaves];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  uint32_t count = 0;                      // of expert threadIdx.x
  for (uint32_t i = 0; i < turns; i++) {
    const uint32_t t0 = (blockIdx.x * turns + i) * kTokens;
    const uint32_t tokens = t0 >= a.T ? 0u : a.T - t0 < kTokens ? a.T - t0 : kTokens;
    if (threadIdx.x < a.E) masks.bits[threadIdx.x] = 0ull;
    __syncthreads();
    for (uint32_t t = wave; t < tokens; t += kWaves) {
      uint32_t expert;
      float weight;
      choose<D, V>(a, t0 + t, expert, weight);
      if (lane < a.k) {
        const size_t at = (size_t)(t0 + t) * a.k + lane;
        a.experts[at] = (int32_t)expert;
        a.weights[at] = weight;
        atomicOr(&masks.bits[expert], 1ull << t);
        if (All) chosen[t][lane] = (uint16_t)expert;
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
  if (!All && threadIdx.x < a.E) a.counts[(size_t)blockIdx.x * a.E + threadIdx.x] = count;
}

__global__ __launch_bounds__(kLanes) void k_place(RouteArgs a, uint32_t turns) {
  __shared__ Masks masks;
  __shared__ uint16_t chosen[kTokens][QR_MAX_CHOSEN];
  __shared__ uint32_t base[QR_MAX_EXPERTS], total[QR_MAX_EXPERTS], sums[kWaves];
  const uint32_t t = threadIdx.x;
  if (t < a.E) base[t] = total[t] = 0u;
  __syncthreads();
  // lanes g*E + e: of expert e, every G-th workgroup's count
  const uint32_t G = kLanes / a.E;
  if (t < G * a.E) {
    const uint32_t e = t % a.E;
    uint32_t all = 0, earlier = 0;
#pragma unroll 4
    for (uint32_t c = t / a.E; c < gridDim.x; c += G) {
      const uint32_t n = a.counts[(size_t)c * a.E + e];
      all += n;
      earlier += c < blockIdx.x ? n : 0u;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&base[e], earlier);
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

template <int D, int V>
hipError_t route(const RouteArgs& a, hipStream_t st) {
  if (a.T <= kTokens) {
    k_choose<D, V, true><<<1, kLanes, 0, st>>>(a, 1);
    return hipGetLastError();
  }
  const Chunks c = chunks_of(a.T);
  k_choose<D, V, false><<<c.count, kLanes, 0, st>>>(a, c.turns);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_place<<<c.count, kLanes, 0, st>>>(a, c.turns);
  return hipGetLastError();
}
template <int D>
hipError_t route_by_experts(const RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) return route<D, 1>(a, st);
  if (a.E <= 128) return route<D, 2>(a, st);
  if (a.E <= 256) return route<D, 4>(a, st);
  if (a.E <= 512) return route<D, 8>(a, st);
  return route<D, 16>(a, st);
}

// ---------------------------------------------------------------------------
// the weighted sum

constexpr uint32_t kSumWaves = 4;          // of a workgroup
constexpr uint32_t kAtOnce = 8;            // rows on their way at a time

// A wave takes 64 vectors of 8 values of one token's row: `pieces` waves to a
// token.
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
  if (a.addend) add = load_vec<E>(a.addend + 2 * ((size_t)t * a.lda + i0), n);
  float y[8] = {};
  for (uint32_t j0 = 0; j0 < a.k; j0 += kAtOnce) {
    u32x4 v[kAtOnce];
    uint32_t row[kAtOnce];
#pragma unroll
    for (uint32_t j = 0; j < kAtOnce; j++) {
      row[j] = j0 + j < a.k ? (uint32_t)place[j0 + j] : ~0u;
      if (row[j] < a.R) v[j] = load_vec<E>(a.c + 2 * ((size_t)row[j] * a.ldc + i0), n);
    }
#pragma unroll
    for (uint32_t j = 0; j < kAtOnce; j++)
      if (row[j] < a.R) {
        const float s = weights[j0 + j];
        float f[8];
        widen<D>(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_fmaf(s, f[i], y[i]);
      }
  }
  if (a.addend) {
    float f[8];
    widen<D>(add, f);
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
  return T <= kTokens ? 0 : (size_t)chunks_of(T).count * E * sizeof(uint32_t);
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
