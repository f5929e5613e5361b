// qr_gemm.hip -- gfx950 kernels of qr_gemm_i8 (include/qr_layer.h): the matrix
// product of 8-bit codes with a scale for each token and each output channel.
//
// c = (sum_k a[m][k] * b[n][k]) * (sa[m] * sb[n]) + bias[n]; the sum in 32-bit
// integers on the matrix units (16x16x64 blocks), so any order of it gives
// the same bits.  Both operands pass through LDS in stages of 128 codes,
// loaded there directly (eight lanes to the 128 bytes of a row: read straight
// into the matrix instructions' operands, where neighbouring lanes hold
// different rows, the same bytes took one cycle a lane, 16 bytes a cycle and
// CU).  Two kernels share the loads and the swizzle (16-byte piece c of row r
// at place c ^ (r & 7): the 16 rows of a fragment fall on all banks):
//   k_split  few tiles: the waves of a workgroup share the sum of one small
//            tile, each with a ring of its own and no barrier; latency bounds
//            a stage (0.065 us at 16x16, 0.24 us at 64x64), so the sum's
//            stages run side by side;
//   k_tile   many tiles: the waves share one tile and one ring; the loads to
//            LDS bound a stage, at 256x256 the matrix units too.
// A stage of k_tile, ns, with 256 workgroups: 64x128 365, without its matrix
// instructions 348, without its reads of LDS 373, without its loads 270;
// 128x128 557, 471, 494, 431; 256x256 1661, 1376, 1748, 1105.
// Measured (cold weights): 1 token over 8192x8192 weights 11.9 to 12.6 us, 5.3
// to 5.6 TB/s (plain reads reach 6.8); 48 tokens, 8192x4096: 11.1 to 13 us;
// 8192^3: 420 to 442 us, 2490 to 2620 TOPS, the matrix units busy 67% of the
// time (a library product of the same codes without scales: 528 us).
#include <type_traits>
#include <utility>

#include "qr.h"
#include "qr_gemm_device.h"
#include "qr_gemm_tiles.h"
#include "qr_layer_internal.h"

namespace qr {
namespace {

// scales and bias of W neighbouring channels
template <int W>
struct Channels {
  float sb[W], bias[W];
  bool biased;
  __device__ __forceinline__ float value(int32_t sum, float sa, int e) const {
    const float v = (float)sum * (sa * sb[e]);
    return biased ? v + bias[e] : v;
  }
};
template <int D, int W>
__device__ __forceinline__ Channels<W> channels(const GemmArgs& g, uint32_t n) {
  Channels<W> ch;
  ch.biased = g.bias != nullptr;
  const uint16_t* b16 = reinterpret_cast<const uint16_t*>(g.bias);
#pragma unroll
  for (int e = 0; e < W; e++) {
    const uint32_t at = n + e < g.N ? n + e : g.N - 1;
    ch.sb[e] = g.sb[at];
    ch.bias[e] = ch.biased ? ld16<D>(b16[at]) : 0.0f;
  }
  return ch;
}

// The sums of W waves, each FN blocks of 16 channels wide and `Apart` entries
// after the one before, joined and written: entry x holds 4 neighbouring
// channels of one token.
template <int D, int BM, int W, int FN, uint32_t Apart>
__device__ __forceinline__ void finish(const GemmArgs& g, uint32_t m0, uint32_t n0, uint32_t x,
                                       const i32x4* part) {
  const uint32_t f = x / 64, m = m0 + f / FN * 16 + x % 16, n = n0 + f % FN * 16 + x % 64 / 16 * 4;
  i32x4 sum = part[x];
#pragma unroll
  for (int w = 1; w < W; w++) sum += part[w * Apart + x];
  if (m < g.M && n < g.N && (BM >= 16 || x % 16 < BM)) {
    const Channels<4> ch = channels<D, 4>(g, n);
    const float sa = g.sa[m];
    u32x2 v;
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      v[e / 2] = st16x2<D>(ch.value(sum[e], sa, e), ch.value(sum[e + 1], sa, e + 1));
    store_row<4>(g, m, n, v);
  }
}

// A BM x BN tile to a workgroup of WM x WN waves, through a ring of S stages of
// 128 codes.  S fills the LDS (S = 4 against 2 at 128x128: 38 us against 60 at
// 1024x1024x8192; at 256x256 two stages are all that fit).
template <int BM, int BN, int WM, int WN, int S, int D, bool Once>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_tile(GemmArgs g, Grid gr) {
  constexpr int T = 64 * WM * WN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // 16x16 blocks of a wave
  constexpr int LA = BM * 8 / T, LB = BN * 8 / T;         // 16-byte pieces a lane loads a stage
  constexpr uint32_t kStage = (BM + BN) * 8;              // pieces of a stage
  __shared__ i32x4 lds[S * kStage];
  __shared__ float lsa[BM], lsb[BN], lbias[BN];

  const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
  uint32_t tm, tn;
  tile_of(gr, blockIdx.x, tm, tn);
  const uint32_t m0 = tm * BM, n0 = tn * BN;
  const uint32_t K16 = (g.K + 15) & ~15u;
  const uint32_t steps = (g.K + kStep - 1) / kStep;
  const bool cut_last = g.K % kStep != 0;

  const int8_t *pa = g.a + (size_t)m0 * g.lda, *pb = g.b + (size_t)n0 * g.ldb;
  // offsets of this lane's pieces in the stage at k; rows past the last one are
  // read as the last one, pieces past a row's end as its last
  uint32_t va[LA], vb[LB];
  const auto offsets = [&](uint32_t k) {
#pragma unroll
    for (int i = 0; i < LA; i++) {
      const uint32_t r = (i * T + t) / 8, c = 16 * (t % 8 ^ (r & 7));
      const uint32_t row = m0 + r < g.M ? r : g.M - 1 - m0;
      va[i] = row * (uint32_t)g.lda + (k + c < K16 ? c : K16 - 16 - k);
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
      const uint32_t r = (i * T + t) / 8, c = 16 * (t % 8 ^ ((r & 3) | (r >> 3 & 1) << 2));
      const uint32_t row = n0 + r < g.N ? r : g.N - 1 - n0;
      vb[i] = row * (uint32_t)g.ldb + (k + c < K16 ? c : K16 - 16 - k);
    }
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds +
                        wave * 1024;
  // piece-loads 0..LA+LB-1 of the stage at code k into the buffer at byte `to`
  const auto load = [&](int i, i32x4 ra, i32x4 rb, uint32_t k, uint32_t to) {
    if (i < LA) load_to_lds<false>(ra, lds0 + to + i * T * 16, va[i < LA ? i : 0], k);
    else load_to_lds<Once>(rb, lds0 + to + (BM * 8 + (i - LA) * T) * 16, vb[i < LA ? 0 : i - LA], k);
  };
  // zeros for the codes of the last stage that lie past K (of a: the products
  // with whatever b holds there are then zero)
  const auto cut_stage = [&](uint32_t at_stage) {
    const uint32_t k0 = (steps - 1) * kStep;
#pragma unroll 1
    for (uint32_t x = t; x < BM * 8; x += T) {
      const uint32_t r = x / 8, k = k0 + 16 * (t % 8 ^ (r & 7));
      i32x4* at = lds + at_stage + x;
      if (k + 16 > g.K) *at = cut(*at, k, g.K);
    }
    __syncthreads();
  };
  // waits for all but this wave's youngest loads and its LDS reads, then everyone's
  constexpr int kYoung = (S - 2) * (LA + LB);
  static_assert(kYoung + LA + LB < 64, "s_waitcnt counts to 63");
  const auto arrived = [](auto left) {
    constexpr int n = decltype(left)::value;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const uint32_t p = lane % 16, q = lane / 16;
  const uint32_t wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
  const uint32_t at = q ^ (lane & 7);
  uint32_t xa = (wm + p) * 8 + at, xb = BM * 8 + (wn + p / 4 * 8 + p % 4) * 8 + at;
  i32x4 acc[FM][FN] = {};
  i32x4 fa[2][FM], fb[2][FN];
  // fragment i of the half, of a then of b
  const auto read = [&](int half, int i) {
    if (i < FM) fa[half][i < FM ? i : 0] = lds[(xa ^ (4 * half)) + i * 128];
    else fb[half][i < FM ? 0 : i - FM] = lds[(xb ^ (4 * half)) + ((i - FM) / 2 * 32 + (i - FM) % 2 * 4) * 8];
  };
  // the products of one half, in chunks of kChunk matrix instructions, with
  // the reads of `other` and with the loads spread over them
  constexpr int kChunk = 4, kChunks = FM * FN / kChunk;
  constexpr int kReads = (2 * (FM + FN) + kChunks - 1) / kChunks;
  constexpr int kLoads = (LA + LB + kChunks - 1) / kChunks;
  const auto multiply = [&](int half, auto loads, i32x4 ra, i32x4 rb, uint32_t k, uint32_t to) {
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
#pragma unroll
      for (int r = 0; r < kReads; r++)
        if (c * kReads + r < FM + FN) read(1 - half, c * kReads + r);
      if constexpr (loads)
#pragma unroll
        for (int r = 0; r < kLoads; r++)
          if (c * kLoads + r < LA + LB) load(c * kLoads + r, ra, rb, k, to);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = c * kChunk; x < (c + 1) * kChunk; x++)
        acc[x % FM][x / FM] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            fb[half][x / FM], fa[half][x % FM], acc[x % FM][x / FM], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // the scales and the bias, for the end
  const uint16_t* bias = reinterpret_cast<const uint16_t*>(g.bias);
  for (uint32_t x = t; x < BM; x += T) lsa[x] = g.sa[m0 + x < g.M ? m0 + x : g.M - 1];
  for (uint32_t x = t; x < BN; x += T) {
    const uint32_t n = n0 + x < g.N ? n0 + x : g.N - 1;
    lsb[x] = g.sb[n];
    lbias[x] = bias ? ld16<D>(bias[n]) : 0.0f;
  }

  i32x4 ra = buffer_at(pa), rb = buffer_at(pb);
  offsets(0);
#pragma unroll
  for (uint32_t s = 0; s < S; s++) {
    if (s + 1 == steps && cut_last) offsets(s * kStep);
    end_buffer(ra, s, steps);
    end_buffer(rb, s, steps);
#pragma unroll
    for (int i = 0; i < LA + LB; i++) load(i, ra, rb, s < steps ? s * kStep : 0u, s * kStage * 16);
  }
  arrived(std::integral_constant<int, kYoung + LA + LB>{});
  if (steps == 1 && cut_last) cut_stage(0);
#pragma unroll
  for (int i = 0; i < FM + FN; i++) read(0, i);

  // One stage a turn.  Its second half is read while the first is multiplied;
  // then, with the next stage arrived and everyone done reading this one, the
  // next one's first half is read and the stage S after this one loaded over
  // it, while the second half is multiplied.
  uint32_t to = 0;                           // this stage's place, in pieces
  for (uint32_t s = 0; s < steps; s++) {
    multiply(0, std::false_type{}, ra, rb, 0, 0);
    arrived(std::integral_constant<int, kYoung>{});
    const uint32_t next = to == (S - 1) * kStage ? 0 : to + kStage;
    if (s + 2 == steps && cut_last) cut_stage(next);
    if (s + 1 + S == steps && cut_last) offsets((s + S) * kStep);
    end_buffer(ra, s + S, steps);
    end_buffer(rb, s + S, steps);
    xa += next - to;
    xb += next - to;
    multiply(1, std::true_type{}, ra, rb, s + S < steps ? (s + S) * kStep : 0u, to * 16);
    to = next;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);        // nothing may still be on its way to LDS

  // this lane holds, of token wm + 16i + p, the channels wn + 32(j/2) + 8q +
  // 4(j%2) + e: 8 neighbours for two j
  float sa[FM];
#pragma unroll
  for (int i = 0; i < FM; i++) sa[i] = lsa[wm + 16 * i + p];
#pragma unroll
  for (int j = 0; j < FN; j += 2) {
    const uint32_t x = wn + 16 * j + 8 * q;
    Channels<8> ch;
    ch.biased = bias != nullptr;
#pragma unroll
    for (int e = 0; e < 8; e++) ch.sb[e] = lsb[x + e];
#pragma unroll
    for (int e = 0; e < 8; e++) ch.bias[e] = lbias[x + e];
#pragma unroll
    for (int i = 0; i < FM; i++) {
      const uint32_t m = m0 + wm + 16 * i + p;
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        w[e / 2] = st16x2<D>(ch.value(acc[i][j][e], sa[i], e),
                             ch.value(acc[i][j][e + 1], sa[i], e + 1));
        w[2 + e / 2] = st16x2<D>(ch.value(acc[i][j + 1][e], sa[i], 4 + e),
                                 ch.value(acc[i][j + 1][e + 1], sa[i], 5 + e));
      }
      if (m < g.M) store_row<8>(g, m, n0 + x, w);
    }
  }
}

// A block of BM tokens by BN channels to a workgroup, whose W waves share the
// sum: wave w takes stages w, w + W, ... through a ring of S stages of its own
// in LDS, so the waves wait for nothing but their own loads until the end.
// Neighbouring tiles start kApart stages apart: all at once they would ask for
// the same lines of a, and for lines of b a power of two apart, which few of the
// caches' and the memory's channels hold.  Cold weights, 16384x4096, us: one
// token 12.2, started together 13.5; 16 tokens 14.0 and 15.7; 48 tokens 15.9 and
// 17.3.  7, 9 or 13 stages apart come out within 4% of 2 there; at 8192x8192,
// one token: 12.1 with 2, 12.4 with 7, 13.2 together.  k_tile starts its tiles
// together: apart, a stage takes 396 ns instead of 365 at 64x128, 597 instead of
// 557 at 128x128, and 1562 instead of 1661 at 256x256.
constexpr uint32_t kApart = 2;

template <int BM, int BN, int W, int S, int D, bool Once>
__global__ __launch_bounds__(64 * W) void k_split(GemmArgs g, Grid gr) {
  constexpr int FM = (BM + 15) / 16, FN = BN / 16;
  constexpr int LA = BM / 8, LB = BN / 8, L = LA + LB;    // loads of a stage
  constexpr uint32_t kStage = (BM + BN) * 8;              // pieces of a stage
  static_assert(FM * FN * 64 <= S * kStage && (S - 1) * L < 64);
  __shared__ i32x4 lds[W * S * kStage];
  const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
  uint32_t tm, tn;
  tile_of(gr, blockIdx.x, tm, tn);
  const uint32_t m0 = tm * BM, n0 = tn * BN;
  const uint32_t K16 = (g.K + 15) & ~15u;
  const uint32_t steps = (g.K + kStep - 1) / kStep;
  const bool cut_last = g.K % kStep != 0;
  const int8_t *pa = g.a + (size_t)m0 * g.lda, *pb = g.b + (size_t)n0 * g.ldb;
  uint32_t va[LA], vb[LB];
  const auto offsets = [&](uint32_t k) {
    const uint32_t c = 16 * (lane % 8 ^ lane / 8), at = k + c < K16 ? c : K16 - 16 - k;
#pragma unroll
    for (int i = 0; i < LA; i++) {
      const uint32_t r = i * 8 + lane / 8;
      va[i] = (m0 + r < g.M ? r : g.M - 1 - m0) * (uint32_t)g.lda + at;
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
      const uint32_t r = i * 8 + lane / 8;
      vb[i] = (n0 + r < g.N ? r : g.N - 1 - n0) * (uint32_t)g.ldb + at;
    }
  };
  i32x4* const ring = lds + wave * S * kStage;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds +
                         wave * S * kStage * 16;
  i32x4 ra = buffer_at(pa), rb = buffer_at(pb);
  // stage s into slot `to`; past the last stage from an empty buffer, from
  // which nothing is fetched
  const uint32_t rest = steps > 1 ? steps - 1 : 1;        // the last one stays last
  const uint32_t turn = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tn * kApart % rest));
  const auto load = [&](uint32_t s, uint32_t to) {
    uint32_t at = s + turn < rest ? s + turn : s + turn - rest;
    if (s + 1 >= steps) at = s < steps ? s : 0;
    const uint32_t k = at * kStep;
    end_buffer(ra, s, steps);
    end_buffer(rb, s, steps);
    if (s + 1 == steps && cut_last) offsets(k);
#pragma unroll
    for (int i = 0; i < LB; i++)
      load_to_lds<Once>(rb, ring0 + (to * kStage + BM * 8 + i * 64) * 16, vb[i], k);
#pragma unroll
    for (int i = 0; i < LA; i++)
      load_to_lds<false>(ra, ring0 + (to * kStage + i * 64) * 16, va[i], k);
  };
  const uint32_t p = lane % 16, q = lane / 16;
  const uint32_t x0 = p * 8 + (q ^ (p & 7)), xa = BM < 16 ? x0 & 63 : x0;
  i32x4 acc[FM][FN] = {};
  offsets(0);
#pragma unroll
  for (uint32_t i = 0; i < S; i++) load(wave + i * W, i);
  uint32_t to = 0;
#pragma unroll 1
  for (uint32_t s = wave; s < steps; s += W) {
    constexpr int n = (S - 1) * L;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 0x0f70);
    asm volatile("" ::: "memory");
    i32x4* const at = ring + to * kStage;
    if (s + 1 == steps && cut_last) {
      // zeros for the codes of a past K
#pragma unroll
      for (int i = 0; i < LA; i++) {
        const uint32_t k = s * kStep + 16 * (lane % 8 ^ lane / 8);
        if (k + 16 > g.K) at[i * 64 + lane] = cut(at[i * 64 + lane], k, g.K);
      }
    }
    i32x4 fa[2][FM], fb[2][FN];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int j = 0; j < FN; j++) fb[h][j] = at[BM * 8 + j * 128 + (x0 ^ (4 * h))];
#pragma unroll
      for (int i = 0; i < FM; i++) fa[h][i] = at[i * 128 + (xa ^ (4 * h))];
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);      // the slot is read: it may be loaded again
    asm volatile("" ::: "memory");
    load(s + S * W, to);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
    to = to + 1 == S ? 0 : to + 1;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);        // nothing may still be on its way to LDS
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) ring[(i * FN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (uint32_t x = t; x < FM * FN * 64; x += 64 * W) finish<D, BM, W, FN, S * kStage>(g, m0, n0, x, lds);
}

// Weights that one row of tiles covers are read by one workgroup only, and a
// model's weights do not stay in the 256 MB cache until they are used again:
// past the caches, one token over cold 8192x8192 weights takes 13.1 us instead
// of 15.4, 8192x4096 8.3 instead of 9.5, 48 tokens 11.9 instead of 12.6 (before
// the tiles' starts were set apart, k_split).  Where the same 67 MB are read
// again and again it costs 12.3 against 11.5.
template <int I>
hipError_t launch_tile(int dtype, const GemmArgs& g, hipStream_t st) {
  constexpr Tile t = kTiles[I];
  const Grid gr{tile_rows(t, g.M), (g.N + t.bn - 1) / t.bn, t.group};
  const dim3 grid(gr.tm * gr.tn), block(64 * t.wm * (t.wn ? t.wn : 1));
  const auto kernel = [&](auto d, auto once) {
    constexpr int D = decltype(d)::value;
    constexpr bool Once = decltype(once)::value;
    if constexpr (t.wn == 0) k_split<t.bm, t.bn, t.wm, t.stages, D, Once><<<grid, block, 0, st>>>(g, gr);
    else k_tile<t.bm, t.bn, t.wm, t.wn, t.stages, D, Once><<<grid, block, 0, st>>>(g, gr);
  };
  const auto of_type = [&](auto d) {
    if constexpr (t.bm <= 8) kernel(d, std::true_type{});    // never more tokens
    else if (gr.tm == 1) kernel(d, std::true_type{});
    else kernel(d, std::false_type{});
  };
  if (dtype == kF16) of_type(std::integral_constant<int, kF16>{});
  else of_type(std::integral_constant<int, kBF16>{});
  return hipGetLastError();
}

using Launch = hipError_t (*)(int, const GemmArgs&, hipStream_t);
template <int... I>
Launch launch_of(int tile, std::integer_sequence<int, I...>) {
  static constexpr Launch table[] = {launch_tile<I>...};
  return table[tile];
}

}  // namespace

hipError_t launch_gemm(int dtype, const GemmArgs& g, hipStream_t st) {
  return launch_of(choose_tile(g.M, g.N, g.K),
                   std::make_integer_sequence<int, kTileCount>{})(dtype, g, st);
}

}  // namespace qr
