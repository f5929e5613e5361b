// qr_gemm.hip -- gfx950 kernels of qr_gemm_i8 (include/qr_layer.h): the matrix
// product of 8-bit codes with a scale for each token and each output channel.
#include <type_traits>

#include "qr.h"
#include "qr_device.h"
#include "qr_layer_internal.h"

namespace qr {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kStep = 128;       // codes of the sum in one stage of the tile kernel

// 16 bytes from base + voff + soff to LDS byte lds + 16*lane, for every lane of
// the wave, without passing through registers; s_waitcnt vmcnt covers it.  In
// assembly since the compiler, where it cannot tell two LDS buffers apart,
// would wait for the load before any LDS read: the caller waits.  It has no
// output register, so nothing is written behind the compiler's back but LDS.
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t lds, uint32_t voff,
                                            uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory");
}
__device__ __forceinline__ i32x4 buffer_at(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  const int lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const int hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xffff;
  return i32x4{lo, hi, __builtin_amdgcn_readfirstlane((int)bytes), 0x00027000};
}

// The 16-byte piece v of a row, which starts at code k, with zeros past K.
__device__ __forceinline__ i32x4 cut(i32x4 v, uint32_t k, uint32_t K) {
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const int left = (int)(K - k) - 4 * w;               // bytes of word w inside the row
    v[w] = left >= 4 ? v[w] : left <= 0 ? 0 : (int)((uint32_t)v[w] & ((1u << (8 * left)) - 1u));
  }
  return v;
}

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

// W/2 words of 16-bit values to c[m][n..]: one store inside the row
template <int W, class V>
__device__ __forceinline__ void store_row(const GemmArgs& g, uint32_t m, uint32_t n, const V& w) {
  uint16_t* c = reinterpret_cast<uint16_t*>(g.c) + (size_t)m * g.ldc + n;
  if (n + W <= g.N) {
    __builtin_memcpy(c, &w, 2 * W);
  } else {
#pragma unroll 1
    for (uint32_t e = 0; n + e < g.N; e++) {
      uint32_t x = w[0];
#pragma unroll
      for (uint32_t k = 1; k < W / 2; k++) x = e / 2 == k ? w[k] : x;
      c[e] = (uint16_t)(x >> (16 * (e % 2)));
    }
  }
}

// order of the tiles: see tile_of
struct Grid {
  uint32_t tm, tn, group;             // tiles along M and N; tile rows of a group
};

__device__ __forceinline__ void tile_of(const Grid& gr, uint32_t b, uint32_t& m, uint32_t& n) {
  const uint32_t total = gr.tm * gr.tn, per = total / 8, extra = total % 8;
  const uint32_t x = b % 8, i = b / 8;
  const uint32_t t = x * per + (x < extra ? x : extra) + i;
  const uint32_t g = t / (gr.group * gr.tn), r = t % (gr.group * gr.tn);
  const uint32_t m0 = g * gr.group;
  const uint32_t rows = gr.tm - m0 < gr.group ? gr.tm - m0 : gr.group;
  m = m0 + r % rows;
  n = r / rows;
}

template <int BM, int BN, int WM, int WN, int D>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_tile(GemmArgs g, Grid gr) {
  constexpr int T = 64 * WM * WN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // 16x16 blocks of a wave
  constexpr int LA = BM * 8 / T, LB = BN * 8 / T;         // 16-byte pieces a lane loads a stage
  constexpr uint32_t kStage = (BM + BN) * 8;              // pieces of a stage
  __shared__ i32x4 lds[2 * kStage];
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
    if (i < LA) load_to_lds(ra, lds0 + to + i * T * 16, va[i < LA ? i : 0], k);
    else load_to_lds(rb, lds0 + to + (BM * 8 + (i - LA) * T) * 16, vb[i < LA ? 0 : i - LA], k);
  };
  // zeros for the codes of the last stage that lie past K (of a: the products
  // with whatever b holds there are then zero)
  const auto cut_stage = [&](uint32_t parity) {
    const uint32_t k0 = (steps - 1) * kStep;
#pragma unroll 1
    for (uint32_t x = t; x < BM * 8; x += T) {
      const uint32_t r = x / 8, k = k0 + 16 * (t % 8 ^ (r & 7));
      i32x4* at = lds + parity * kStage + x;
      if (k + 16 > g.K) *at = cut(*at, k, g.K);
    }
    __syncthreads();
  };
  const auto arrived = [] {                  // this wave's loads and LDS reads, then everyone's
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);
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

  const i32x4 ra = buffer_at(pa, ~0u), rb = buffer_at(pb, ~0u);
  offsets(0);
#pragma unroll
  for (int i = 0; i < LA + LB; i++) load(i, ra, rb, 0, 0);
  arrived();
  if (steps == 1 && cut_last) cut_stage(0);
  if (steps > 1) {
    if (steps == 2 && cut_last) offsets(kStep);
#pragma unroll
    for (int i = 0; i < LA + LB; i++) load(i, ra, rb, kStep, kStage * 16);
  }
#pragma unroll
  for (int i = 0; i < FM + FN; i++) read(0, i);

  // One stage a turn.  Its second half is read while the first is multiplied;
  // then, with the next stage arrived and everyone done reading this one, the
  // next one's first half is read and the stage after it loaded over this one,
  // while the second half is multiplied.
  uint32_t to = 0;                           // byte offset of this stage's buffer
  for (uint32_t s = 0; s < steps; s++) {
    multiply(0, std::false_type{}, ra, rb, 0, 0);
    arrived();
    if (s + 2 == steps && cut_last) cut_stage(1 - s % 2);
    if (s + 3 == steps && cut_last) offsets((s + 2) * kStep);
    // past the last stage: an empty buffer, from which nothing is fetched
    const bool more = s + 2 < steps;
    const i32x4 ma = buffer_at(pa, more ? ~0u : 0u), mb = buffer_at(pb, more ? ~0u : 0u);
    const uint32_t k = more ? (s + 2) * kStep : 0u;
    xa = to ? xa - kStage : xa + kStage;
    xb = to ? xb - kStage : xb + kStage;
    multiply(1, std::true_type{}, ma, mb, k, to);
    to = kStage * 16 - to;
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

// bytes [k, k+16) of a row, zeros past K; rows are readable up to K16
__device__ __forceinline__ i32x4 load_cut(const int8_t* row, uint32_t k, uint32_t K) {
  if (k >= K) return i32x4{0, 0, 0, 0};
  return cut(*reinterpret_cast<const i32x4*>(row + k), k, K);
}

// M <= 16*MT tokens; a workgroup's eight waves share the sum of 16*NT channels
template <int MT, int NT, int U, int D>
__global__ __launch_bounds__(512) void k_few(GemmArgs g) {
  constexpr int W = 8;
  __shared__ i32x4 part[W][MT * NT][64];
  const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
  const uint32_t p = lane % 16, q = lane / 16, n0 = blockIdx.x * 16 * NT;
  const int8_t *pa[MT], *pb[NT];
#pragma unroll
  for (int i = 0; i < MT; i++)
    pa[i] = g.a + (size_t)(16 * i + p < g.M ? 16 * i + p : g.M - 1) * g.lda;
#pragma unroll
  for (int j = 0; j < NT; j++)
    pb[j] = g.b + (size_t)(n0 + 16 * j + p < g.N ? n0 + 16 * j + p : g.N - 1) * g.ldb;
  i32x4 acc[MT][NT] = {};
  const uint32_t groups = g.K / (64 * U);
  for (uint32_t s = wave; s < groups; s += W) {
    i32x4 fa[U][MT], fb[U][NT];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t k = (s * U + u) * 64 + 16 * q;
#pragma unroll
      for (int j = 0; j < NT; j++)
        fb[u][j] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb[j] + k));
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t k = (s * U + u) * 64 + 16 * q;
#pragma unroll
      for (int i = 0; i < MT; i++) fa[u][i] = *reinterpret_cast<const i32x4*>(pa[i] + k);
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][j], fa[u][i], acc[i][j], 0, 0, 0);
  }
  // at most U pieces of 64 codes are left, one to a wave
  const uint32_t k0 = groups * U * 64 + wave * 64;
  if (k0 < g.K) {
    const uint32_t k = k0 + 16 * q;
    i32x4 fa[MT], fb[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) fb[j] = load_cut(pb[j], k, g.K);
#pragma unroll
    for (int i = 0; i < MT; i++) fa[i] = load_cut(pa[i], k, g.K);
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int j = 0; j < NT; j++)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (uint32_t x = t; x < MT * NT * 64; x += 512) {
    const uint32_t f = x / 64, m = f / NT * 16 + x % 16, n = n0 + f % NT * 16 + x % 64 / 16 * 4;
    i32x4 sum = part[0][f][x % 64];
#pragma unroll
    for (int w = 1; w < W; w++) sum += part[w][f][x % 64];
    if (m < g.M && n < g.N) {
      const Channels<4> ch = channels<D, 4>(g, n);
      const float sa = g.sa[m];
      u32x2 w;
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        w[e / 2] = st16x2<D>(ch.value(sum[e], sa, e), ch.value(sum[e + 1], sa, e + 1));
      store_row<4>(g, m, n, w);
    }
  }
}

template <int BM, int BN, int WM, int WN>
hipError_t tiles(int dtype, const GemmArgs& g, uint32_t group, hipStream_t st) {
  const Grid gr{(g.M + BM - 1) / BM, (g.N + BN - 1) / BN, group};
  const dim3 grid(gr.tm * gr.tn), block(64 * WM * WN);
  if (dtype == kF16) k_tile<BM, BN, WM, WN, kF16><<<grid, block, 0, st>>>(g, gr);
  else k_tile<BM, BN, WM, WN, kBF16><<<grid, block, 0, st>>>(g, gr);
  return hipGetLastError();
}

template <int MT, int NT, int U>
hipError_t few(int dtype, const GemmArgs& g, hipStream_t st) {
  const dim3 grid((g.N + 16 * NT - 1) / (16 * NT));
  if (dtype == kF16) k_few<MT, NT, U, kF16><<<grid, 512, 0, st>>>(g);
  else k_few<MT, NT, U, kBF16><<<grid, 512, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace

size_t gemm_workspace_bytes(size_t, size_t, size_t) { return 0; }

hipError_t launch_gemm(int dtype, const GemmArgs& g, hipStream_t st) {
  if (g.M <= 16) return few<1, 1, 4>(dtype, g, st);
  if (g.M <= 32) return few<2, 2, 4>(dtype, g, st);
  if (g.M <= 64) return few<4, 2, 4>(dtype, g, st);
  const size_t big = (size_t)((g.M + 255) / 256) * ((g.N + 255) / 256);
  if (big >= 256) return tiles<256, 256, 2, 4>(dtype, g, 4, st);
  return tiles<128, 128, 2, 2>(dtype, g, 8, st);
}

}  // namespace qr
