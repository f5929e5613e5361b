// qr_gemm_f8.hip -- gfx950 kernels of qr_gemm_f8 and qr_gemm_f8_grouped
// (include/qr_f8.h): matrix products of E4M3FN codes with a scale for each block
// of 128, the tokens in one group or grouped by expert.
//
// c = sum_kb (sum_{k in kb} a[m][k] * b[n][k]) * (sa[m][kb] * sb[n/128][kb]) + bias.
// A block's sum is one matrix instruction (16x16x128, 32 cycles): it starts from
// zero, and its four results a lane are multiplied by the token's scale times the
// weights' block scale and added to binary32 sums with one fused multiply-add each,
// while the matrix unit works on the next (33.7 cycles a product with them, from
// registers).  Stages of the sum are therefore blocks.  Loads, rings, swizzle and
// the two kernels (k_split, k_tile) are as in qr_gemm.hip; the tokens' and the
// weights' scales pass through LDS beside the codes (of k_split the weights'
// through the scalar cache).
//
// The one rounding to fewer than 32 bits is c's; the matrix unit's own cut of the
// products is in include/qr_f8.h.
//
// By experts: the grid has a workgroup for every tile that there may be; each
// finds its expert and rows from the offsets.  Nothing is read back by the host.
//
// Measured (cold weights; a copy reaches 5.2 TB/s, plain reads 6.8, a library
// product of 8192^3 such codes with one scale for all 355 to 418 us):
//   1 token, 8192 x 8192       12 to 14 us, 4.8 to 5.6 TB/s: the weights' bytes
//   8192^3, bias               435 to 480 us on several cards, 2.29 to 2.53 PFLOP/s;
//                              (the library's 382 where this took 447); the
//                              matrix units are busy 65% of the time
//   16 tokens over 4 of 32 experts of 2048 x 8192   69 us, 6.6 TB/s of the 454 MB
//                              of the 27 experts hit (63 with some in the cache)
//   4096 tokens over 8 of 64 experts of 8192 x 1024   455 to 510 us, 1.1 to 1.2
//                              PFLOP/s, 2.4 TB/s: sums of 8 blocks, between which a
//                              CU loads its first stage and writes 128 KB of c with
//                              its matrix units idle (35% busy)
#include <type_traits>
#include <utility>

#include "qr_f8.h"
#include "qr_f8_internal.h"
#include "qr_gemm_device.h"
#include "qr_gemm_f8_tiles.h"

namespace qr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// 4 bytes a lane, as load_to_lds
__device__ __forceinline__ void load_word_to_lds(i32x4 rsrc, uint32_t lds, uint32_t voff,
                                                 uint32_t soff) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "{m0}"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
}

// The compiler may move what makes v no further down than here.  Left alone it
// gathers the additions of a whole stage behind its last product, with all the
// products' results held until then (256x256: 128 registers spilled).
__device__ __forceinline__ void here(f32x4& v) { asm volatile("" : "+v"(v)); }

// 16x16 sums over the 128 codes of a block
__device__ __forceinline__ f32x4 block_sum(const i32x4 (&b)[2], const i32x4 (&a)[2]) {
  const i32x8 x = __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7);
  const i32x8 y = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0,
                                                          0, 0, 0, 0);
}
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& d, float s) {
#pragma unroll
  for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(d[e], s, acc[e]);
}

typedef const __attribute__((address_space(4))) float* ConstF;
__device__ __forceinline__ ConstF constant(const float* p) {
  return (ConstF)(uintptr_t)p;
}

// what a workgroup works on
struct Job {
  uint32_t m0, end;                   // its first row, and the end of its expert's rows
  uint32_t n0;
  const uint8_t* b;
  const float* sb;
  const uint8_t* bias;
};

// Rows [lo, hi) of expert e.  Offsets are taken into 0..M, falling ones as equal.
__device__ __forceinline__ void rows_of(const F8Args& g, uint32_t e, uint32_t& lo, uint32_t& hi) {
  const int32_t x = g.offsets[e], y = g.offsets[e + 1], M = (int32_t)g.M;
  const int32_t l = x < 0 ? 0 : x > M ? M : x, h = y < l ? l : y > M ? M : y;
  lo = (uint32_t)l;
  hi = (uint32_t)h;
}

// false: there is no such tile.  Every wave adds up the experts' tiles by itself,
// 64 experts at a time.
template <uint32_t BM, uint32_t BN, bool Grouped>
__device__ __forceinline__ bool find_job(const F8Args& g, Grid gr, Job& job) {
  uint32_t tm, tn;
  job = Job{0, g.M, 0, g.b, g.sb, g.bias};
  if constexpr (!Grouped) {
    tile_of(gr, blockIdx.x, tm, tn);
    job.m0 = tm * BM;
  } else {
    const uint32_t lane = threadIdx.x % 64;
    const auto tiles_up_to = [&](uint32_t e0, uint32_t& lo, uint32_t& hi) {
      lo = hi = 0;
      if (e0 + lane < g.E) rows_of(g, e0 + lane, lo, hi);
      uint32_t n = (hi - lo + BM - 1) / BM;
#pragma unroll
      for (uint32_t d = 1; d < 64; d *= 2) {
        const uint32_t up = (uint32_t)__shfl_up((int)n, d);
        if (lane >= d) n += up;
      }
      return n;
    };
    const auto at = [](uint32_t v, uint32_t from) {
      return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)from);
    };
    uint32_t lo, hi, n = tiles_up_to(0, lo, hi), total = at(n, 63), e0 = 0;
    for (uint32_t e = 64; e < g.E; e += 64) {
      uint32_t l, h;
      total += at(tiles_up_to(e, l, h), 63);
    }
    // offsets that fall back again and again could ask for more than there are
    total = total < gr.tm ? total : gr.tm;
    if (blockIdx.x >= total * gr.tn) return false;
    // experts one after another, each in groups of its own rows, so that most
    // weights are fetched once (8192 x 1024 of 64 experts with 512 rows each: 689 MB
    // fetched, 861 where groups cross experts; 2048 x 4096 with 32 rows each 130 us
    // instead of 143)
    const uint32_t t = tile_number(total * gr.tn, blockIdx.x);
    uint32_t before = t / gr.tn;
    while (before >= at(n, 63)) {          // ends: before < total
      before -= at(n, 63);
      e0 += 64;
      n = tiles_up_to(e0, lo, hi);
    }
    const uint32_t in = (uint32_t)__builtin_ctzll(__ballot(n > before));
    const uint32_t first = in == 0 ? 0 : at(n, in - 1);
    gr.tm = at(n, in) - first;
    tile_at(gr, (before - first) * gr.tn + t % gr.tn, tm, tn);
    job.m0 = at(lo, in) + tm * BM;
    job.end = at(hi, in);
    const size_t e = e0 + in;
    job.b += e * g.gb;
    job.sb += e * g.gsb;
    if (job.bias) job.bias += 2 * e * g.ldbias;
  }
  job.n0 = tn * BN;
  return true;
}

// Where row m of a product lies in a: its number, counted from a's start (by
// index) or from the tile's first row.  Rows past the last one are read as the
// last one, an index outside a as row 0; what they give is not written.
template <bool Grouped>
__device__ __forceinline__ uint32_t row_of(const F8Args& g, const Job& job, uint32_t r) {
  const uint32_t m = job.m0 + r < job.end ? job.m0 + r : job.end - 1;
  if (Grouped && g.rows) {
    const uint32_t at = (uint32_t)g.rows[m];
    return at < g.tokens ? at : 0u;
  }
  return m - job.m0;
}
// whether row m of c takes a row of a
template <bool Grouped>
__device__ __forceinline__ bool real_row(const F8Args& g, uint32_t m) {
  return !Grouped || !g.rows || (uint32_t)g.rows[m] < g.tokens;
}
template <bool Grouped>
__device__ __forceinline__ size_t first_row(const F8Args& g, const Job& job) {
  return Grouped && g.rows ? 0 : job.m0;
}

// A BM x BN tile to a workgroup of WM x WN waves, through a ring of S stages of
// one block each.  Bound by the loads to LDS up to 128 x 128 (60 bytes/ns a CU), at
// 256 x 256 by the matrix units, and by its ends where sums are short: a tile of 256
// x 256 takes 1.67 us a block and 9 us besides (8192 x 8192: K = 512 63 us, K = 8192
// 465 on the same card).  128 x 256 spills 2 of its 256 registers, outside the stages;
// no other tile spills any.
//
// The tokens' scales come 8 blocks at a time (two 16-byte pieces a row), one load
// a lane, into the one of two buffers that is not in use.
template <int BM, int BN, int WM, int WN, int S, int D, bool Once, bool Grouped>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_tile_f8(F8Args g, Grid gr) {
  constexpr int T = 64 * WM * WN;
  constexpr bool Turns = S == 2 && T == 512;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // 16x16 blocks of a wave
  constexpr int LA = BM * 8 / T, LB = BN * 8 / T;         // 16-byte pieces a lane loads a stage
  constexpr uint32_t kStage = (BM + BN) * 8;              // pieces of a stage
  constexpr uint32_t kChunk = 8;                          // blocks whose scales come together
  static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0 && BM * 2 <= T);
  __shared__ i32x4 lds[S * kStage];
  __shared__ __attribute__((aligned(16))) float lsa[2][BM * kChunk];
  __shared__ float lsb[2][T], lbias[BN];

  const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
  Job job;
  if (!find_job<BM, BN, Grouped>(g, gr, job)) return;
  const uint32_t m0 = job.m0, n0 = job.n0;
  const uint32_t K16 = (g.K + 15) & ~15u;
  const uint32_t steps = (g.K + kF8Step - 1) / kF8Step;
  const bool cut_last = g.K % kF8Step != 0;

  // offsets of this lane's pieces in the stage at k; rows past the last one are
  // read as the last one, pieces past a row's end as its last
  uint32_t ra0[LA], va[LA], vb[LB];
#pragma unroll
  for (int i = 0; i < LA; i++) ra0[i] = row_of<Grouped>(g, job, (i * T + t) / 8) * (uint32_t)g.lda;
  const auto offsets = [&](uint32_t k) {
#pragma unroll
    for (int i = 0; i < LA; i++) {
      const uint32_t r = (i * T + t) / 8, c = 16 * (t % 8 ^ (r & 7));
      va[i] = ra0[i] + (k + c < K16 ? c : K16 - 16 - k);
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
      const uint32_t r = (i * T + t) / 8, c = 16 * (t % 8 ^ ((r & 3) | (r >> 3 & 1) << 2));
      const uint32_t row = n0 + r < g.N ? r : g.N - 1 - n0;
      vb[i] = row * (uint32_t)g.ldb + (k + c < K16 ? c : K16 - 16 - k);
    }
  };
  // Scales: place x of a row holds its piece x ^ (row / 8 & 1), so that 16 rows'
  // scales of a block lie in 16 banks; lanes beyond the rows load what others load,
  // to the same place.
  const uint32_t srow = t / 2 % BM, spiece = (t ^ srow / 8) & 1;
  const uint32_t vs = row_of<Grouped>(g, job, srow) * (uint32_t)g.ldsa * 4;
  const uint32_t last_piece = (steps + 3) / 4 - 1;
  const auto lds_at = [](const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
  };
  const uint32_t lds0 = lds_at(lds) + wave * 1024;
  const uint32_t lsa0 = lds_at(lsa) + wave * 1024 % (BM * kChunk * 4);
  const auto load_scales = [&](i32x4 rs, uint32_t chunk) {
    const uint32_t piece = 2 * chunk + spiece;
    load_to_lds<false>(rs, lsa0 + (chunk & 1) * (BM * kChunk * 4),
                       vs + 16 * (piece < last_piece ? piece : last_piece), 0);
  };
  // piece-loads 0..LA+LB-1 of the stage at code k into the buffer at byte `to`
  const auto load = [&](int i, i32x4 ra, i32x4 rb, uint32_t k, uint32_t to) {
    if (i < LA) load_to_lds<false>(ra, lds0 + to + i * T * 16, va[i < LA ? i : 0], k);
    else load_to_lds<Once>(rb, lds0 + to + (BM * 8 + (i - LA) * T) * 16, vb[i < LA ? 0 : i - LA], k);
  };
  // zeros for the codes of the last stage that lie past K, of a and b: either may
  // hold NaN codes there.  Every lane's own pieces, once they have arrived.
  const auto cut_stage = [&](uint32_t at_stage) {
    const uint32_t k0 = (steps - 1) * kF8Step;
#pragma unroll
    for (int i = 0; i < LA + LB; i++) {
      const uint32_t r = ((i < LA ? i : i - LA) * T + t) / 8;
      const uint32_t k = k0 + 16 * (t % 8 ^ (i < LA ? r & 7 : (r & 3) | (r >> 3 & 1) << 2));
      i32x4* at = lds + at_stage + i * T + t;
      if (k + 16 > g.K) *at = cut(*at, k, g.K);
    }
  };
  // waits for all but this wave's youngest `left` loads
  const auto arrived = [](auto left) {
    constexpr int n = decltype(left)::value;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 0x0f70);
    asm volatile("" ::: "memory");
  };
  // for everyone, with this wave's LDS reads and writes done
  const auto together = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr int L = LA + LB, kYoung = (S - 2) * L, kEarly = LA + LB / 2;
  static_assert(kYoung + L < 64, "s_waitcnt counts to 63");

  const uint32_t p = lane % 16, q = lane / 16;
  const uint32_t wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
  const uint32_t at = q ^ (lane & 7);
  uint32_t xa = (wm + p) * 8 + at, xb = BM * 8 + (wn + p / 4 * 8 + p % 4) * 8 + at;
  constexpr int kHeld = Turns ? FN / 2 : FN;  // columns whose codes are held
  constexpr int kSets = Turns ? 1 : 2;
  f32x4 acc[FM][FN] = {};
  i32x4 fa[kSets][FM][2], fb[kSets][kHeld][2];
  float s[FM] = {}, sa[kSets][FM];
  const auto read_a = [&](int set, int i) {
#pragma unroll
    for (int h = 0; h < 2; h++) fa[set][i][h] = lds[(xa ^ (4 * h)) + i * 128];
  };
  const auto read_b = [&](int set, int j) {
#pragma unroll
    for (int h = 0; h < 2; h++)
      fb[set][j % kHeld][h] = lds[(xb ^ (4 * h)) + (j / 2 * 32 + j % 2 * 4) * 8];
  };
  // the tokens' scales of a block
  const auto read_scales = [&](int set, uint32_t step) {
    const float* const from = lsa[step / kChunk & 1] + (wm + p) * kChunk +
                              ((step % kChunk / 4 ^ p / 8) & 1) * 4 + step % 4;
#pragma unroll
    for (int i = 0; i < FM; i++) sa[set][i] = from[i * 16 * kChunk];
  };
  // The weights' scales of this wave's channels, 64 blocks at a time: a word a
  // lane, in a place of the wave's own.
  const uint32_t nb = (n0 + wn < g.N ? n0 + wn : g.N - 1) / 128;
  const i32x4 rsb = buffer_at(job.sb + (size_t)nb * g.ldsb);
  const auto load_sb = [&](uint32_t from) {
    const uint32_t at = from + lane < steps ? from + lane : steps - 1;
    load_word_to_lds(rsb, lds_at(lsb) + (from / 64 & 1) * (T * 4) + wave * 256, 4 * at, 0);
  };
  const auto read_sb = [&](uint32_t step) { return lsb[step / 64 & 1][wave * 64 + step % 64]; };

  // the bias, for the end
  const uint16_t* bias = reinterpret_cast<const uint16_t*>(job.bias);
  for (uint32_t x = t; x < BN; x += T)
    lbias[x] = bias ? ld16<D>(bias[n0 + x < g.N ? n0 + x : g.N - 1]) : 0.0f;

  const size_t from = first_row<Grouped>(g, job);
  i32x4 ra = buffer_at(g.a + from * g.lda), rb = buffer_at(job.b + (size_t)n0 * g.ldb);
  const i32x4 rs = buffer_at(g.sa + from * g.ldsa);
  load_scales(rs, 0);
  load_scales(rs, 1);
  load_sb(0);
  load_sb(64);
  offsets(0);
#pragma unroll
  for (uint32_t s = 0; s < S; s++) {
    if (s + 1 == steps && cut_last) offsets(s * kF8Step);
    end_buffer(ra, s, steps);
    end_buffer(rb, s, steps);
#pragma unroll
    for (int i = 0; i < L; i++)
      if (!Turns || s == 0 || i < LA || (i - LA) % 2 == 0)
        load(i, ra, rb, s < steps ? s * kF8Step : 0u, s * kStage * 16);
  }
  arrived(std::integral_constant<int, Turns ? kEarly : kYoung + L>{});
  if (steps == 1 && cut_last) cut_stage(0);
  together();

  constexpr int kProducts = FM * FN, kLag = 2;
  uint32_t to = 0;                           // this stage's place, in pieces
  if constexpr (Turns) {
    // The two waves of a SIMD take turns: while one multiplies half a stage, the
    // other reads the codes of its own next half and issues its loads, which would
    // hold up the products (a turn of 16 products took 790 cycles with two loads
    // among them, 940 with six, and takes 540 by itself).  Waves 4 to 7 are one turn
    // behind: counting from the first waves' first reads of a stage, it is read in
    // turns 0 to 3, all of a and the first half of b (kEarly loads: of every 128
    // channels the first 64) in turns 0 and 1.  Over these the stage after the next
    // is loaded in turns 2 and 3, over the second half of b in turns 4 and 5; it has
    // arrived at the end of turn 7.
    const bool late = wave >= WM * WN / 2;
    f32x4 d[4] = {};
    // the x-th product of a stage, and the one before the last added to its sum
    const auto multiply = [&](int x) {
      d[x % 4] = block_sum(fb[0][x / FM % kHeld], fa[0][x % FM]);
      __builtin_amdgcn_sched_barrier(0);
    };
    const auto add = [&](int x) {
      add_scaled(acc[x % FM][x / FM], d[x % 4], s[x % FM]);
      here(acc[x % FM][x / FM]);
    };
    // loads n0 to n1 of `stage`
    const auto load_part = [&](int n0, int n1, uint32_t stage) {
      if (n0 == 0 && stage + 1 == steps && cut_last) offsets(stage * kF8Step);
      end_buffer(ra, stage, steps);
      end_buffer(rb, stage, steps);
#pragma unroll
      for (int n = n0; n < n1; n++) {
        const int i = n < LA ? n : n < kEarly ? LA + 2 * (n - LA) : LA + 1 + 2 * (n - kEarly);
        load(i, ra, rb, stage < steps ? stage * kF8Step : 0u, stage % 2 * kStage * 16);
      }
    };
    const auto stage_arrived = [&](uint32_t stage) {
      arrived(std::integral_constant<int, kEarly>{});
      if (stage + 1 == steps && cut_last) cut_stage(stage % 2 * kStage);
    };
    const auto turn = [&](int half) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int y = 0; y < kProducts / 2; y++) {
        const int x = half * (kProducts / 2) + y;
        __builtin_amdgcn_sched_barrier(0);
        multiply(x);
        if (y >= kLag) add(x - kLag);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    if (late) together();
#pragma unroll 1
    for (uint32_t step = 0; step < steps; step++) {
      const float sb = read_sb(step);
#pragma unroll
      for (int j = 0; j < FN / 2; j++) read_b(0, j);
#pragma unroll
      for (int i = 0; i < FM; i++) read_a(0, i);
      read_scales(0, step);
      __builtin_amdgcn_sched_barrier(0);
      load_part(kEarly, L, step + 1);
#pragma unroll
      for (int x = kProducts - kLag; x < kProducts; x++) add(x);
      together();
#pragma unroll
      for (int i = 0; i < FM; i++) s[i] = sa[0][i] * sb;
      turn(0);
      together();
#pragma unroll
      for (int j = FN / 2; j < FN; j++) read_b(0, j);
      __builtin_amdgcn_sched_barrier(0);
      load_part(0, kEarly, step + 2);
#pragma unroll
      for (int x = kProducts / 2 - kLag; x < kProducts / 2; x++) add(x);
      if (late) stage_arrived(step + 1);
      xa += kStage - 2 * to;
      xb += kStage - 2 * to;
      to = kStage - to;
      together();
      turn(1);
      if (!late) stage_arrived(step + 1);
      if ((step + 1) % kChunk == 0) load_scales(rs, step / kChunk + 2);
      if (step % 64 == 63) load_sb(step + 65);
      together();
    }
#pragma unroll
    for (int x = kProducts - kLag; x < kProducts; x++) add(x);
    if (!late) together();
  } else {
    // A stage's codes are read into registers while the one before it is
    // multiplied.  At its start the next stage has arrived and everyone has read this
    // one, over which the stage S after it is loaded.  The last results of a stage
    // join the sums during the next one, with that one's scales.
    f32x4 d[4] = {};
    float old[FM];
    constexpr int kReads = (2 * (FM + FN) + kProducts - 1) / kProducts;
    constexpr int kLoads = (L + kProducts - 1) / kProducts;
    float sb[2];
#pragma unroll
    for (int j = 0; j < FN; j++) read_b(0, j);
#pragma unroll
    for (int i = 0; i < FM; i++) read_a(0, i);
    read_scales(0, 0);
    sb[0] = read_sb(0);
    const auto stage = [&](uint32_t step, auto now) {
      constexpr int P = decltype(now)::value;
      const uint32_t next = to == (S - 1) * kStage ? 0 : to + kStage;
      arrived(std::integral_constant<int, kYoung>{});
      if (step + 2 == steps && cut_last) cut_stage(next);
      together();
      xa += next - to;
      xb += next - to;
      const uint32_t after = step + 1 < steps ? step + 1 : step, coming = step + S;
#pragma unroll
      for (int i = 0; i < FM; i++) {
        old[i] = s[i];
        s[i] = sa[P][i] * sb[P];
      }
      read_scales(1 - P, after);
      sb[1 - P] = read_sb(after);
      if (coming + 1 == steps && cut_last) offsets(coming * kF8Step);
      end_buffer(ra, coming, steps);
      end_buffer(rb, coming, steps);
      const uint32_t k = coming < steps ? coming * kF8Step : 0u;
#pragma unroll
      for (int x = 0; x < kProducts; x++) {
        __builtin_amdgcn_sched_barrier(0);
        d[x % 4] = block_sum(fb[P][x / FM], fa[P][x % FM]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = x * kReads; i < (x + 1) * kReads; i++)
          if (i < FN) read_b(1 - P, i);
          else if (i < FM + FN) read_a(1 - P, i - FN);
#pragma unroll
        for (int r = x * kLoads; r < (x + 1) * kLoads; r++)
          if (r < L) load(r, ra, rb, k, to * 16);
        const int y = x < kLag ? kProducts - kLag + x : x - kLag;
        add_scaled(acc[y % FM][y / FM], d[y % 4], x < kLag ? old[y % FM] : s[y % FM]);
        here(acc[y % FM][y / FM]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if ((step + 1) % kChunk == 0) load_scales(rs, step / kChunk + 2);
      if (step % 64 == 63) load_sb(step + 65);
      to = next;
    };
#pragma unroll 1
    for (uint32_t step = 0; step < steps; step += 2) {
      stage(step, std::integral_constant<int, 0>{});
      if (step + 1 < steps) stage(step + 1, std::integral_constant<int, 1>{});
    }
#pragma unroll
    for (int y = kProducts - kLag; y < kProducts; y++) add_scaled(acc[y % FM][y / FM], d[y % 4], s[y % FM]);
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);        // nothing may still be on its way to LDS

  // this lane holds, of token wm + 16i + p, the channels wn + 32(j/2) + 8q +
  // 4(j%2) + e: 8 neighbours for two j
#pragma unroll
  for (int i = 0; i < FM; i++) {
    const uint32_t m = m0 + wm + 16 * i + p;
    if (m >= job.end) continue;
    const bool real = real_row<Grouped>(g, m);
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
      const uint32_t x = wn + 16 * j + 8 * q;
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 4; h++) {
        const f32x4& v = acc[i][j + h / 2];
        const int e = h % 2 * 2;
        w[h] = real ? st16x2<D>(v[e] + lbias[x + 2 * h], v[e + 1] + lbias[x + 2 * h + 1]) : 0u;
      }
      store_row<8>(g, m, n0 + x, w);
    }
  }
}

// A block of BM tokens by BN channels to a workgroup, whose W waves share the
// sum (few tiles, or few rows an expert: bound by the weights' bytes, or by the
// latency of a stage, 0.05 to 0.13 us): wave w takes blocks w, w + W, ... through a
// ring of S stages of its own in LDS, the tokens' scales beside the codes.
constexpr uint32_t kApart = 2;               // stages from one tile's start to its neighbour's

template <int BM, int BN, int W, int S, int D, bool Once, bool Grouped>
__global__ __launch_bounds__(64 * W) void k_split_f8(F8Args g, Grid gr) {
  constexpr int FM = (BM + 15) / 16, FN = BN / 16;
  constexpr int LA = BM / 8, LB = BN / 8, L = LA + LB + 1;  // loads of a stage
  constexpr uint32_t kScales = (BM + BN) * 8;             // where the scales lie
  constexpr uint32_t kStage = kScales + 16;               // pieces of a stage
  static_assert(FM * FN * 64 <= S * kStage && (S - 1) * L < 64 && BM <= 64 && BN <= 128);
  __shared__ i32x4 lds[W * S * kStage];
  const uint32_t t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
  Job job;
  if (!find_job<BM, BN, Grouped>(g, gr, job)) return;
  const uint32_t n0 = job.n0;
  const uint32_t K16 = (g.K + 15) & ~15u;
  const uint32_t steps = (g.K + kF8Step - 1) / kF8Step;
  const bool cut_last = g.K % kF8Step != 0;
  uint32_t ra0[LA], va[LA], vb[LB];
#pragma unroll
  for (int i = 0; i < LA; i++) ra0[i] = row_of<Grouped>(g, job, i * 8 + lane / 8) * (uint32_t)g.lda;
  const uint32_t vs = row_of<Grouped>(g, job, lane < BM ? lane : BM - 1) * (uint32_t)g.ldsa * 4;
  const auto offsets = [&](uint32_t k) {
    const uint32_t c = 16 * (lane % 8 ^ lane / 8), at = k + c < K16 ? c : K16 - 16 - k;
#pragma unroll
    for (int i = 0; i < LA; i++) va[i] = ra0[i] + at;
#pragma unroll
    for (int i = 0; i < LB; i++) {
      const uint32_t r = i * 8 + lane / 8;
      vb[i] = (n0 + r < g.N ? r : g.N - 1 - n0) * (uint32_t)g.ldb + at;
    }
  };
  i32x4* const ring = lds + wave * S * kStage;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds +
                         wave * S * kStage * 16;
  const size_t from = first_row<Grouped>(g, job);
  i32x4 ra = buffer_at(g.a + from * g.lda), rb = buffer_at(job.b + (size_t)n0 * g.ldb);
  i32x4 rs = buffer_at(g.sa + from * g.ldsa);
  const ConstF sbp = constant(job.sb + (size_t)(n0 / 128) * g.ldsb);
  // block s into slot `to`; past the last block from an empty buffer, from which
  // nothing is fetched
  const uint32_t rest = steps > 1 ? steps - 1 : 1;        // the last one stays last
  const uint32_t turn = (uint32_t)__builtin_amdgcn_readfirstlane((int)(n0 / BN * kApart % rest));
  const auto block_of = [&](uint32_t s) {
    const uint32_t at = s + turn < rest ? s + turn : s + turn - rest;
    return s + 1 >= steps ? (s < steps ? s : 0u) : at;
  };
  const auto load = [&](uint32_t s, uint32_t to) {
    const uint32_t at = block_of(s), k = at * kF8Step;
    end_buffer(ra, s, steps);
    end_buffer(rb, s, steps);
    end_buffer(rs, s, steps);
    if (s + 1 == steps && cut_last) offsets(k);
#pragma unroll
    for (int i = 0; i < LB; i++)
      load_to_lds<Once>(rb, ring0 + (to * kStage + BM * 8 + i * 64) * 16, vb[i], k);
#pragma unroll
    for (int i = 0; i < LA; i++)
      load_to_lds<false>(ra, ring0 + (to * kStage + i * 64) * 16, va[i], k);
    load_word_to_lds(rs, ring0 + (to * kStage + kScales) * 16, vs, 4 * at);
  };
  const uint32_t p = lane % 16, q = lane / 16;
  const uint32_t x0 = p * 8 + (q ^ (p & 7)), xa = BM < 16 ? x0 & 63 : x0;
  f32x4 acc[FM][FN] = {};
  offsets(0);
#pragma unroll
  for (uint32_t i = 0; i < S; i++) load(wave + i * W, i);
  float sb = sbp[block_of(wave)];
  uint32_t to = 0;
#pragma unroll 1
  for (uint32_t s = wave; s < steps; s += W) {
    constexpr int n = (S - 1) * L;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 0x0f70);
    asm volatile("" ::: "memory");
    i32x4* const at = ring + to * kStage;
    if (s + 1 == steps && cut_last) {
      // zeros for the codes past K, of a and b: either may hold NaN codes there
      const uint32_t k = s * kF8Step + 16 * (lane % 8 ^ lane / 8);
#pragma unroll
      for (int i = 0; i < LA + LB; i++)
        if (k + 16 > g.K) at[i * 64 + lane] = cut(at[i * 64 + lane], k, g.K);
    }
    i32x4 fa[FM][2], fb[FN][2];
    float sa[FM];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int j = 0; j < FN; j++) fb[j][h] = at[BM * 8 + j * 128 + (x0 ^ (4 * h))];
#pragma unroll
      for (int i = 0; i < FM; i++) fa[i][h] = at[i * 128 + (xa ^ (4 * h))];
    }
    const float* const scales = reinterpret_cast<const float*>(at + kScales);
#pragma unroll
    for (int i = 0; i < FM; i++) sa[i] = scales[BM < 16 ? p % BM : 16 * i + p] * sb;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);      // the slot is read: it may be loaded again
    asm volatile("" ::: "memory");
    load(s + S * W, to);
    sb = sbp[block_of(s + W)];
    __builtin_amdgcn_sched_barrier(0);
    f32x4 d[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) d[i][j] = block_sum(fb[j], fa[i]);
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) add_scaled(acc[i][j], d[i][j], sa[i]);
    to = to + 1 == S ? 0 : to + 1;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);        // nothing may still be on its way to LDS
  asm volatile("" ::: "memory");
  f32x4* const sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) sums[wave * S * kStage + (i * FN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // the waves' sums, in their order: entry x holds 4 neighbouring channels of one
  // token
  for (uint32_t x = t; x < FM * FN * 64; x += 64 * W) {
    const uint32_t f = x / 64, m = job.m0 + f / FN * 16 + x % 16;
    const uint32_t n = n0 + f % FN * 16 + x % 64 / 16 * 4;
    f32x4 sum = sums[x];
#pragma unroll
    for (int w = 1; w < W; w++) sum += sums[w * S * kStage + x];
    if (m < job.end && n < g.N && (BM >= 16 || x % 16 < BM)) {
      const uint16_t* const bias = reinterpret_cast<const uint16_t*>(job.bias);
      if (bias)
#pragma unroll
        for (uint32_t e = 0; e < 4; e++) sum[e] += ld16<D>(bias[n + e < g.N ? n + e : g.N - 1]);
      u32x2 v = {0u, 0u};
      if (real_row<Grouped>(g, m))
#pragma unroll
        for (int e = 0; e < 4; e += 2) v[e / 2] = st16x2<D>(sum[e], sum[e + 1]);
      store_row<4>(g, m, n, v);
    }
  }
}

template <int I>
hipError_t launch_tile(int dtype, const F8Args& g, hipStream_t st) {
  constexpr F8Tile t = kF8Tiles[I];
  const Grid gr{f8_tile_rows(t.bm, g.M, g.E), (g.N + t.bn - 1) / t.bn, t.group};
  const dim3 grid(gr.tm * gr.tn), block(64 * t.wm * (t.wn ? t.wn : 1));
  const auto kernel = [&](auto d, auto once, auto grouped) {
    constexpr int D = decltype(d)::value;
    constexpr bool Once = decltype(once)::value, Grouped = decltype(grouped)::value;
    if constexpr (t.wn == 0) k_split_f8<t.bm, t.bn, t.wm, t.stages, D, Once, Grouped><<<grid, block, 0, st>>>(g, gr);
    else k_tile_f8<t.bm, t.bn, t.wm, t.wn, t.stages, D, Once, Grouped><<<grid, block, 0, st>>>(g, gr);
  };
  const auto of_type = [&](auto d) {
    const bool once = f8_weights_once(t.bm, g.M, g.E);
    if (g.E == 0) {
      // tiles of 8 rows: up to 8 tokens only (choose_f8_tile)
      if constexpr (t.bm == 8) kernel(d, std::true_type{}, std::false_type{});
      else if (once) kernel(d, std::true_type{}, std::false_type{});
      else kernel(d, std::false_type{}, std::false_type{});
    } else {
      if (once) kernel(d, std::true_type{}, std::true_type{});
      else kernel(d, std::false_type{}, std::true_type{});
    }
  };
  if (dtype == kF16) of_type(std::integral_constant<int, kF16>{});
  else of_type(std::integral_constant<int, kBF16>{});
  return hipGetLastError();
}

using Launch = hipError_t (*)(int, const F8Args&, hipStream_t);
template <int... I>
Launch launch_of(int tile, std::integer_sequence<int, I...>) {
  static constexpr Launch table[] = {launch_tile<I>...};
  return table[tile];
}

}  // namespace

hipError_t launch_gemm_f8(int tile, int dtype, const F8Args& g, hipStream_t st) {
  return launch_of(tile, std::make_integer_sequence<int, kF8TileCount>{})(dtype, g, st);
}

}  // namespace qr
