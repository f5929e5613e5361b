// qr_gemm_f8_tiles.h -- which kernel and tile the products of include/qr_f8.h
// take for a size.  Plain host C++, shared by the launch (qr_gemm_f8.hip) and by
// the tests that run every tile.  Not part of the ABI.
#pragma once

#include <cmath>
#include <initializer_list>
#include <stddef.h>
#include <stdint.h>

namespace qr {

// Tiles, and what they were measured to take, in ns.  Their workgroups come in
// rounds of `at_once` on each of 256 CUs; a round takes `start` and `stage` for
// each block of 128 of the sum.  Where there are many, a CU takes `more` and
// `full` a block for each workgroup.  The weights' bytes take their time beside
// that (6000 a ns where they are read once, else 5300): of the shorter of the two
// `once` or `again` percent are added.
// Fitted to the times of all tiles at 380 sizes (1 to 8192 tokens, sums and
// channels of 64 to 16384, one product or 4 to 128 experts, cold weights) and 100
// more of small groups.  The tile that choose_f8_tile takes against the fastest at
// each of these: 1.00 at the median; one product within 1.11 at nine of ten and 1.45
// at worst (206 tokens, 9263 x 12902), groups within 1.12 and 1.35.  At 304 sizes
// that the fit has not seen: one product 1.00, 1.13 and 1.45 (405 tokens, 2048 x
// 16128), groups 1.01, 1.17 and 1.42 (88 rows over 4 experts of 1095 x 100).
struct F8Tile {
  uint32_t bm, bn;                    // tokens and channels
  uint32_t wm, wn;                    // waves; wn == 0: wm waves that share the sum
  uint32_t stages;                    // of a ring
  uint32_t group;                     // tile rows that neighbouring workgroups share
  uint32_t at_once, start, stage, more, full, once, again;
};
constexpr F8Tile kF8Tiles[] = {
    {8, 16, 4, 0, 3, 1, 3, 2860, 64, 350, 47, 54, 61},
    {16, 16, 8, 0, 2, 16, 2, 2880, 50, 1590, 35, 83, 87},
    {16, 32, 4, 0, 3, 16, 2, 3230, 97, 890, 85, 66, 80},
    {32, 32, 4, 0, 2, 16, 2, 3440, 131, 2010, 48, 61, 83},
    {64, 64, 2, 2, 4, 8, 2, 3930, 307, 120, 243, 44, 120},
    {64, 128, 2, 4, 5, 8, 1, 4450, 422, 20, 404, 25, 78},
    {128, 64, 4, 2, 5, 8, 1, 4370, 425, 4870, 148, 11, 85},
    {128, 128, 2, 4, 4, 8, 1, 5280, 552, 2920, 598, 16, 120},
    {128, 256, 2, 4, 3, 8, 1, 6640, 868, 790, 1145, 11, 97},
    {256, 256, 4, 2, 2, 4, 1, 8080, 1162, 1450, 1423, 36, 119},
};
constexpr int kF8TileCount = sizeof(kF8Tiles) / sizeof(kF8Tiles[0]);
constexpr uint32_t kF8Step = 128;     // codes of a block

// Rows of tiles of `bm` rows that M rows of E experts fill at most (E == 0: one
// product), whatever their offsets: every expert with rows may end in a short
// tile.
constexpr uint32_t f8_tile_rows(uint32_t bm, uint32_t M, uint32_t E) {
  const uint32_t some = E < M ? E : M;           // experts with rows
  return E == 0 ? (M + bm - 1) / bm : (M - some) / bm + some;
}
// about as many as there will be: half a tile of each expert stays empty
constexpr uint32_t f8_tile_rows_likely(uint32_t bm, uint32_t M, uint32_t E) {
  const uint32_t most = f8_tile_rows(bm, M, E), some = E < M ? E : M;
  const uint32_t likely = M / bm + (some + 1) / 2;
  return E == 0 ? most : likely < some ? some : likely < most ? likely : most;
}

// Whether most weights are read by one workgroup alone, and go past the caches:
// one row of tiles, or experts of half a tile's rows on average.  Weights of 32
// experts, 2048 x 8192, us: 64 rows in tiles of 8 67 to 69 (through the caches 77), of 16
// 82 (90); 2048 x 4096: 256 rows in tiles of 16 53 (57), 512 rows in tiles of 32 61
// (64), but in tiles of 16 74 (67).
constexpr bool f8_weights_once(uint32_t bm, uint32_t M, uint32_t E) {
  return E == 0 ? M <= bm : 2 * (uint64_t)M <= (uint64_t)bm * (E < M ? E : M);
}

struct F8Time {
  double work, weights;               // of the products, of the weights' bytes
  double all;
};
inline F8Time f8_estimate(const F8Tile& t, uint32_t M, uint32_t N, uint32_t K, uint32_t E) {
  const uint32_t steps = (K + kF8Step - 1) / kF8Step;
  const double blocks = (double)f8_tile_rows_likely(t.bm, M, E) * ((N + t.bn - 1) / t.bn);
  const double few = std::ceil(blocks / (256 * t.at_once)) * (t.start + (double)steps * t.stage);
  const double many = blocks / 256 * (t.more + (double)steps * t.full);
  const double work = few > many ? few : many;
  // experts that get a row, were all chosen alike
  const double hit = E == 0 ? 1 : E * (1 - std::exp(-(double)M / E));
  const bool once = f8_weights_once(t.bm, M, E);
  const double weights = hit * N * K / (once ? 6000 : 5300);
  const double more = 0.01 * (once ? t.once : t.again);
  return {work, weights, work > weights ? work + weights * more : weights + work * more};
}

// A launch counts its lanes in 32 bits.
constexpr bool f8_grid_fits(const F8Tile& t, uint32_t M, uint32_t N, uint32_t E) {
  const uint64_t tiles = (uint64_t)f8_tile_rows(t.bm, M, E) * ((N + t.bn - 1) / t.bn);
  return tiles * (64 * t.wm * (t.wn ? t.wn : 1)) < (uint64_t)1 << 32;
}

// Index into kF8Tiles; -1 if no tile's grid fits.
inline int choose_f8_tile(uint32_t M, uint32_t N, uint32_t K, uint32_t E) {
  if (E == 0 && M <= kF8Tiles[0].bm) return 0;
  // Few rows an expert, and mostly weights to read: the smallest tile that reads
  // them once (of those that are 8, 16 and 32 rows high and fastest there).  The estimate
  // alone takes wider ones: 64 rows over 32 experts of 2048 x 8192 take 67 to 69 us in
  // tiles of 8 x 16, 95 in 64 x 128.  At 135 of 460 timed sizes of groups the two differ:
  // against the fastest tile this rule takes 1.00 at the median, 1.13 at nine of ten and
  // 1.31 at worst, the estimate 1.08, 1.27 and 1.67.
  if (E != 0)
    for (int i : {0, 2, 3})
      if (f8_weights_once(kF8Tiles[i].bm, M, E)) {
        const F8Time t = f8_estimate(kF8Tiles[i], M, N, K, E);
        if (t.weights >= 0.7 * t.work && f8_grid_fits(kF8Tiles[i], M, N, E)) return i;
        break;
      }
  int best = -1;
  double least = 0;
  for (int i = E == 0 ? 1 : 0; i < kF8TileCount; i++) {   // tiles of 8 rows: one row of them, or experts
    if (!f8_grid_fits(kF8Tiles[i], M, N, E)) continue;
    const double ns = f8_estimate(kF8Tiles[i], M, N, K, E).all;
    if (best < 0 || ns < least) {
      least = ns;
      best = i;
    }
  }
  return best;
}

}  // namespace qr
