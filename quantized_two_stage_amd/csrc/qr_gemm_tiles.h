// qr_gemm_tiles.h -- which kernel and tile qr_gemm_i8 takes for a size.  Plain
// host C++, shared by the launch (qr_gemm.hip) and by the tests that run every
// tile.  Not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qr {

constexpr uint32_t kStep = 128;       // codes of the sum in one stage

// Tiles and what a workgroup of each was measured to take where every CU has
// one at most: ns to start and end, and ns for each stage of the sum.  The
// launch takes the one whose rounds of 256 workgroups are estimated to end
// first.  Measured with cold weights at 1024 tokens x 1024 channels, K = 8192
// (64 stages), us: 16x16 58, 32x32 31 (four rounds), 64x64 of k_split 20.9;
// at 2048 x 16384, K = 1024: 64x64 of k_tile 97, 64x128 98, 128x64 101, 128x128
// 75, 128x256 59, 256x256 50.
// The rule against the fastest of these tiles at each of 158 sizes (10 shapes of
// weights from 300x16384 to 16384x1024, 1 to 2048 tokens, cold weights): 1.00
// at the median, within 1.024 at nine of ten, 1.14 at worst (48 tokens, 5003x2050:
// 9.8 us against 8.6 in 16x32).  The estimate has no term for the weights' bytes:
// they take as long in every tile of one row of tiles.
struct Tile {
  uint32_t bm, bn;                    // tokens and channels
  uint32_t wm, wn;                    // waves; wn == 0: wm waves that share the sum (k_split)
  uint32_t stages;                    // of a ring
  uint32_t group;                     // tile rows that neighbouring workgroups share
  uint32_t start, stage;              // ns; 0: not estimated, see choose_tile
};
constexpr Tile kTiles[] = {
    {8, 16, 8, 0, 2, 1, 0, 0},
    {8, 16, 4, 0, 3, 1, 0, 0},
    {16, 16, 8, 0, 2, 16, 2800, 65},
    {16, 32, 4, 0, 3, 16, 2900, 100},
    {32, 32, 4, 0, 2, 16, 3100, 130},
    {64, 32, 4, 0, 3, 16, 4000, 190},
    {64, 64, 4, 0, 2, 16, 4500, 240},
    {64, 64, 2, 2, 4, 8, 3000, 290},
    {64, 128, 2, 4, 5, 8, 3400, 360},
    {128, 64, 4, 2, 5, 8, 3400, 380},
    {128, 128, 2, 4, 4, 8, 4000, 520},
    {128, 256, 2, 4, 3, 8, 4500, 780},
    {256, 256, 4, 2, 2, 4, 5500, 1350},
};
constexpr int kTileCount = sizeof(kTiles) / sizeof(kTiles[0]);

// tiles along M; with one row of them the weights are read once
constexpr uint32_t tile_rows(const Tile& t, uint32_t M) { return (M + t.bm - 1) / t.bm; }

// Index into kTiles.
// Up to 8 tokens only 8 rows of a are staged: 1 token, 2048x8192 7.1 us
// against 8.8 (16x32) with 16 rows; 16384x1024 6.4 against 6.6.
// Eight waves where a CU has one workgroup at most and the sum is long: 1
// token, 300x16384 8.1 against 9.3 with four, 2048x8192 6.0 and 6.7; elsewhere
// four: 16384x4096 12.1 against 14.1, 1000x1000 3.2 and 3.3.
inline int choose_tile(uint32_t M, uint32_t N, uint32_t K) {
  if (M <= 8) return N <= 16 * 256 && K >= 32 * kStep ? 0 : 1;
  const uint64_t steps = (K + kStep - 1) / kStep;
  int best = -1;
  uint64_t least = ~0ull;
  for (int i = 2; i < kTileCount; i++) {
    const Tile& t = kTiles[i];
    const uint64_t tm = tile_rows(t, M), blocks = tm * ((N + t.bn - 1) / t.bn);
    uint64_t ns = (blocks + 255) / 256 * (t.start + steps * t.stage);
    // the weights are read once, past the caches: where this decides, 96 tokens
    // over 11008x4096 take 16.8 us against 18.7 (128x64, 64x128), 128 over
    // 16384x1024 8.4 against 9.3
    if (tm == 1) ns -= ns / 10;
    if (ns < least) {
      least = ns;
      best = i;
    }
  }
  return best;
}

}  // namespace qr
