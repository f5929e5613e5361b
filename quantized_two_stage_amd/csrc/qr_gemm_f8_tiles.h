// qr_gemm_f8_tiles.h -- which kernel and tile the products of include/qr_f8.h
// take for a size.  Plain host C++, shared by the launch (qr_gemm_f8.hip) and by
// the tests that run every tile.  Not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qr_gemm_tiles.h"

namespace qr {

// As kTiles: what a workgroup takes to start and end, and for each block of 128
// of the sum, ns, where every CU has one at most.
constexpr Tile kF8Tiles[] = {
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
constexpr int kF8TileCount = sizeof(kF8Tiles) / sizeof(kF8Tiles[0]);

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
  const uint32_t likely = E == 0 ? most : M / bm + (some + 1) / 2;
  return E == 0 ? most : likely < some ? some : likely < most ? likely : most;
}

// Index into kF8Tiles.
inline int choose_f8_tile(uint32_t M, uint32_t N, uint32_t K, uint32_t E) {
  if (E == 0 && M <= 8) return N <= 16 * 256 && K >= 32 * kStep ? 0 : 1;
  const uint64_t steps = (K + kStep - 1) / kStep;
  int best = -1;
  uint64_t least = ~0ull;
  for (int i = 2; i < kF8TileCount; i++) {
    const Tile& t = kF8Tiles[i];
    const uint64_t tm = f8_tile_rows_likely(t.bm, M, E), blocks = tm * ((N + t.bn - 1) / t.bn);
    uint64_t ns = (blocks + 255) / 256 * (t.start + steps * t.stage);
    if (tm == 1) ns -= ns / 10;
    if (ns < least) {
      least = ns;
      best = i;
    }
  }
  return best;
}

}  // namespace qr
