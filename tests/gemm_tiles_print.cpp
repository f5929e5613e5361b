// Reads sizes "M N K" and prints the tile that qr_gemm_i8 takes for each:
// index, tokens, channels, waves (two numbers), stages of a ring, rows of tiles.
#include <cstdio>

#include "../quantized_two_stage_amd/csrc/qr_gemm_tiles.h"

int main() {
  unsigned M, N, K;
  while (std::scanf("%u %u %u", &M, &N, &K) == 3) {
    const int i = qr::choose_tile(M, N, K);
    const qr::Tile& t = qr::kTiles[i];
    std::printf("%d %u %u %u %u %u %u\n", i, t.bm, t.bn, t.wm, t.wn, t.stages, qr::tile_rows(t, M));
  }
  return 0;
}
