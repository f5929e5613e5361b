// Reads sizes "E M N K" and prints the index of the tile that the products of
// include/qr_f8.h take for each; with no input line, the tiles.
#include <cstdio>

#include "../quantized_two_stage_amd/csrc/qr_gemm_f8_tiles.h"

int main(int argc, char**) {
  if (argc > 1) {
    for (const qr::F8Tile& t : qr::kF8Tiles) std::printf("%u %u %u %u %u\n", t.bm, t.bn, t.stages, t.wn, 64 * t.wm * (t.wn ? t.wn : 1));
    return 0;
  }
  unsigned E, M, N, K;
  while (std::scanf("%u %u %u %u", &E, &M, &N, &K) == 4)
    std::printf("%d\n", qr::choose_f8_tile(M, N, K, E));
  return 0;
}
