// qr_f8_internal.h -- kernel launchers behind include/qr_f8.h, shared by its host
// code (qr_f8_api.cpp) and the kernels (qr_rows_f8.hip, qr_gemm_f8.hip,
// qr_experts.hip).  Not part of the ABI.
#pragma once

#include "qr_layer_internal.h"

namespace qr {

constexpr uint32_t kF8Block = 128;       // values with one scale

// M rows of d values to codes with a scale a block.  Strides in elements.
struct F8Out {
  uint8_t* q;
  size_t ldq;
  float* scales;
  size_t lds;
  uint8_t* y;              // the norm's values in 16 bits; nullptr: not written
  size_t ldy;
  uint32_t M, d;
};

hipError_t launch_norm_f8(int dtype, const NormArgs& a, const F8Out& o, hipStream_t st);
hipError_t launch_silu_f8(int dtype, const uint8_t* gu, size_t ldg, const F8Out& o,
                          hipStream_t st);

struct F8Args {
  const uint8_t* a;
  size_t lda;
  const float* sa;
  size_t ldsa;
  const uint8_t* b;
  size_t ldb;
  const float* sb;
  size_t ldsb;
  const uint8_t* bias;     // nullptr: none
  uint8_t* c;
  size_t ldc;
  uint32_t M, N, K;
  // by experts (E > 0)
  uint32_t E, tokens;
  const int32_t* offsets;
  const int32_t* rows;     // nullptr: row i of a
  size_t gb, gsb, ldbias;  // from one expert's weights, scales and bias to the next
};

// tile: choose_f8_tile of the sizes
hipError_t launch_gemm_f8(int tile, int dtype, const F8Args& g, hipStream_t st);

struct RouteArgs {
  const uint8_t* logits;
  size_t ldl;
  uint32_t T, E, k;
  bool renormalize;
  float* weights;
  int32_t *experts, *offsets, *rows, *place;
  uint16_t* counts;        // workspace
};

// type of the logits where they are not 16-bit
constexpr int kF32 = 3;

size_t route_workspace_bytes(uint32_t T, uint32_t E);
hipError_t launch_route(int dtype, const RouteArgs& a, hipStream_t st);

struct CombineArgs {
  const uint8_t* c;
  size_t ldc;
  uint32_t R;
  const int32_t* place;
  const float* weights;
  uint32_t T, k, d;
  const uint8_t* addend;   // nullptr: none
  size_t lda;
  uint8_t* y;
  size_t ldy;
};

hipError_t launch_combine(int dtype, const CombineArgs& a, hipStream_t st);

}  // namespace qr
