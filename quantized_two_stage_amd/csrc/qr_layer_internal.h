// qr_layer_internal.h -- kernel launchers behind include/qr_layer.h, shared by
// its host code (qr_layer_api.cpp) and the kernels (qr_rows.hip, qr_gemm.hip).
// Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qr {

// Row operators: M rows of d values to codes and scales.  Strides in elements.
struct RowsOut {
  int8_t* q;
  size_t ldq;
  float* scales;
  uint32_t M, d;
};

struct NormArgs {
  const uint8_t* x;        // rows of 16-bit values, or a planar wire image
  size_t ldx;
  size_t off_s, off_z;     // the wire image's planes
  const uint8_t* residual; // nullptr: none
  size_t ldr;
  const uint8_t* weight;
  uint8_t* h;              // nullptr: not written
  size_t ldh;
  float eps;
};

// codec < 0: x holds 16-bit rows
hipError_t launch_norm(int codec, int dtype, const NormArgs& a, const RowsOut& o, hipStream_t st);
hipError_t launch_silu(int dtype, const uint8_t* gu, size_t ldg, const RowsOut& o,
                       hipStream_t st);

struct GemmArgs {
  const int8_t* a;
  size_t lda;
  const float* sa;
  const int8_t* b;
  size_t ldb;
  const float* sb;
  const uint8_t* bias;     // nullptr: none
  uint8_t* c;
  size_t ldc;
  uint32_t M, N, K;
};

hipError_t launch_gemm(int dtype, const GemmArgs& g, hipStream_t st);

}  // namespace qr
