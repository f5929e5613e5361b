// qr_gemm.hip -- gfx950 kernels of qr_gemm_i8 (include/qr_layer.h): the matrix
// product of 8-bit codes with a scale for each token and each output channel.
#include "qr.h"
#include "qr_device.h"
#include "qr_layer_internal.h"

namespace qr {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// bytes [k, k+16) of a row of K codes, zeros past K
__device__ __forceinline__ i32x4 load16(const int8_t* row, uint32_t k, uint32_t K) {
  if (k >= K) return i32x4{0, 0, 0, 0};
  i32x4 v = *reinterpret_cast<const i32x4*>(row + k);
  if (k + 16 > K) {
#pragma unroll
    for (int w = 0; w < 4; w++) {
      const int left = (int)(K - k) - 4 * w;             // bytes of word w inside the row
      v[w] = left >= 4 ? v[w] : left <= 0 ? 0 : (int)((uint32_t)v[w] & ((1u << (8 * left)) - 1u));
    }
  }
  return v;
}

// One workgroup computes 64 tokens x 64 channels, four waves 32 x 32 each,
// 64 codes of the sum a step.
template <int D>
__global__ __launch_bounds__(256) void k_gemm(GemmArgs g) {
  __shared__ i32x4 la[64][5], lb[64][5];                 // 64 codes a row, padded
  const uint32_t n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t wn = 32 * (wave & 1), wm = 32 * (wave >> 1);
  const uint32_t r = threadIdx.x / 4, part = threadIdx.x % 4;
  const uint32_t am = m0 + r < g.M ? m0 + r : g.M - 1, bn = n0 + r < g.N ? n0 + r : g.N - 1;
  const int8_t* ap = g.a + (size_t)am * g.lda;
  const int8_t* bp = g.b + (size_t)bn * g.ldb;
  i32x4 acc[2][2] = {};
  for (uint32_t k0 = 0; k0 < g.K; k0 += 64) {
    const i32x4 va = load16(ap, k0 + 16 * part, g.K), vb = load16(bp, k0 + 16 * part, g.K);
    __syncthreads();
    la[r][part] = va;
    lb[r][part] = vb;
    __syncthreads();
    i32x4 fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      fa[i] = la[wm + 16 * i + lane % 16][lane / 16];
      fb[i] = lb[wn + 16 * i + lane % 16][lane / 16];
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < 2; j++)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint32_t m = m0 + wm + 16 * i + lane % 16, n = n0 + wn + 16 * j + 4 * (lane / 16) + e;
        if (m >= g.M || n >= g.N) continue;
        float v = (float)acc[i][j][e] * (g.sa[m] * g.sb[n]);
        if (g.bias) v += ld16<D>(reinterpret_cast<const uint16_t*>(g.bias)[n]);
        reinterpret_cast<uint16_t*>(g.c)[(size_t)m * g.ldc + n] = (uint16_t)st16<D>(v);
      }
}

}  // namespace

size_t gemm_workspace_bytes(size_t, size_t, size_t) { return 0; }

hipError_t launch_gemm(int dtype, const GemmArgs& g, hipStream_t st) {
  const dim3 grid((g.N + 63) / 64, (g.M + 63) / 64);
  if (dtype == kF16)
    k_gemm<kF16><<<grid, 256, 0, st>>>(g);
  else
    k_gemm<kBF16><<<grid, 256, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace qr
