// qr_gemm_device.h -- what the matrix products' kernels share (qr_gemm.hip,
// qr_gemm_f8.hip): loads that go to LDS directly, the order of the tiles, and
// the stores of a row.  Not part of the ABI.
#pragma once

#include "qr_device.h"

namespace qr {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes from base + voff + soff to LDS byte lds + 16*lane, for every lane of
// the wave, without passing through registers; s_waitcnt vmcnt covers it.  In
// assembly since the compiler, where it cannot tell two LDS buffers apart,
// would wait for the load before any LDS read: the caller waits.  It has no
// output register, so nothing is written behind the compiler's back but LDS:
// m0, which holds the LDS address, is an input that the compiler sets.  The wait
// states are those that a memory instruction needs after a vector instruction
// wrote its scalar operands: the compiler, which does not see the load, may restore
// spilled ones (v_readlane_b32) right before the statement.  They cost 2% at most:
// qr_gemm_i8 with one wait state and with five, on several cards: 1 token over 8192 x
// 8192 12.0 to 12.6 us and 11.9 to 12.1, 48 over 8192 x 4096 11.1 to 13.0 and 11.7,
// 333 x 5003 x 2050 14.5 and 14.6 to 14.8, 8192^3 424 to 442 and 420 to 428.
// The buffer must be in scalar registers when it gets here: one that the compiler
// holds in vector registers, because it cannot tell that all lanes hold the same,
// would be misread (a test reads the assembly for it).
// Once: past the caches, for what no other workgroup reads.
template <bool Once>
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t lds, uint32_t voff,
                                            uint32_t soff) {
  if constexpr (Once)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :
                 : "{m0}"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
  else
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "{m0}"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}
// A buffer that starts at p, for load_to_lds.
__device__ __forceinline__ i32x4 buffer_at(const void* p) {
  const uint64_t a = (uint64_t)p;
  const int lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const int hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xffff;
  return i32x4{lo, hi, -1, 0x00027000};
}
// all of the buffer while s < steps, afterwards nothing (and nothing is fetched)
__device__ __forceinline__ void end_buffer(i32x4& r, uint32_t s, uint32_t steps) {
  int bytes;
  asm("s_cmp_lt_u32 %1, %2\n\ts_cselect_b32 %0, -1, 0"
      : "=s"(bytes)
      : "s"(s), "s"(steps)
      : "scc");
  r[2] = bytes;
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

// W/2 words of 16-bit values to c[m][n..]: one store inside the row
template <int W, class Args, class V>
__device__ __forceinline__ void store_row(const Args& g, uint32_t m, uint32_t n, const V& w) {
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

// Workgroups go to the 8 XCDs in turn: the tile of workgroup b of `total`, so that
// each XCD has neighbouring tiles.
__device__ __forceinline__ uint32_t tile_number(uint32_t total, uint32_t b) {
  const uint32_t per = total / 8, extra = total % 8;
  const uint32_t x = b % 8, i = b / 8;
  return x * per + (x < extra ? x : extra) + i;
}
// the t-th tile, down the rows of a group of tile rows first
__device__ __forceinline__ void tile_at(const Grid& gr, uint32_t t, uint32_t& m, uint32_t& n) {
  const uint32_t g = t / (gr.group * gr.tn), r = t % (gr.group * gr.tn);
  const uint32_t m0 = g * gr.group;
  const uint32_t rows = gr.tm - m0 < gr.group ? gr.tm - m0 : gr.group;
  m = m0 + r % rows;
  n = r / rows;
}
__device__ __forceinline__ void tile_of(const Grid& gr, uint32_t b, uint32_t& m, uint32_t& n) {
  tile_at(gr, tile_number(gr.tm * gr.tn, b), m, n);
}

}  // namespace
}  // namespace qr
