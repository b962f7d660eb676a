// Staged key tiles of quantised caches -> f16 operand tiles of the tensor
// cores, shared by the prompt / verify kernel and the attention-weight kernel.
#pragma once

#include "common.cuh"
#include "params.h"

namespace tfpa {

// e4m3 staging tile [128 rows][128 B] (128B swizzle) -> f16 operand tile
// [128 rows][2 halves of 64] (128B swizzle), THREADS threads (thread t of
// them); rows >= z0 become 0.
template <int THREADS>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int z0, int t) {
  const uint32_t sb = smem_u32(src), db = smem_u32(dst);
#pragma unroll
  for (int k = 0; k < 1024 / THREADS; ++k) {
    const int i = t + THREADS * k;             // (row, 16-byte source chunk)
    const int row = i >> 3, c8 = i & 7;    // source chunk c8 = head dims 16*c8 .. +15
    uint4 w = lds128(swz128(sb, row, c8));
    if (row >= z0) w = make_uint4(0, 0, 0, 0);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      h[2 * q] = e4m3x2_to_f16x2((uint16_t)(ws[q] & 0xFFFF));
      h[2 * q + 1] = e4m3x2_to_f16x2((uint16_t)(ws[q] >> 16));
    }
    const uint32_t half = db + (uint32_t)(c8 >> 2) * 16384u;
    const int c16 = 2 * (c8 & 3);
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(swz128(half, row, c16)),
                 "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(swz128(half, row, c16 + 1)),
                 "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
  }
}

// The same for a staged half-block of a 4-bit cache (128 rows' codes, then
// their scales): code * block scale, exact in f16.  A thread turns 32 head
// dims of a row at a time.  Its lane fixes the row and which quarter of a
// 64-column half it takes, the loop the half, so that eight neighbouring
// lanes' 16-byte stores fall into eight different bank groups.  In two parts,
// so that a caller may read the next tile before it writes this one.  Holds
// STEPS of the 512 / THREADS steps from step k0 on.
template <int THREADS, int STEPS = 512 / THREADS>
struct Fp4Tile {
  static constexpr int kSteps = STEPS;
  uint4 w[kSteps];
  uint32_t s[kSteps];
  static __device__ __forceinline__ int row(int k, int t) {
    return (t >> 1) + THREADS / 2 * (k >> 1);
  }
  __device__ __forceinline__ void read(const uint8_t* src, int z0, int t, int k0 = 0) {
    const uint32_t sb = smem_u32(src);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = row(k0 + k, t), c = 2 * ((k0 + k) & 1) + (t & 1);   // head dims 32 c .. + 31
      w[k] = lds128(sb + r * kFp4CodeBytes + 16 * c);
      s[k] = lds16(sb + kFp4ScaleOff + r * kFp4ScaleBytes + 2 * c);
      if (r >= z0) s[k] = 0;
    }
  }
  __device__ __forceinline__ void write(uint8_t* dst, int t, int k0 = 0) const {
    const uint32_t db = smem_u32(dst);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)s[k]);
      const uint32_t sc[2] = {prmt(s2, s2, 0x1010), prmt(s2, s2, 0x3232)};
      const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t h[4];
        e2m1x8_to_f16x8(ws[u], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = hmul2(h[j], sc[u >> 1]);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                         swz128(db + ((k0 + k) & 1) * 16384u, row(k0 + k, t), 4 * (t & 1) + u)),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
      }
    }
  }
};

// A whole tile, STEPS steps' reads ahead of their writes (the prompt path's
// converters, which have a warp per sub-partition: all four 1753 us on a
// chunk of 4,096 rows over 32,768 keys, one at a time 1769 us; the attention-weight
// kernel's, which have two: 87.2 against 85.1 us on a 32-row window).
template <int THREADS, int STEPS>
__device__ __forceinline__ void convert_tile_fp4(const uint8_t* src, uint8_t* dst, int z0,
                                                 int t) {
#pragma unroll
  for (int k0 = 0; k0 < 512 / THREADS; k0 += STEPS) {
    Fp4Tile<THREADS, STEPS> x;
    x.read(src, z0, t, k0);
    x.write(dst, t, k0);
  }
}

}  // namespace tfpa
