// Stored keys as packed pairs of 16-bit numbers, for the block kernels.
#pragma once

#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {

// Head dims 8 t .. 8 t + 7 of a storage row: loaded, then as four words of two
// values each without the head's scale, bf16 of a bf16 cache and else f16, exact.
template <int KV>
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const void* base, size_t row, int t) {
    const uint8_t* b = static_cast<const uint8_t*>(base);
    if (KV == kKvBf16) {
      w = *(reinterpret_cast<const uint4*>(b + (row * kHeadDim + t * 8) * 2));
    } else if (KV == kKvFp8) {
      const uint2 v = *(reinterpret_cast<const uint2*>(b + row * kHeadDim + t * 8));
      w.x = v.x;
      w.y = v.y;
    } else {
      w.x = *(reinterpret_cast<const uint32_t*>(b + fp4_codes(row) + t * 4));
      w.y = *(b + fp4_scales(row) + (t >> 1));
    }
  }
  __device__ __forceinline__ void words(uint32_t (&h)[4]) const {
    if (KV == kKvBf16) {
      h[0] = w.x;
      h[1] = w.y;
      h[2] = w.z;
      h[3] = w.w;
    } else if (KV == kKvFp8) {
      h[0] = e4m3x2_to_f16x2((uint16_t)(w.x & 0xFFFF));
      h[1] = e4m3x2_to_f16x2((uint16_t)(w.x >> 16));
      h[2] = e4m3x2_to_f16x2((uint16_t)(w.y & 0xFFFF));
      h[3] = e4m3x2_to_f16x2((uint16_t)(w.y >> 16));
    } else {
      e2m1x8_to_f16x8(w.x, h);
      const uint32_t s = e4m3x2_to_f16x2((uint16_t)w.y);
      const uint32_t s2 = prmt(s, s, 0x1010);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = hmul2(h[i], s2);
    }
  }
};

// All ones in the halves of a word that are numbers, zeros in NaNs.
template <int KV>
__device__ __forceinline__ uint32_t number_mask(uint32_t x) {
  if (KV == kKvBf16) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&x);
    return __heq2_mask(v, v);
  }
  const __half2 v = *reinterpret_cast<const __half2*>(&x);
  return __heq2_mask(v, v);
}
template <int KV>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (KV == kKvBf16)
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int KV>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (KV == kKvBf16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return pack_bf16x2(f.x, f.y);
}

}  // namespace tfpa
