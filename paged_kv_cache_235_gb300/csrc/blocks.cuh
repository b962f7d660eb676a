// Loads of stored rows for the block kernels.
#pragma once

#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {

// Head dims 8 t .. 8 t + 7 of storage row `row`, as stored values without the
// head's scale (float32, exact).
template <int KV>
__device__ __forceinline__ void load8(const void* base, size_t row, int t, float (&x)[8]) {
  const uint8_t* b = static_cast<const uint8_t*>(base);
  if (KV == kKvBf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(b + (row * kHeadDim + t * 8) * 2)), x);
    return;
  }
  uint32_t h[4];
  if (KV == kKvFp8) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(b + row * kHeadDim + t * 8));
    h[0] = e4m3x2_to_f16x2((uint16_t)(w.x & 0xFFFF));
    h[1] = e4m3x2_to_f16x2((uint16_t)(w.x >> 16));
    h[2] = e4m3x2_to_f16x2((uint16_t)(w.y & 0xFFFF));
    h[3] = e4m3x2_to_f16x2((uint16_t)(w.y >> 16));
  } else {
    e2m1x8_to_f16x8(__ldg(reinterpret_cast<const uint32_t*>(b + fp4_codes(row) + t * 4)), h);
    const uint32_t s = e4m3x2_to_f16x2((uint16_t)__ldg(b + fp4_scales(row) + (t >> 1)));
    const uint32_t s2 = prmt(s, s, 0x1010);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = hmul2(h[i], s2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}

}  // namespace tfpa
