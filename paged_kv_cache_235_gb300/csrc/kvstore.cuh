// Element conversions and row addresses of the KV store, shared by the KV
// write kernel and the decode partial kernel's append path, so that both
// store the same bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "params.h"

namespace tfpa {

// Byte offsets of storage row `row` of a 4-bit cache from its base.
__device__ __forceinline__ size_t fp4_codes(size_t row) {
  return (row >> 7) * kFp4HalfBytes + (row & (kHalfRows - 1)) * kFp4CodeBytes;
}
__device__ __forceinline__ size_t fp4_scales(size_t row) {
  return (row >> 7) * kFp4HalfBytes + kFp4ScaleOff + (row & (kHalfRows - 1)) * kFp4ScaleBytes;
}

// Sixteen head dims of a 4-bit row, eight in this thread (x) and eight in
// the lane that differs in bit 0 (`lanes`: the shuffle's participants, both
// of them among them).  The block's scale is e4m3(amax / (6 g)), rounded to
// nearest even and saturating, so that its largest magnitude lands near the
// largest code, 6; a code is e2m1(x / (scale g)), rounded to nearest even
// and saturating.  Every product and quotient is rounded to float32 on its
// own (IEEE division), so the stored bytes are a function of the inputs
// alone.  A NaN is stored as zero, and a block whose scale rounds to zero as
// zeros.  Returns the eight codes; `scale` gets the scale byte.
__device__ __forceinline__ uint32_t quant8_fp4(float (&x)[8], float g, unsigned lanes,
                                               uint32_t& scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (x[i] != x[i]) x[i] = 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, 1));
  const float u = __fdiv_rn(amax, __fmul_rn(g, 6.f));
  const __nv_fp8_storage_t s =
      u > 0.f ? __nv_cvt_float_to_fp8(u, __NV_SATFINITE, __NV_E4M3) : (__nv_fp8_storage_t)0;
  scale = s;
  const float step = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3))), g);
  if (!(step > 0.f)) return 0u;
  // A code only depends on which side of seven borders the quotient falls.
  // x times the reciprocal is off by at most 2^-22 of it (two roundings, a
  // subnormal reciprocal aside), so where that much more and that much less
  // give the same codes, the quotient does too; else (a border that near:
  // about one block of 10^5) the quotients are formed.
  const float r = __frcp_rn(step);
  uint32_t out = 0, other = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __fmul_rn(x[2 * i], r), b = __fmul_rn(x[2 * i + 1], r);
    constexpr float kMore = 1.f + 0x1p-21f, kLess = 1.f - 0x1p-21f;
    out |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(__fmul_rn(a, kLess), __fmul_rn(b, kLess)),
                                              __NV_E2M1, cudaRoundNearest) << (8 * i);
    other |= (uint32_t)__nv_cvt_float2_to_fp4x2(
                 make_float2(__fmul_rn(a, kMore), __fmul_rn(b, kMore)), __NV_E2M1,
                 cudaRoundNearest) << (8 * i);
  }
  if (out == other && step >= 0x1p-100f && step <= 0x1p100f) return out;
  out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(x[2 * i], step), __fdiv_rn(x[2 * i + 1], step));
    out |= (uint32_t)__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return out;
}

// Eight float32 values -> eight e4m3 codes: value / scale rounded to float32
// (IEEE division), then e4m3 RNE, saturating.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float s) {
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
    const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    if (i & 1)
      out[i >> 1] |= (uint32_t)b << 16;
    else
      out[i >> 1] = (uint32_t)b;
  }
  return make_uint2(out[0], out[1]);
}

// Eight bf16 (one 16-byte load) -> eight float32.
__device__ __forceinline__ void unpack8(const uint4& in, float (&x)[8]) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

}  // namespace tfpa
