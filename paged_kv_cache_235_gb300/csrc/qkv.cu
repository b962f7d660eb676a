// From the q / k / v projection to the cache: rotary tables, and a
// projection's rows normed, rotated, handed out (q) and stored (K, V).
//
// Tables.  cos and sin of position t and frequency f are those of the
// fraction of a turn t f / 2 pi mod 1.  f / 2 pi is kept as a fraction of
// 2^64, so the product modulo one turn is a 64-bit integer product that
// wraps: exact for any position, where an angle in float32 would have lost
// its low bits and one in float64 costs its slow sine.  The fraction is
// taken to within an eighth of a turn of a quarter turn (its top bits) and
// only then rounded to float32.  Bound by the stores, 8 bytes an entry.
//
// Rows.  One 16-thread group per (row, head) as in the KV write kernel, a
// q head or a kv head's K and V; a thread holds 8 head dims.  The mean
// square is added up pair by pair (a thread's 8, then lanes 1, 2, 4, 8
// apart), and every product, sum, quotient and root is rounded to float32 on
// its own, so that the stored codes are a function of the inputs alone.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {

namespace {
constexpr int kTableThreads = 256;
}

__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(const __grid_constant__ TableParams p) {
  allow_next_grid();
  wait_prior_grid();
  const int quads = p.half / 4;                    // four frequencies a thread
  const int64_t i = (int64_t)blockIdx.x * kTableThreads + threadIdx.x;
  if (i >= (int64_t)p.n * quads) return;
  const int64_t row = i / quads;
  const int f0 = (int)(i - row * quads) * 4;
  const uint64_t t = (uint64_t)(p.first + row);
  float c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t turn = t * p.turns[f0 + j];
    // the nearest quarter turn, and what is left of it in half turns
    const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
    const float x = (float)(int64_t)(turn - ((uint64_t)quarter << 62)) * 0x1p-63f;
    float sn, cs;
    sincospif(x, &sn, &cs);
    const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
    c[j] = p.attn_scale * (quarter == 1 || quarter == 2 ? -a : a);
    s[j] = p.attn_scale * (quarter >= 2 ? -b : b);
  }
  const size_t at = (size_t)row * p.half + f0;
  *reinterpret_cast<float4*>(p.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
  *reinterpret_cast<float4*>(p.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
}

namespace {

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// x over the root of its mean square over the head, times w.
__device__ __forceinline__ void norm8(float (&x)[8], const float* w, float eps, int t,
                                      unsigned lanes) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s[i] = __fadd_rn(__fmul_rn(x[2 * i], x[2 * i]), __fmul_rn(x[2 * i + 1], x[2 * i + 1]));
  float sum = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) sum = __fadd_rn(sum, __shfl_xor_sync(lanes, sum, d));
  const float inv =
      __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / kHeadDim), eps)));
  const float4* wp = reinterpret_cast<const float4*>(w + t * 8);
  const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
  const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), wv[i]);
}

// The first rot_dim dims of a head rotated by table row `rpos`.  All 16 lanes
// take part in the exchange.
__device__ __forceinline__ void rotate8(float (&x)[8], const QkvParams& p, int rpos, int t,
                                        unsigned lanes) {
  const int half = p.rot_dim / 2;
  const float* cp = p.rope_cos + (size_t)rpos * half;
  const float* sp = p.rope_sin + (size_t)rpos * half;
  if (p.interleaved) {                       // dims 2i and 2i + 1: a thread's own
    if (t * 8 >= p.rot_dim) return;
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cp + t * 4));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sp + t * 4));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    }
    return;
  }
  // dims i and i + half: the thread half / 8 lanes away holds the partners
  const int hl = half / 8;
  const bool second = t >= hl;
  const int from = (threadIdx.x & 16) + (t >= 2 * hl ? t : second ? t - hl : t + hl);
  float other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(lanes, x[i], from);
  if (t >= 2 * hl) return;
  const int i0 = (second ? t - hl : t) * 8;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(cp + i0));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(cp + i0 + 4));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(sp + i0));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(sp + i0 + 4));
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = second ? other[e] : x[e];   // dim i
    const float b = second ? x[e] : other[e];   // dim i + half
    x[e] = second ? __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]))
                  : __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
  }
}

}  // namespace

__global__ void __launch_bounds__(256) write_qkv_kernel(const __grid_constant__ QkvParams p) {
  allow_next_grid();
  wait_prior_grid();
  const int slots = p.q_heads + p.hkv;                     // heads of a row: q, then kv
  const int gid = blockIdx.x * 16 + (threadIdx.x >> 4);
  const int t = threadIdx.x & 15;                          // 8-element slice
  if (gid >= p.rows * slots) return;
  const unsigned lanes = 0xFFFFu << (threadIdx.x & 16);    // the head's 16 threads
  const int row = gid / slots;
  const int slot = gid - row * slots;
  int ri = 0;
  while (ri + 1 < p.nruns && p.runs[ri + 1].row0 <= row) ++ri;
  const WriteRun& run = p.runs[ri];
  const int pos = run.pos0 + (row - run.row0);
  int rpos = pos;
  if (p.rope_cos && p.rope_pos) rpos = __ldg(p.rope_pos + row);
  const bool off_table = p.rope_cos && (unsigned)rpos >= (unsigned)p.rope_n;
  float x[8];
  if (slot < p.q_heads) {
    const uint4 in = *reinterpret_cast<const uint4*>(p.q + (size_t)row * p.q_stride +
                                                     slot * kHeadDim + t * 8);
    if (off_table) {                                       // all 16 lanes alike
      if (t == 0) flag_error(p.err_flag, kErrRopeRange);
      return;
    }
    unpack8(in, x);
    if (p.q_weight) norm8(x, p.q_weight, p.eps, t, lanes);
    if (p.rope_cos) rotate8(x, p, rpos, t, lanes);
    *reinterpret_cast<uint4*>(p.q_out + ((size_t)row * p.q_heads + slot) * kHeadDim + t * 8) =
        p.q_weight || p.rope_cos ? pack8(x) : in;
    return;
  }
  const int g = slot - p.q_heads;
  const int pid = run.page_table ? __ldg(run.page_table + (pos >> 8)) : 0;
  const uint4 kv = *reinterpret_cast<const uint4*>(p.k + (size_t)row * p.k_stride +
                                                   g * kHeadDim + t * 8);
  const uint4 vv = *reinterpret_cast<const uint4*>(p.v + (size_t)row * p.v_stride +
                                                   g * kHeadDim + t * 8);
  if (off_table) {
    if (t == 0) flag_error(p.err_flag, kErrRopeRange);
    return;
  }
  size_t dst_row;
  if (run.page_table) {
    if ((unsigned)pid >= (unsigned)p.num_pages) {
      if (t == 0) flag_error(p.err_flag, kErrBadPage);
      return;
    }
    dst_row = ((size_t)pid * p.hkv + g) * kPage + (pos & (kPage - 1));
  } else {
    dst_row = (size_t)g * run.slab_cap + pos;
  }
  unpack8(kv, x);
  if (p.k_weight) norm8(x, p.k_weight, p.eps, t, lanes);
  if (p.rope_cos) rotate8(x, p, rpos, t, lanes);
  if (p.kv == kKvBf16) {
    __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(run.k_dst) + dst_row * kHeadDim + t * 8;
    __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(run.v_dst) + dst_row * kHeadDim + t * 8;
    *reinterpret_cast<uint4*>(kd) = p.k_weight || p.rope_cos ? pack8(x) : kv;
    *reinterpret_cast<uint4*>(vd) = vv;
    return;
  }
  float vf[8];
  unpack8(vv, vf);
  uint8_t* kb = static_cast<uint8_t*>(run.k_dst);
  uint8_t* vb = static_cast<uint8_t*>(run.v_dst);
  if (p.kv == kKvFp4) {
    const size_t codes = fp4_codes(dst_row) + t * 4, scales = fp4_scales(dst_row) + (t >> 1);
    uint32_t ks, vs;
    *reinterpret_cast<uint32_t*>(kb + codes) = quant8_fp4(x, __ldg(p.k_scale + g), lanes, ks);
    *reinterpret_cast<uint32_t*>(vb + codes) = quant8_fp4(vf, __ldg(p.v_scale + g), lanes, vs);
    if (!(t & 1)) {
      kb[scales] = (uint8_t)ks;
      vb[scales] = (uint8_t)vs;
    }
    return;
  }
  *reinterpret_cast<uint2*>(kb + dst_row * kHeadDim + t * 8) = quant8(x, __ldg(p.k_scale + g));
  *reinterpret_cast<uint2*>(vb + dst_row * kHeadDim + t * 8) = quant8(vf, __ldg(p.v_scale + g));
}

cudaError_t launch_rope_table(const TableParams& p, cudaStream_t s) {
  const int64_t threads = (int64_t)p.n * (p.half / 4);
  const int grid = (int)((threads + kTableThreads - 1) / kTableThreads);
  return launch_pdl(rope_table_kernel, dim3(grid), dim3(kTableThreads), 0, s, p);
}

cudaError_t launch_write_qkv(const QkvParams& p, cudaStream_t s) {
  const int heads = p.rows * (p.q_heads + p.hkv);
  return launch_pdl(write_qkv_kernel, dim3((heads + 15) / 16), dim3(256), 0, s, p);
}

}  // namespace tfpa
