// From the q / k / v projection to the cache: rotary tables, and a
// projection's rows normed, rotated, handed out (q) and stored (K, V).
//
// Tables.  cos and sin of position t and frequency f are those of the
// fraction of a turn t f / 2 pi mod 1.  f / 2 pi is kept as a fraction of
// 2^64, so the product modulo one turn is a 64-bit integer product that
// wraps: exact for the fraction as it is kept, at any position, where an angle in
// float32 would have lost its low bits and one in float64 costs its slow sine.  The
// fraction is taken to within an eighth of a turn of a quarter turn (its top bits) and
// only then rounded to float32.  Bound by the stores, 8 bytes an entry: 131,072
// positions of 64 frequencies (67 MB) in 11.5 us, 5.8 TB/s, the integer pipe close
// behind (five instructions an entry more, for the signs, cost 0.7 us).
//
// Rows.  A half-warp takes a q head, or a kv head's K and V, of a row, and where
// there are rows enough several times four q heads or two kv heads: their
// loads are then in flight together, they share the row's angles and the
// weights, and their roots are taken at once.  A thread holds 8 head dims.  The mean
// square is added up pair by pair (a thread's 8, then lanes 1, 2, 4, 8
// apart), and every product, sum, quotient and root is rounded to float32 on
// its own, so that the stored codes are a function of the inputs alone.  Bound by a
// warp's chain from its loads over the root to its stores, and by how many such
// chains the registers of 16 warps a SM allow: 4,096 rows of 32, 8 and 8 heads over
// bf16 (103 MB) in 25.6 us, 4.0 TB/s; over e4m3 (94 MB) and 4 bits (91 MB) in 29 us,
// 3.2 TB/s, for a quarter and a third more instructions (issue 59 and 61 %); 2,044 rows
// over 4 bits (45 MB, neighbouring dims, no norm) in 14.8 us; eight rows in 2.8 us (e4m3
// and 4 bits 3.4), two latencies.
// (No read-only loads in these kernels and the block kernels: they may start
// while the kernel before them still writes what they will read.)
#include <cuda_fp8.h>

#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {

namespace {
constexpr int kTableThreads = 256;
constexpr int kTableBlocks = 5;             // of a SM

// sin and cos of |x| <= pi / 4, times scale + rest, by their Taylor polynomials, cut
// where the next term is below 2^-29 (x^11 / 11! and x^12 / 12!).  The factor goes in
// before the last step, whose rounding is then most of a value's error.
__device__ __forceinline__ void sin_cos(float x, float scale, float rest, float& sn, float& cs) {
  const float y = x * x, z = x * scale;
  float a = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(y, a, 1.f / 120.f);
  a = fmaf(y, a, -1.f / 6.f);
  sn = fmaf(z * y, a, z);
  float b = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  b = fmaf(y, b, -1.f / 720.f);
  b = fmaf(y, b, 1.f / 24.f);
  b = fmaf(y, b, -0.5f);
  cs = fmaf(y * scale, b, rest) + scale;
}

// x, its sign flipped where the top bit of w is set.
__device__ __forceinline__ float signed_as(float x, uint32_t w) {
  return __uint_as_float(__float_as_uint(x) ^ (w & 0x80000000u));
}
}  // namespace

// A thread keeps four frequencies and walks over rows, the whole grid at a time:
// a position's fractions are the last one's and a step's (indexing the launch
// parameters by lane costs a pass through the constant cache each).
__global__ void __launch_bounds__(kTableThreads, kTableBlocks)
    rope_table_kernel(const __grid_constant__ TableParams p) {
  allow_next_grid();
  wait_prior_grid();
  const int quads = p.half / 4, rows = kTableThreads / quads;
  const int r = threadIdx.x / quads, f0 = (threadIdx.x - r * quads) * 4;
  if (r >= rows) return;
  int64_t row = (int64_t)blockIdx.x * rows + r;
  const int64_t step = (int64_t)gridDim.x * rows;
  uint64_t at[4], more[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t f = p.turns[f0 + j];
    at[j] = f * (uint64_t)(p.first + row);
    more[j] = f * (uint64_t)step;
  }
  for (; row < p.n; row += step) {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t turn = at[j];
      at[j] += more[j];
      // the nearest quarter turn (the top two bits of hi), and what is left of it (at
      // most an eighth) in radians; the low word counts where the angle itself is small
      const uint32_t hi = (uint32_t)(turn >> 32) + (1u << 29);
      const float x = fmaf((float)((int32_t)(hi & 0x3FFFFFFFu) - (1 << 29)), 0x1p32f,
                           (float)(uint32_t)turn) *
                      (float)(6.283185307179586 * 0x1p-64);
      float sn, cs;
      sin_cos(x, p.attn_scale, p.attn_rest, sn, cs);
      const bool odd = hi & 0x40000000u;
      c[j] = signed_as(odd ? sn : cs, hi + 0x40000000u);
      s[j] = signed_as(odd ? cs : sn, hi);
    }
    const size_t to = (size_t)row * p.half + f0;
    *reinterpret_cast<float4*>(p.cos + to) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(p.sin + to) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

namespace {

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8f(const float* a, float (&x)[8]) {
  const float4 u = *(reinterpret_cast<const float4*>(a));
  const float4 v = *(reinterpret_cast<const float4*>(a) + 1);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}

// Every exchange is the whole warp's, whose halves go through their heads in step:
// one under a mask of 16 lanes costs several instructions more (4,096 rows of 40
// heads 30 us).
constexpr unsigned kAll = 0xFFFFFFFFu;

// A lane's eight dims as pairs of floats, dims i and i + 4 in one: sums over
// neighbours then take both halves of the eight at once.
struct Dims {
  f2 v[4];
};
__device__ __forceinline__ Dims unpack(const uint4& w) {
  auto lo = [](uint32_t a) { return __uint_as_float(a << 16); };
  auto hi = [](uint32_t a) { return __uint_as_float(a & 0xFFFF0000u); };
  Dims d;
  d.v[0] = f2{lo(w.x), lo(w.z)};
  d.v[1] = f2{hi(w.x), hi(w.z)};
  d.v[2] = f2{lo(w.y), lo(w.w)};
  d.v[3] = f2{hi(w.y), hi(w.w)};
  return d;
}
__device__ __forceinline__ Dims dims_of(const float (&x)[8]) {
  Dims d;
#pragma unroll
  for (int i = 0; i < 4; ++i) d.v[i] = f2{x[i], x[i + 4]};
  return d;
}
__device__ __forceinline__ void floats_of(const Dims& d, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = d.v[i].x;
    x[i + 4] = d.v[i].y;
  }
}

// (A packed sum of packed products would become a packed multiply-add, rounded
// once: sums of products are scalar.)
__device__ __forceinline__ f2 add_each(f2 a, f2 b) {
  return f2{__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)};
}

// The lane's share of the sum of squares: neighbours first.
__device__ __forceinline__ float squares(const Dims& d) {
  const f2 a = add_each(fmul2(d.v[0], d.v[0]), fmul2(d.v[1], d.v[1]));
  const f2 b = add_each(fmul2(d.v[2], d.v[2]), fmul2(d.v[3], d.v[3]));
  const f2 c = add_each(a, b);
  return __fadd_rn(c.x, c.y);
}

// 1 / sqrt(mean square + eps) of H heads from the lanes' shares.  Four heads:
// the lanes 1 and 2 apart split the heads among them while they add, so that
// each lane sums, and takes the root of, one head, and the roots are handed
// round.  Every sum is the same pair of numbers as one head alone would add.
template <int H>
__device__ __forceinline__ void roots(float (&s)[H], float eps, int t) {
  auto root = [&](float sum) {
    return __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / kHeadDim), eps)));
  };
  if (H == 4) {
    const bool b0 = t & 1, b1 = t & 2;
    float k0 = b0 ? s[2 % H] : s[0], k1 = b0 ? s[3 % H] : s[1 % H];
    k0 = __fadd_rn(k0, __shfl_xor_sync(kAll, b0 ? s[0] : s[2 % H], 1));
    k1 = __fadd_rn(k1, __shfl_xor_sync(kAll, b0 ? s[1 % H] : s[3 % H], 1));
    float k = __fadd_rn(b1 ? k1 : k0, __shfl_xor_sync(kAll, b1 ? k0 : k1, 2));
    k = __fadd_rn(k, __shfl_xor_sync(kAll, k, 4));
    k = __fadd_rn(k, __shfl_xor_sync(kAll, k, 8));
    const float inv = root(k);
#pragma unroll
    for (int h = 0; h < H; ++h)
      s[h] = __shfl_sync(kAll, inv, (threadIdx.x & 16) + (h >> 1) + 2 * (h & 1));
  } else {
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int d = 1; d < 16; d *= 2) s[h] = __fadd_rn(s[h], __shfl_xor_sync(kAll, s[h], d));
      s[h] = root(s[h]);
    }
  }
}

// How a lane's eight dims turn: cos and sin of its pairs, and where the other
// halves of the pairs are.  (Interleaved: pairs of neighbours, four of each.)
struct Turn {
  Dims c, s;               // s negated where a lane holds the pairs' first dims
  int from;                // the lane (of the warp) that holds the partners
  bool on;                 // this lane's dims turn
};

__device__ __forceinline__ Turn make_turn(const QkvParams& p, int rpos, int t) {
  Turn u;
  const int half = p.rot_dim / 2;
  const size_t row = (size_t)rpos * half;
  u.from = 0;
  u.on = t * 8 < p.rot_dim;
  if (p.interleaved) {                       // dims 2i and 2i + 1: a lane's own
    if (!u.on) return u;
    const float4 c4 = *(reinterpret_cast<const float4*>(p.rope_cos + row + t * 4));
    const float4 s4 = *(reinterpret_cast<const float4*>(p.rope_sin + row + t * 4));
    const float c[8] = {c4.x, c4.x, c4.y, c4.y, c4.z, c4.z, c4.w, c4.w};
    const float s[8] = {-s4.x, s4.x, -s4.y, s4.y, -s4.z, s4.z, -s4.w, s4.w};
    u.c = dims_of(c);
    u.s = dims_of(s);
    return u;
  }
  const int hl = half / 8;                   // dims i and i + half: half / 8 lanes apart
  const bool second = t >= hl;
  u.from = (threadIdx.x & 16) + (!u.on ? t : second ? t - hl : t + hl);
  if (!u.on) return u;
  const int i0 = (second ? t - hl : t) * 8;
  float c[8], s[8];
  load8f(p.rope_cos + row + i0, c);
  load8f(p.rope_sin + row + i0, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = second ? s[i] : -s[i];
  u.c = dims_of(c);
  u.s = dims_of(s);
  return u;
}

// Eight dims of a head rotated: a c - b s and b c + a s are both the dim's own
// product and, rounded on its own, its partner's under sin's sign.  The whole warp
// takes part in the exchange.
__device__ __forceinline__ void rotate(Dims& x, const Turn& u, bool interleaved) {
  Dims o;
  if (interleaved) {                         // dims 0, 1 and 2, 3 of each four
    o.v[0] = x.v[1];
    o.v[1] = x.v[0];
    o.v[2] = x.v[3];
    o.v[3] = x.v[2];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[i].x = __shfl_sync(kAll, x.v[i].x, u.from);
      o.v[i].y = __shfl_sync(kAll, x.v[i].y, u.from);
    }
  }
  if (!u.on) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x.v[i] = add_each(fmul2(x.v[i], u.c.v[i]), fmul2(o.v[i], u.s.v[i]));
}

// A row's K (x, and kx as bf16) and V of one kv head into the cache, if it is
// there; the whole warp comes here.
template <int KV>
__device__ __forceinline__ void store_kv(const QkvParams& p, const WriteRun& run, size_t dst_row,
                                         int g, int t, bool live, float (&x)[8],
                                         const uint4& kx, const uint4& vv) {
  if (KV == kKvBf16) {
    if (!live) return;
    __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(run.k_dst) + dst_row * kHeadDim + t * 8;
    __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(run.v_dst) + dst_row * kHeadDim + t * 8;
    *reinterpret_cast<uint4*>(kd) = kx;
    *reinterpret_cast<uint4*>(vd) = vv;
    return;
  }
  float vf[8];
  unpack8(vv, vf);
  uint8_t* kb = static_cast<uint8_t*>(run.k_dst);
  uint8_t* vb = static_cast<uint8_t*>(run.v_dst);
  const float gk = *(p.k_scale + g), gv = *(p.v_scale + g);
  if (KV == kKvFp4) {
    const size_t codes = fp4_codes(dst_row) + t * 4, scales = fp4_scales(dst_row) + (t >> 1);
    uint32_t ks, vs;
    const uint32_t kc = quant8_fp4(x, gk, kAll, ks), vc = quant8_fp4(vf, gv, kAll, vs);
    if (!live) return;
    *reinterpret_cast<uint32_t*>(kb + codes) = kc;
    *reinterpret_cast<uint32_t*>(vb + codes) = vc;
    if (!(t & 1)) {
      kb[scales] = (uint8_t)ks;
      vb[scales] = (uint8_t)vs;
    }
    return;
  }
  if (!live) return;
  *reinterpret_cast<uint2*>(kb + dst_row * kHeadDim + t * 8) = quant8(x, gk);
  *reinterpret_cast<uint2*>(vb + dst_row * kHeadDim + t * 8) = quant8(vf, gv);
}

}  // namespace

// A warp takes an equal run of the call's units in row order; a unit is a pair of
// steps, one a half-warp: H query heads, or half as many kv heads (but one) with
// their K and V.  A row's angles, and the weights, stay in registers.
template <int KV, int H>
__global__ void __launch_bounds__(H > 1 ? 256 : 64, H > 1 ? 2 : 8)
    write_qkv_kernel(const __grid_constant__ QkvParams p) {
  constexpr int HK = H > 1 ? H / 2 : 1;
  allow_next_grid();
  wait_prior_grid();
  const int wid = blockIdx.x * (blockDim.x / 32) + (int)same_in_warp(threadIdx.x >> 5);
  if (wid >= p.warps) return;
  const int t = threadIdx.x & 15;                          // 8-element slice
  const int side = (threadIdx.x >> 4) & 1;                 // half-warp: its step of a unit
  const int q_units = (p.q_heads + 2 * H - 1) / (2 * H);
  const int units = q_units + (p.hkv + 2 * HK - 1) / (2 * HK);
  const int64_t all = (int64_t)p.rows * units;
  int left = (int)(all * (wid + 1) / p.warps);
  int unit = (int)(all * wid / p.warps);
  left -= unit;
  int row = unit / units;
  unit -= row * units;
  int ri = run_holding(p.runs, p.nruns, &WriteRun::row0, row);

  uint4 in[H], vin[HK];
  Turn turn;
  Dims w;
  float inv[H];
  int pos = 0, pid = 0;
  const float* weight = nullptr;           // whose values w holds
  bool fresh = true, on_table = true;      // a row's first unit of this warp; its angles are there
  for (; left > 0; --left) {
    const bool is_q = unit < q_units;
    // ---- the unit's dims are on their way before anything else is looked at.  n:
    // heads that are there (none: a half-warp that only keeps in step)
    const int h0 = is_q ? (2 * unit + side) * H : (2 * (unit - q_units) + side) * HK;
    const int n = is_q ? p.q_heads - h0 : min(HK, p.hkv - h0);
    const __nv_bfloat16* from =
        (is_q ? p.q + (size_t)row * p.q_stride : p.k + (size_t)row * p.k_stride) +
        h0 * kHeadDim + t * 8;
#pragma unroll
    for (int h = 0; h < H; ++h)
      in[h] = h < n ? *(reinterpret_cast<const uint4*>(from + h * kHeadDim))
                    : make_uint4(0, 0, 0, 0);
    if (!is_q) {
      const __nv_bfloat16* vp = p.v + (size_t)row * p.v_stride + h0 * kHeadDim + t * 8;
#pragma unroll
      for (int h = 0; h < HK; ++h)
        vin[h] = h < n ? *(reinterpret_cast<const uint4*>(vp + h * kHeadDim))
                       : make_uint4(0, 0, 0, 0);
    }
    if (fresh) {
      while (ri + 1 < p.nruns && p.runs[ri + 1].row0 <= row) ++ri;
      const WriteRun& run = p.runs[ri];
      pos = run.pos0 + (row - run.row0);
      pid = run.page_table ? *(run.page_table + (pos >> 8)) : 0;
      if (p.rope_cos) {
        const int rpos = p.rope_pos ? *(p.rope_pos + row) : pos;
        on_table = (unsigned)rpos < (unsigned)p.rope_n;    // the whole warp's row
        if (on_table)
          turn = make_turn(p, rpos, t);
        else if ((threadIdx.x & 31) == 0)
          flag_error(p.err_flag, kErrRopeRange);
      }
      fresh = false;
    }
    const float* need = is_q ? p.q_weight : p.k_weight;
    if (need && need != weight) {
      float f[8];
      load8f(need + t * 8, f);
      w = dims_of(f);
      weight = need;
    }
    const WriteRun& run = p.runs[ri];
    const bool on_page = is_q || !run.page_table || (unsigned)pid < (unsigned)p.num_pages;
    if (!on_page && (threadIdx.x & 31) == 0) flag_error(p.err_flag, kErrBadPage);
    if (on_table && on_page) {
      // ---- the heads' roots together; then head by head
      const bool turns = need || p.rope_cos;
      if (need) {
#pragma unroll
        for (int h = 0; h < H; ++h) inv[h] = squares(unpack(in[h]));
        roots<H>(inv, p.eps, t);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (!is_q && h >= HK) break;
        Dims x = unpack(in[h]);
        if (need) {
          const f2 r = f2{inv[h], inv[h]};
#pragma unroll
          for (int i = 0; i < 4; ++i) x.v[i] = fmul2(fmul2(x.v[i], r), w.v[i]);
        }
        if (p.rope_cos) rotate(x, turn, p.interleaved);
        float f[8];
        floats_of(x, f);
        const uint4 y = turns ? pack8(f) : in[h];
        const bool live = h < n;
        if (is_q) {
          if (live)
            *reinterpret_cast<uint4*>(
                p.q_out + ((size_t)row * p.q_heads + h0 + h) * kHeadDim + t * 8) = y;
        } else if (h < HK) {
          const int g = live ? h0 + h : 0;
          const size_t dst_row = run.page_table
                                     ? ((size_t)pid * p.hkv + g) * kPage + (pos & (kPage - 1))
                                     : (size_t)g * run.slab_cap + pos;
          store_kv<KV>(p, run, dst_row, g, t, live, f, y, vin[h < HK ? h : 0]);
        }
      }
    }
    if (++unit == units) {
      unit = 0;
      ++row;
      fresh = true;
    }
  }
}

cudaError_t launch_rope_table(const TableParams& p, int sms, cudaStream_t s) {
  const int rows = kTableThreads / (p.half / 4);
  const int grid = (int)min((int64_t)kTableBlocks * sms, ((int64_t)p.n + rows - 1) / rows);
  return launch_pdl(rope_table_kernel, dim3(grid), dim3(kTableThreads), 0, s, p);
}

namespace {
template <int KV>
cudaError_t launch_rows(const QkvParams& p, cudaStream_t s) {
  return p.wide
             ? launch_pdl(write_qkv_kernel<KV, 4>, dim3((p.warps + 7) / 8), dim3(256), 0, s, p)
             : launch_pdl(write_qkv_kernel<KV, 1>, dim3((p.warps + 1) / 2), dim3(64), 0, s, p);
}
}  // namespace

cudaError_t launch_write_qkv(const QkvParams& p, int kv, cudaStream_t s) {
  return kv == kKvBf16  ? launch_rows<kKvBf16>(p, s)
         : kv == kKvFp8 ? launch_rows<kKvFp8>(p, s)
                        : launch_rows<kKvFp4>(p, s);
}

}  // namespace tfpa
