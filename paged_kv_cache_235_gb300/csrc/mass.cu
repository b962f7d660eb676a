// Accumulated attention weight of the cached keys: for every segment with
// rows in the call, kv head g and key j
//   mass[s][g][j] = decay mass[s][g][j]
//                   + sum over rows r at or after j, heads h of g, of
//                     2^(q_rh . k_j scale log2(e) - lse[r][h] log2(e)),
// the weights that the rows' attention (which left lse) gave the key.  K is
// read once and V not at all.
//
// A block of four warps takes 128 keys of one (segment, kv head), 32 a warp.
// A warp turns its keys into the A fragments of mma.sync m16n8k16 (keys x
// head dims) straight from global memory, every load issued before the first
// use, and keeps them while the segment's query vectors pass by, eight at a
// time, as B fragments from shared memory.  So a key's weights lie in four
// neighbouring lanes' registers, their sum needs two shuffles at the very
// end, and one thread owns a key's entry: no atomics, and a fixed order.
// e4m3 and 4-bit keys go through f16 (exact), with each query vector scaled
// into f16 range by a power of two.
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32 * kWarps;       // keys of a block
constexpr int kVec = 64;                 // query vectors staged at once
constexpr int kQStride = 320;            // bytes: eight rows' 64-byte reads fall in all banks

// Byte offset, within a staged query vector, of head dim d (a multiple of
// 8).  Lane c of a quad holds 32 of a key's head dims, 16 bytes of the
// cache's row at a time; its j-th 16 bytes of the query sit at 64 j + 16 c.
template <int KV>
__device__ __forceinline__ int q_off(int d) {
  if (KV == kKvBf16) return d * 2;
  if (KV == kKvFp8) {
    const int id = d >> 4;
    return (2 * (id >> 2) + ((d >> 3) & 1)) * 64 + (id & 3) * 16;
  }
  return ((d & 31) >> 3) * 64 + (d >> 5) * 16;
}

// Lane (gq, c)'s 32 head dims of one stored row, as 16 operand pairs.
template <int KV>
struct RawRow {
  uint4 w[KV == kKvBf16 ? 4 : KV == kKvFp8 ? 2 : 1];
  uint16_t s;
  __device__ __forceinline__ void load(const uint8_t* base, size_t row, int c) {
    if (KV == kKvFp4) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(base + fp4_codes(row)) + c);
      s = __ldg(reinterpret_cast<const uint16_t*>(base + fp4_scales(row)) + c);
    } else {
      constexpr int n = KV == kKvBf16 ? 4 : 2;
      const uint4* p = reinterpret_cast<const uint4*>(base + row * (n * 64)) + c;
#pragma unroll
      for (int j = 0; j < n; ++j) w[j] = __ldg(p + 4 * j);
    }
  }
  __device__ __forceinline__ void pairs(uint32_t (&r)[16]) const {
    if (KV == kKvBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[4 * j] = w[j].x;
        r[4 * j + 1] = w[j].y;
        r[4 * j + 2] = w[j].z;
        r[4 * j + 3] = w[j].w;
      }
    } else if (KV == kKvFp8) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[8 * j + 2 * i] = e4m3x2_to_f16x2((uint16_t)(v[i] & 0xFFFF));
          r[8 * j + 2 * i + 1] = e4m3x2_to_f16x2((uint16_t)(v[i] >> 16));
        }
      }
    } else {
      const uint32_t s2 = e4m3x2_to_f16x2(s);
      const uint32_t sc[2] = {prmt(s2, s2, 0x1010), prmt(s2, s2, 0x3232)};
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[4];
        e2m1x8_to_f16x8(v[i], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[4 * i + j] = hmul2(h[j], sc[i >> 1]);
      }
    }
  }
};

template <int KV>
__global__ void __launch_bounds__(32 * kWarps) key_mass_kernel(
    const __grid_constant__ MassParams p) {
  __shared__ __align__(16) uint8_t q_s[kVec * kQStride];
  __shared__ float sc_s[kVec], lse_s[kVec];
  __shared__ int lim_s[kVec];
  allow_next_grid();
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, c = lane & 3;
  int si = 0;
  while (si + 1 < p.nsegs && p.segs[si + 1].item0 <= (int)blockIdx.x) ++si;
  const MassSeg& sg = p.segs[si];
  const int tiles = (sg.seq_len + kKeys - 1) / kKeys;
  const int local = blockIdx.x - sg.item0;
  const int g = local / tiles;
  const int key0 = (local - g * tiles) * kKeys;
  size_t row0;                                            // storage row of key0
  if (sg.page_table) {
    const int pid = __ldg(sg.page_table + (key0 >> 8));
    if ((unsigned)pid >= (unsigned)p.num_pages) {         // its keys keep their entries
      if (threadIdx.x == 0) flag_error(p.err_flag, kErrBadPage);
      return;
    }
    row0 = ((size_t)pid * p.hkv + g) * kPage + (key0 & (kPage - 1));
  } else {
    row0 = (size_t)g * sg.slab_cap + key0;
  }
  // ---- this warp's 32 keys as A fragments: m-tile t holds keys 16 t + gq
  // and 16 t + 8 + gq of the warp
  const int wkey = key0 + 32 * warp;
  uint32_t a[2][2][16];
  if (wkey < sg.seq_len) {
    RawRow<KV> raw[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr)
        raw[t][hr].load(static_cast<const uint8_t*>(sg.k_base),
                        row0 + 32 * warp + 16 * t + 8 * hr + gq, c);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) raw[t][hr].pairs(a[t][hr]);
  }
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  const float ks = KV == kKvBf16 ? 1.f : __ldg(p.k_scale + g);
  const int G = p.group;
  for (int ri = sg.run0; ri < sg.run0 + sg.nruns; ++ri) {
    const MassRun ru = p.runs[ri];
    if (ru.pos0 + ru.nrows - 1 < key0) continue;          // no row of it sees the block's keys
    const int nq = ru.nrows * G;
    for (int v0 = 0; v0 < nq; v0 += kVec) {
      const int nv = min(kVec, nq - v0);
      __syncthreads();                                    // the previous vectors are done with
      // four threads a vector, 32 head dims each
      for (int i = threadIdx.x >> 2; i < ((nv + 7) & ~7); i += 8 * kWarps) {
        const int part = threadIdx.x & 3;
        const int v = v0 + i;
        uint4 w[4];
        int lim = -1;
        float sc = 0.f, l2 = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = make_uint4(0, 0, 0, 0);
        if (i < nv) {
          const int r = v / G;
          const int h = g * G + (v - r * G);
          const size_t rh = (size_t)(ru.row0 + r) * p.hq + h;
          const uint4* qp = reinterpret_cast<const uint4*>(p.q + rh * kHeadDim) + 4 * part;
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = __ldg(qp + j);
          lim = ru.pos0 + r;
          sc = p.scale_log2 * ks;
          const float lse = __ldg(p.lse + rh);
          // a row without keys has lse -inf and gives no weight
          l2 = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
        }
        if (KV != kKvBf16) {
          // f16, the vector's largest magnitude brought into [2^13, 2^14):
          // exact for every element within 2^28 of it
          float amax = 0.f;
          uint32_t* e = reinterpret_cast<uint32_t*>(w);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            amax = fmaxf(amax, fabsf(__uint_as_float(e[j] << 16)));
            amax = fmaxf(amax, fabsf(__uint_as_float(e[j] & 0xFFFF0000u)));
          }
          const unsigned quad = 0xFu << (lane & 28);      // a vector's four threads
          amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
          int ex;
          frexpf(amax, &ex);
          ex = max(min(ex, 120), -100);
          const float up = __int_as_float((127 + 14 - ex) << 23);
          sc *= __int_as_float((127 - 14 + ex) << 23);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            e[j] = pack_f16x2(__uint_as_float(e[j] << 16) * up,
                              __uint_as_float(e[j] & 0xFFFF0000u) * up);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(q_s + i * kQStride + q_off<KV>(32 * part + 8 * j)) = w[j];
        if (part == 0) {
          sc_s[i] = sc;
          lse_s[i] = l2;
          lim_s[i] = lim;
        }
      }
      __syncthreads();
      if (wkey >= sg.seq_len) continue;
      for (int n0 = 0; n0 < nv; n0 += 8) {
        uint32_t b[16];
        const uint32_t qa = smem_u32(q_s) + (n0 + gq) * kQStride + 16 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 t = lds128(qa + 64 * j);
          b[4 * j] = t.x;
          b[4 * j + 1] = t.y;
          b[4 * j + 2] = t.z;
          b[4 * j + 3] = t.w;
        }
        float d[2][4] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t af[4] = {a[t][0][2 * k], a[t][1][2 * k], a[t][0][2 * k + 1],
                                    a[t][1][2 * k + 1]};
            if (KV == kKvBf16)
              mma_bf16(d[t], af, b[2 * k], b[2 * k + 1]);
            else
              mma_f16(d[t], af, b[2 * k], b[2 * k + 1]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {                     // vectors n0 + 2 c + e
          const int v = n0 + 2 * c + e;
          const float sc = sc_s[v], l2 = lse_s[v];
          const int lim = lim_s[v];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
              const float w = fast_exp2(__fmaf_rn(d[t][2 * hr + e], sc, -l2));
              acc[t][hr] += wkey + 16 * t + 8 * hr + gq <= lim ? w : 0.f;
            }
        }
      }
    }
  }
  if (wkey >= sg.seq_len) return;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float s = acc[t][hr];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      const int key = wkey + 16 * t + 8 * hr + gq;
      if (c == 0 && key < sg.seq_len) {
        float* m = p.mass + (size_t)(sg.index * p.hkv + g) * p.mass_cap + key;
        // decay 0 does not read the old entry
        *m = sg.decay == 0.f ? s : __fmaf_rn(*m, sg.decay, s);
      }
    }
}

}  // namespace

cudaError_t launch_key_mass(const MassParams& p, int kv, int grid, cudaStream_t s) {
  if (grid <= 0) return cudaSuccess;
  const dim3 b(32 * kWarps);
  switch (kv) {
    case kKvBf16: return launch_pdl(key_mass_kernel<kKvBf16>, dim3(grid), b, 0, s, p);
    case kKvFp8: return launch_pdl(key_mass_kernel<kKvFp8>, dim3(grid), b, 0, s, p);
    default: return launch_pdl(key_mass_kernel<kKvFp4>, dim3(grid), b, 0, s, p);
  }
}

}  // namespace tfpa
