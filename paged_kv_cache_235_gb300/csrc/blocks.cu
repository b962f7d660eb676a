// Attention over a part of a long cache: bounds of the keys of each block of
// 64, 128 or 256 positions, the blocks of largest bound for a row, and
// attention over them.
//
// Bounds.  For head dim d, lo_d and hi_d are the smallest and the largest
// stored key element of a block.  A query head's score with any key of the
// block is at most sum_d max(q_d lo_d, q_d hi_d), which is linear in the
// positive and the negative part of q; summed over a kv head's query heads,
//   score = sum_d (sum_h max(q_hd, 0)) hi_d + (sum_h min(q_hd, 0)) lo_d,
// one product of 256 terms a block whatever the number of heads.  Bounds are
// held as stored values without the head's scale: those of every cache type
// are bf16 numbers, so no bound is rounded, and the scale, common to all
// blocks, does not change their order.
#include "blocks.cuh"
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

// ---------------------------------------------------------------- bounds
constexpr int kBoundThreads = 128;

// One CTA a (block, kv head): 16 lanes a row, 8 head dims a lane, 8 rows at a
// time.
template <int KV>
__global__ void __launch_bounds__(kBoundThreads)
    key_bounds_kernel(const __grid_constant__ BoundsParams p) {
  __shared__ uint4 part[2][kBoundThreads];
  allow_next_grid();
  wait_prior_grid();
  const int g = blockIdx.x % p.hkv;
  const int item = blockIdx.x / p.hkv;
  int ri = 0;
  while (ri + 1 < p.nruns && p.runs[ri + 1].item0 <= item) ++ri;
  const BoundsRun& run = p.runs[ri];
  const int block = run.block0 + (item - run.item0);
  const int64_t key0 = (int64_t)block * p.block;
  const int n = (int)min((int64_t)p.block, run.seq_len - key0);
  const int page = (int)(key0 >> 8);
  const int per_page = kPage / p.block, in_page = block % per_page;
  size_t row0, at;
  if (run.page_table) {
    const int pid = __ldg(run.page_table + page);
    if ((unsigned)pid >= (unsigned)p.num_pages) {
      if (threadIdx.x == 0) flag_error(p.err_flag, kErrBadPage);
      return;
    }
    const size_t pg = (size_t)pid * p.hkv + g;
    row0 = pg * kPage + in_page * p.block;
    at = pg * per_page + in_page;
  } else {
    row0 = (size_t)g * run.slab_cap + key0;
    at = (size_t)g * (run.slab_cap / p.block) + block;
  }
  const int t = threadIdx.x & 15;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  for (int r = threadIdx.x >> 4; r < n; r += kBoundThreads / 16) {
    float x[8];
    load8<KV>(run.k_base, row0 + r, t, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = x[i] != x[i] ? 0.f : x[i];
      lo[i] = fminf(lo[i], v);
      hi[i] = fmaxf(hi[i], v);
    }
  }
  auto pack = [](const float (&v)[8]) {      // exact: see above
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  };
  part[0][threadIdx.x] = pack(lo);
  part[1][threadIdx.x] = pack(hi);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int which = threadIdx.x >> 4;        // lanes 0-15 the smallest, 16-31 the largest
  float m[8];
  unpack8(part[which][t], m);
  for (int r = 1; r < kBoundThreads / 16; ++r) {
    float x[8];
    unpack8(part[which][r * 16 + t], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = which ? fmaxf(m[i], x[i]) : fminf(m[i], x[i]);
  }
  reinterpret_cast<uint4*>(run.bounds)[(at * 2 + which) * 16 + t] = pack(m);
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kNear = 64;                    // near candidates ranked one against all
constexpr uint32_t kTaken = 0xFFFFFFFFu;     // order key of a block that is in whatever its score
constexpr uint32_t kAbsent = 0u;             // and of one that is not

// Larger score, larger key.  Never kAbsent or kTaken for a number.
__device__ __forceinline__ uint32_t order32(float s) {
  const uint32_t b = __float_as_uint(s + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// The same of a float64 score; a NaN above every number.
__device__ __forceinline__ uint64_t order64(double s) {
  if (s != s) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

struct SelShared {
  double q64[256];           // sum_h min(q, 0) (0..127), sum_h max(q, 0) (128..255)
  uint32_t hist[256];
  uint32_t warp_s[kSelWarps];
  uint32_t digit, above, count, forced, free_blocks;
  uint32_t most;             // largest |bound|, as bits
  float q1;                  // sum_d |q64|
  int nonfinite;
  int near_i[kNear];
  uint64_t near_k[kNear];
};

__device__ __forceinline__ uint32_t sel_prefix(uint32_t x, uint32_t* warp_s, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  const uint32_t w = lane < kSelWarps ? warp_s[lane] : 0;
  uint32_t winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += y;
  }
  total = __shfl_sync(0xffffffffu, winc, 31);
  return __shfl_sync(0xffffffffu, winc - w, warp) + inc - x;
}

// Sum over the block's threads.
__device__ __forceinline__ uint32_t sel_sum(uint32_t x, uint32_t* warp_s) {
  uint32_t total;
  sel_prefix(x, warp_s, total);
  return total;
}

// This lane's 16 bytes of block b's bounds (lanes 0-15 the smallest, 16-31
// the largest), or nullptr on a page out of range.
__device__ __forceinline__ const uint4* bound_ptr(const SelectParams& p, const SelRun& run, int g,
                                                  int b, int lane) {
  const int per_page = kPage / p.block;
  size_t at;
  if (run.page_table) {
    const int pid = __ldg(run.page_table + b / per_page);
    if ((unsigned)pid >= (unsigned)p.num_pages) return nullptr;
    at = ((size_t)pid * p.hkv + g) * per_page + b % per_page;
  } else {
    at = (size_t)g * (run.slab_cap / p.block) + b;
  }
  return static_cast<const uint4*>(run.bounds) + at * 32 + lane;
}

// The score of a block from the whole warp's bounds, in 64 bits.  Every block's
// sum runs in the same order, so equal bounds give equal scores.
__device__ __forceinline__ double score64(const SelShared& sh, const uint4& w, int lane) {
  float x[8];
  unpack8(w, x);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma(sh.q64[lane * 8 + i], (double)x[i], s);
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// One CTA a (row, kv head).
__global__ void __launch_bounds__(kSelThreads)
    select_blocks_kernel(const __grid_constant__ SelectParams p) {
  __shared__ SelShared sh;
  extern __shared__ uint64_t dyn[];          // [cap] exact keys, then [cap] keys
  allow_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.hkv, g = blockIdx.x % p.hkv;
  int ri = 0;
  while (ri + 1 < p.nruns && p.runs[ri + 1].row0 <= row) ++ri;
  const SelRun& run = p.runs[ri];
  const int pos = run.pos0 + (row - run.row0);
  const int last = pos / p.block, n = last + 1;
  int32_t* out = p.blocks + ((size_t)row * p.hkv + g) * p.nsel;
  uint64_t* key64 = dyn;
  uint32_t* key32 = reinterpret_cast<uint32_t*>(dyn + p.cap);
  auto forced = [&](int b) { return b < p.sink || b > last - p.recent; };

  // ---- the query heads' positive and negative parts, summed
  if (tid == 0) {
    sh.most = 0;
    sh.nonfinite = 0;
    sh.q1 = 0.f;
  }
  __syncthreads();
  if (tid < 256) {
    const int d = tid & 127;
    const __nv_bfloat16* q = p.q + ((size_t)row * p.hq + (size_t)g * p.group) * kHeadDim + d;
    double s = 0.0;
    for (int h = 0; h < p.group; ++h) {
      const float x = __bfloat162float(q[(size_t)h * kHeadDim]);
      s += tid < 128 ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x);
    }
    sh.q64[tid] = s;
    float a = fabsf((float)s);
#pragma unroll
    for (int d2 = 16; d2; d2 >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d2);
    if (lane == 0) atomicAdd(&sh.q1, a);     // only a bound hangs on the order
  }
  __syncthreads();
  float qf[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qf[i] = (float)sh.q64[lane * 8 + i];

  // ---- every visible block's score in float32
  float most = 0.f;
  int nonfinite = 0;
  for (int b = warp; b < n; b += kSelWarps) {
    const uint4* at = bound_ptr(p, run, g, b, lane);
    uint32_t key = kAbsent;
    if (!at) {
      if (lane == 0) flag_error(p.err_flag, kErrBadPage);
    } else if (forced(b)) {
      key = kTaken;
    } else {
      float x[8];
      unpack8(__ldg(at), x);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s = fmaf(qf[i], x[i], s);
        most = fmaxf(most, fabsf(x[i]));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (!(fabsf(s) < INFINITY)) {
        nonfinite = 1;
        s = 0.f;
      }
      key = order32(s);
    }
    if (lane == 0) key32[b] = key;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
  if (lane == 0) atomicMax(&sh.most, __float_as_uint(most));
  if (nonfinite) sh.nonfinite = 1;
  __syncthreads();
  uint32_t nforced = 0, nfree = 0;
  for (int b = tid; b < n; b += kSelThreads) {
    nforced += key32[b] == kTaken;
    nfree += key32[b] != kTaken && key32[b] != kAbsent;
  }
  nforced = sel_sum(nforced, sh.warp_s);
  nfree = sel_sum(nfree, sh.warp_s);
  const uint32_t want = min(nfree, p.nsel > (int)nforced ? p.nsel - nforced : 0u);

  if (want == nfree) {                       // all of them
    for (int b = tid; b < n; b += kSelThreads)
      if (key32[b] != kAbsent) key32[b] = kTaken;
  } else if (want == 0) {
    for (int b = tid; b < n; b += kSelThreads)
      if (key32[b] != kTaken) key32[b] = kAbsent;
  } else {
    // ---- the want-th largest key, a digit of 8 bits at a time
    uint32_t prefix = 0, rest = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int b = tid; b < n; b += kSelThreads) {
        const uint32_t k = key32[b];
        if (k == kTaken || k == kAbsent) continue;
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&sh.hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t seen = 0;
        int d = 255;
        while (seen + sh.hist[d] < rest) seen += sh.hist[d--];
        sh.digit = d;
        sh.above = seen;
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      rest -= sh.above;
    }
    // ---- who is in, who is out, and who is too near to tell.  A float32 score
    // is off by at most e: its 14 roundings of 2^-24 each, the sums' own parts
    // among them, weigh sum |q| |bound| (twice that for good measure).  The
    // exact want-th largest is within e of the one found, so a score beyond it
    // by more than 2 e is decided.
    const float e = 0x1p-19f * sh.q1 * __uint_as_float(sh.most) + 1e-40f;
    const float at = value32(prefix);
    const bool all = sh.nonfinite || !(e < INFINITY);
    const float top = at + 2.125f * e, low = at - 2.125f * e;
    uint32_t in = 0, near = 0;
    for (int b = tid; b < n; b += kSelThreads) {
      const uint32_t k = key32[b];
      if (k == kTaken || k == kAbsent) continue;
      const float s = value32(k);
      if (all || (s >= low && s <= top))
        ++near;
      else if (s > top)
        ++in;
    }
    in = sel_sum(in, sh.warp_s);
    near = sel_sum(near, sh.warp_s);
    const uint32_t need = want - in;         // of the near ones
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if (near == need || near <= kNear) {
      for (int b = tid; b < n; b += kSelThreads) {
        const uint32_t k = key32[b];
        if (k == kTaken || k == kAbsent) continue;
        const float s = value32(k);
        if (all || (s >= low && s <= top)) {
          if (near == need) {
            key32[b] = kTaken;
          } else {
            sh.near_i[atomicAdd(&sh.count, 1u)] = b;
            key32[b] = kAbsent;
          }
        } else {
          key32[b] = s > top ? kTaken : kAbsent;
        }
      }
      __syncthreads();
      if (near != need) {
        for (uint32_t i = warp; i < near; i += kSelWarps) {
          const double s = score64(sh, __ldg(bound_ptr(p, run, g, sh.near_i[i], lane)), lane);
          if (lane == 0) sh.near_k[i] = order64(s);
        }
        __syncthreads();
        if (tid < (int)near) {
          const uint64_t k = sh.near_k[tid];
          const int b = sh.near_i[tid];
          uint32_t before = 0;
          for (uint32_t i = 0; i < near; ++i)
            before += sh.near_k[i] > k || (sh.near_k[i] == k && sh.near_i[i] < b);
          if (before < need) key32[b] = kTaken;
        }
      }
    } else {
      // ---- many near ones (equal blocks, scores that are not numbers): their
      // exact keys, and the need-th largest among them
      for (int b = warp; b < n; b += kSelWarps) {
        const uint32_t k = key32[b];
        const float s = value32(k);
        const bool is_near = k != kTaken && k != kAbsent && (all || (s >= low && s <= top));
        uint64_t x = 0;
        if (is_near) {
          x = order64(score64(sh, __ldg(bound_ptr(p, run, g, b, lane)), lane));
          if (x == 0) x = 1;                 // 0 marks a block that is not near
        }
        __syncwarp();
        if (lane == 0) {
          key64[b] = x;
          if (!is_near) key32[b] = k == kTaken || (k != kAbsent && s > top) ? kTaken : kAbsent;
        }
      }
      __syncthreads();
      uint64_t prefix64 = 0;
      uint32_t left = need;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int b = tid; b < n; b += kSelThreads) {
          const uint64_t k = key64[b];
          if (k && (shift == 56 || (k >> (shift + 8)) == (prefix64 >> (shift + 8))))
            atomicAdd(&sh.hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
          uint32_t seen = 0;
          int d = 255;
          while (seen + sh.hist[d] < left) seen += sh.hist[d--];
          sh.digit = d;
          sh.above = seen;
        }
        __syncthreads();
        prefix64 |= (uint64_t)sh.digit << shift;
        left -= sh.above;
      }
      // those above the need-th, and of the ones equal to it the first `left`
      uint32_t seen = 0;
      for (int b0 = 0; b0 < n; b0 += kSelThreads) {
        const int b = b0 + tid;
        const uint64_t k = b < n ? key64[b] : 0;
        uint32_t total;
        const uint32_t before = seen + sel_prefix(k == prefix64, sh.warp_s, total);
        if (k) key32[b] = k > prefix64 || (k == prefix64 && before < left) ? kTaken : kAbsent;
        seen += total;
      }
    }
  }
  __syncthreads();
  // ---- the chosen blocks, ascending
  uint32_t filled = 0;
  for (int b0 = 0; b0 < n; b0 += kSelThreads) {
    const int b = b0 + tid;
    const bool in = b < n && key32[b] == kTaken;
    uint32_t total;
    const uint32_t before = filled + sel_prefix(in, sh.warp_s, total);
    if (in) out[before] = b;
    filled += total;
  }
  for (uint32_t i = filled + tid; i < (uint32_t)p.nsel; i += kSelThreads) out[i] = -1;
}

}  // namespace

cudaError_t launch_key_bounds(const BoundsParams& p, int kv, cudaStream_t s) {
  const dim3 grid(p.items * p.hkv), block(kBoundThreads);
  switch (kv) {
    case kKvBf16: return launch_pdl(key_bounds_kernel<kKvBf16>, grid, block, 0, s, p);
    case kKvFp8: return launch_pdl(key_bounds_kernel<kKvFp8>, grid, block, 0, s, p);
    default: return launch_pdl(key_bounds_kernel<kKvFp4>, grid, block, 0, s, p);
  }
}

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s) {
  static PerDeviceOnce configured;
  const cudaError_t e = configured.run([] {
    return cudaFuncSetAttribute(select_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSelectBlocks * 12);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(select_blocks_kernel, dim3(p.rows * p.hkv), dim3(kSelThreads),
                    (size_t)p.cap * 12, s, p);
}

}  // namespace tfpa
