// Accumulated attention weight of the cached keys: for every segment with
// rows in the call, kv head g and key j
//   mass[s][g][j] = decay mass[s][g][j]
//                   + sum over rows r at or after j, heads h of g, of
//                     2^(q_rh . k_j scale log2(e) - lse[r][h] log2(e)),
// the weights that the rows' attention (which left lse) gave the key.  K is
// read once and V not at all.
//
// Keys are the rows of the products and query vectors their columns:
//   D [128 keys][N vectors] = K Q^T (tcgen05, one MMA chain a key tile),
// so that a key is a TMEM lane and its weights one thread's columns: the
// thread sums them in a fixed order and owns the key's entry; no shuffles, no
// atomics.  Persistent CTAs, each an equal run of the call's key tiles
// (segment, kv head, 128 keys), so mostly of one (segment, kv head), whose
// query vectors it stages once as the B operand (up to 256; more go in
// passes over the same keys).
//   warp 0       producer: key tiles into a ring, by TMA (bf16: the operand
//                itself; e4m3: staging) or bulk copies (4 bits: staging)
//   warp 1       TMEM owner and MMA issuer, two or four D buffers
//   warps 4-11   epilogue: two groups of four, tiles in turn
//   warps 12-19  (e4m3, 4 bits) converters: staged tiles -> f16 operand tiles,
//                two groups of four, tiles in turn
// e4m3 and 4-bit keys are exact in f16; a pass's query vectors are scaled into
// f16 range by one power of two (exact for every element within 2^30 of the
// pass's largest), so that all of its scores have one factor and a column's
// only constant is its -lse.  Those constants come from shared memory, and a
// read that gives all lanes one value costs as much of its bandwidth as one
// that gives each its own: the epilogue takes two key tiles at a time, each
// constant read once for both.
// Measured: one row of 8 streams of 8,192 bf16 keys 26.8 us a call, 22 of them in
// the kernel, whose bytes need 20.4 (HBM); 32 rows of 4 streams of 32,001 to
// 65,001 4-bit keys, 128 vectors a kv head, 69 us (the epilogue: an exponential,
// a multiply-add and an add a score, and its waits for D buffers; the products
// alone need 26).
#include <climits>

#include "common.cuh"
#include "convert.cuh"
#include "params.h"
#include "tcgen05.cuh"

namespace tfpa {
namespace {

constexpr int kTile = 128;               // keys of a tile
constexpr int kVec = 256;                // query vectors of a pass, at most
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kConvWarp0 = 12, kConvWarps = 8;
template <int KV>
struct MassCfg {
  static constexpr bool kF16 = KV != kKvBf16;
  static constexpr int kThreads = kF16 ? 640 : 384;
  static constexpr int kStageBytes =
      KV == kKvBf16 ? 32768 : KV == kKvFp8 ? 16384 : kFp4HalfBytes;
  // An even number: the converter groups take tiles in turn, and a stage has to
  // be the same group's every time (a barrier's parity only tells phases apart
  // for those who wait for every one of them).
  static constexpr int kStages = KV == kKvFp4 ? 8 : 4;
  static_assert(kStages % 2 == 0, "a stage belongs to one converter group");
  static constexpr int kOps = kF16 ? 2 : 0;              // f16 operand tiles
  static constexpr int kOffQ = 0;                        // 64 KB
  static constexpr int kOffOp = 65536;
  static constexpr int kOffStage = kOffOp + kOps * 32768;
  static constexpr int kOffTab = (kOffStage + kStages * kStageBytes + 1023) & ~1023;
  static constexpr int kOffLim = kOffTab + kVec * 4;
  static constexpr int kOffBar = kOffLim + kVec * 4;
  static constexpr int kBars = 2 * kStages + 2 * 2 + 2 * 4 + 1;
  static constexpr int kSmem = kOffBar + kBars * 8 + 64 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct MassBars {
  uint64_t *full, *empty;        // [kStages]: the ring
  uint64_t *op_full, *op_empty;  // [2]: f16 operand tiles
  uint64_t *d_full, *d_empty;    // [4]: D buffers
  uint64_t* drain;
  uint32_t* tmem_slot;
  volatile int* abort;
  int* amax;                     // [2], by pass parity: largest |q| of the pass (its bits)
  int* stop;                     // [2], by pass parity: a wait has given up
  int* none;                     // [2], by pass parity: a row of the pass saw no key
};

// Vector v of segment sg: its run and row.
__device__ __forceinline__ void find_vector(const MassParams& p, const MassSeg& sg, int v,
                                            int& row, int& pos, int& head) {
  int r = sg.run0;
  while (v >= p.runs[r].nrows * p.group) v -= p.runs[r++].nrows * p.group;
  const int k = v / p.group;
  row = p.runs[r].row0 + k;
  pos = p.runs[r].pos0 + k;
  head = v - k * p.group;
}

// Least and largest position of the rows of vectors [v0, v0 + nv).
__device__ __forceinline__ void pass_span(const MassParams& p, const MassSeg& sg, int v0, int nv,
                                          int& lo, int& hi) {
  lo = INT_MAX;
  hi = -1;
  int at = 0;                            // first vector of run r
  for (int r = sg.run0; r < sg.run0 + sg.nruns; ++r) {
    const int n = p.runs[r].nrows * p.group;
    const int a = max(v0, at) - at, z = min(v0 + nv, at + n) - at;
    if (a < z) {
      lo = min(lo, p.runs[r].pos0 + a / p.group);
      hi = max(hi, p.runs[r].pos0 + (z - 1) / p.group);
    }
    at += n;
  }
}

// Query vectors [v0, v0 + nv) as the B operand ([n rows][2 halves of 64],
// 128B swizzle) with each one's -lse and position; all warps but the
// producer's, 16 threads a vector.  Rows from nv on repeat the first vector
// with -lse = -inf: a weight of 0 by any key that gives the first one a finite
// weight or 0, an infinite key among them, where zeros would give a NaN.  A row
// that saw no key (lse -inf) becomes zeros, whatever its q holds, and *none_s
// says that there is one.  Returns the scores' factor.
template <int KV>
__device__ float stage_q(const MassParams& p, const MassSeg& sg, int g, int v0, int nv, int n,
                         uint8_t* smem, int* amax_s, int* none_s) {
  using C = MassCfg<KV>;
  constexpr int kStep = (C::kThreads - 32) / 16;
  const uint32_t qb = smem_u32(smem + C::kOffQ);
  float* negs = reinterpret_cast<float*>(smem + C::kOffTab);
  int* lims = reinterpret_cast<int*>(smem + C::kOffLim);
  const int t = threadIdx.x & 15, i0 = (threadIdx.x - 32) >> 4;
  // A thread's vectors i0, i0 + kStep, ...: all of a batch's loads at once.
  constexpr int kMost = (kVec + kStep - 1) / kStep, kBatch = C::kF16 ? kMost : 4;
  uint4 w[kBatch];
  int lim[kBatch];
  float neg[kBatch];
  auto load_batch = [&](int i) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u, i += kStep) {
      w[u] = make_uint4(0, 0, 0, 0);
      lim[u] = -1;
      neg[u] = INFINITY;
      if (i >= n) continue;
      int row, head, pos;
      find_vector(p, sg, i < nv ? v0 + i : v0, row, pos, head);
      const size_t rh = (size_t)row * p.hq + g * p.group + head;
      w[u] = __ldg(reinterpret_cast<const uint4*>(p.q + rh * kHeadDim) + t);
      neg[u] = __ldg(p.lse + rh);
      if (i < nv) lim[u] = pos;
    }
    // all loads are on their way by now
    i -= kBatch * kStep;
#pragma unroll
    for (int u = 0; u < kBatch; ++u, i += kStep) {
      if (neg[u] == -INFINITY) {
        w[u] = make_uint4(0, 0, 0, 0);
        lim[u] = -1;
        *none_s = 1;
      }
      if (t == 0 && i < n) {
        negs[i] = lim[u] < 0 ? -INFINITY : -neg[u] * 1.4426950408889634f;
        lims[i] = lim[u];
      }
    }
  };
  float up = 1.f, sc = p.scale_log2;
  if (C::kF16) {
    // the pass's largest magnitude goes to [2^13, 2^14)
    load_batch(i0);
    // The largest of the batch's magnitudes up to `top` (a NaN is none), over
    // all threads, in *amax_s.
    auto largest = [&](float top) {
      float amax = 0.f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t e[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = fabsf(__uint_as_float(e[j] << 16));
          const float hi = fabsf(__uint_as_float(e[j] & 0xFFFF0000u));
          amax = fmaxf(amax, top == INFINITY || lo <= top ? lo : 0.f);
          amax = fmaxf(amax, top == INFINITY || hi <= top ? hi : 0.f);
        }
      }
      __syncwarp();
      const int most = __reduce_max_sync(0xffffffffu, __float_as_int(amax));   // not negative
      if ((threadIdx.x & 31) == 0) atomicMax(amax_s, most);
      __syncwarp();
      named_bar_sync(2, C::kThreads - 32);
      return __int_as_float(*amax_s);
    };
    float amax = largest(INFINITY);
    if (amax == INFINITY) {
      // an infinity stays one in f16 and sets no other row's scale: the
      // largest finite magnitude instead, in the same word
      named_bar_sync(2, C::kThreads - 32);
      if (threadIdx.x == 32) *amax_s = 0;
      __syncwarp();
      named_bar_sync(2, C::kThreads - 32);
      amax = largest(__uint_as_float(0x7F7F0000u));     // bf16's largest number
    }
    int ex;
    frexpf(amax, &ex);
    ex = max(min(ex, 120), -100);
    up = __int_as_float((127 + 14 - ex) << 23);
    sc = p.scale_log2 * __int_as_float((127 - 14 + ex) << 23) * __ldg(p.k_scale + g);
  }
  for (int ib = i0; ib < n; ib += kBatch * kStep) {
    if (!C::kF16) load_batch(ib);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = ib + u * kStep;
      if (i >= n) break;
      uint32_t e[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      if (C::kF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          e[j] = pack_f16x2(__uint_as_float(e[j] << 16) * up,
                            __uint_as_float(e[j] & 0xFFFF0000u) * up);
      }
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                       swz128(qb + (uint32_t)(t >> 3) * (uint32_t)n * 128u, i, t & 7)),
                   "r"(e[0]), "r"(e[1]), "r"(e[2]), "r"(e[3]) : "memory");
    }
  }
  fence_proxy_async_smem();
  return sc;
}

// Adds the weights of columns [0, n) (n a multiple of 16) of one or two D
// tiles, of the keys key0 and key1; the D buffers are handed back (empty) as
// soon as their last columns are in registers.
template <bool TWO, bool MASKED>
__device__ __forceinline__ void add_columns(uint32_t d0, uint32_t d1, int n, const float* negs,
                                            const int* lims, float sc, int key0, int key1,
                                            uint64_t* empty, float& sum0, float& sum1) {
  float a[2][4] = {};
  for (int c0 = 0; c0 < n; c0 += 16) {
    uint32_t v[2][16];
    umma::tmem_ld16(d0 + c0, v[0]);
    if (TWO) umma::tmem_ld16(d1 + c0, v[1]);
    float4 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float4*>(negs + c0 + 4 * j);
    umma::tmem_ld_wait();
    if (c0 + 16 == n) {
      umma::fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive(empty);
        if (TWO) mbar_arrive(empty + 1);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float neg = j % 4 == 0 ? f[j / 4].x : j % 4 == 1 ? f[j / 4].y
                        : j % 4 == 2 ? f[j / 4].z : f[j / 4].w;
      const int lim = MASKED ? lims[c0 + j] : 0;
#pragma unroll
      for (int u = 0; u < (TWO ? 2 : 1); ++u) {
        const float w = fast_exp2(__fmaf_rn(__uint_as_float(v[u][j]), sc, neg));
        a[u][j & 3] += !MASKED || (u ? key1 : key0) <= lim ? w : 0.f;
      }
    }
  }
  sum0 = (a[0][0] + a[0][1]) + (a[0][2] + a[0][3]);
  if (TWO) sum1 = (a[1][0] + a[1][1]) + (a[1][2] + a[1][3]);
}

// Keeps a value in its register (not read again from where it came).
__device__ __forceinline__ void hold(int& x) { asm volatile("" : "+r"(x)); }
__device__ __forceinline__ void hold(float& x) { asm volatile("" : "+f"(x)); }
template <typename T>
__device__ __forceinline__ void hold(T*& x) { asm volatile("" : "+l"(x)); }

template <int KV>
__global__ void __launch_bounds__(MassCfg<KV>::kThreads, 1)
    key_mass_kernel(const __grid_constant__ MassParams p) {
  using C = MassCfg<KV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  MassBars b;
  b.full = bars;
  b.empty = bars + C::kStages;
  b.op_full = bars + 2 * C::kStages;
  b.op_empty = b.op_full + 2;
  b.d_full = b.op_full + 4;
  b.d_empty = b.op_full + 8;
  b.drain = b.op_full + 12;
  b.tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  b.abort = reinterpret_cast<volatile int*>(b.tmem_slot + 1);
  b.amax = reinterpret_cast<int*>(b.tmem_slot + 2);
  b.stop = b.amax + 2;
  b.none = b.stop + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], C::kF16 ? kConvWarps / 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.op_full[i], kConvWarps / 2);
      mbar_init(&b.op_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.d_full[i], 1);
      mbar_init(&b.d_empty[i], kEpiWarps / 2);
    }
    mbar_init(b.drain, 1);
    *b.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) umma::tmem_alloc(b.tmem_slot, 512);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *b.tmem_slot;
  allow_next_grid();
  wait_prior_grid();

  const int t0 = (int)((int64_t)p.tiles * blockIdx.x / gridDim.x);
  const int t1 = (int)((int64_t)p.tiles * (blockIdx.x + 1) / gridDim.x);
  const float* negs = reinterpret_cast<const float*>(smem + C::kOffTab);
  const int* lims = reinterpret_cast<const int*>(smem + C::kOffLim);
  // D buffers: four of 128 columns where the launch's passes are that narrow,
  // so that the epilogue can take two tiles at a time, else two of 256
  const int nb = p.dbufs, lnb = nb == 4 ? 2 : 1, dcols = 512 >> lnb;
  uint32_t cnt = 0;                      // tiles multiplied so far (every role's count)
  int si = 0, pass = 0;
  for (int t = t0; t < t1;) {
    while (si + 1 < p.nsegs && p.segs[si + 1].item0 <= t) ++si;
    const MassSeg& sg = p.segs[si];
    const int tiles = (sg.seq_len + kTile - 1) / kTile;
    const int local = t - sg.item0;
    const int g = local / tiles, kt0 = local - g * tiles;
    const int nt = min(t1 - t, tiles - kt0);
    int total = 0;                       // the segment's query vectors
    for (int r = sg.run0; r < sg.run0 + sg.nruns; ++r) total += p.runs[r].nrows * p.group;
    for (int v0 = 0; v0 < total; v0 += kVec, ++pass) {
      const int nv = min(kVec, total - v0);
      const int n = (nv + 15) & ~15;     // the MMA's N
      int minlim, maxlim;
      pass_span(p, sg, v0, nv, minlim, maxlim);
      // tiles past the last row's position get no weight
      const int mt = max(0, min(nt, maxlim / kTile + 1 - kt0));
      // the producer runs ahead of the passes; the others stage each one's
      // vectors once all of them are done with the last
      float sc = 0.f;
      if (warp != 0) {
        // one thread's look at the flag decides for all (the other parity's
        // words may still be read)
        if (threadIdx.x == 32) {
          b.amax[pass & 1] = 0;
          b.none[pass & 1] = 0;
          b.stop[pass & 1] = *b.abort;
        }
        __syncwarp();
        named_bar_sync(2, C::kThreads - 32);
        if (b.stop[pass & 1]) goto out;
        sc = stage_q<KV>(p, sg, g, v0, nv, n, smem, b.amax + (pass & 1), b.none + (pass & 1));
        __syncwarp();
        named_bar_sync(2, C::kThreads - 32);
        // a row that saw no key: every tile's limits are looked at, as a key
        // that is not finite has no finite product with its zeros
        if (b.none[pass & 1]) minlim = -1;
      }
      if (warp == 0) {
        bool ok = true;
        if (lane == 0) {
          int page_at = -1, pid = 0;
          const int32_t* table = sg.page_table;
          const void* base = sg.k_base;
          int slab_cap = sg.slab_cap, src = sg.src;
          hold(table);
          hold(base);
          hold(slab_cap);
          hold(src);
          for (int i = 0; i < mt; ++i) {
            const int key0 = (kt0 + i) * kTile;
            int row;
            if (table) {
              const int page = key0 >> 8;
              if (page != page_at) {
                page_at = page;
                pid = __ldg(table + page);
                if ((unsigned)pid >= (unsigned)p.num_pages) {
                  flag_error(p.err_flag, kErrBadPage);
                  pid = 0;
                }
              }
              row = (pid * p.hkv + g) * kPage + (key0 & (kPage - 1));
            } else {
              row = g * slab_cap + key0;
            }
            const uint32_t st = cnt + i;
            const int s = st % C::kStages;
            ok = mbar_wait_or_abort(&b.empty[s], ((st / C::kStages) & 1) ^ 1, p.err_flag, b.abort);
            if (!ok) break;
            uint8_t* dst = smem + C::kOffStage + s * C::kStageBytes;
            mbar_arrive_expect_tx(&b.full[s], C::kStageBytes);
            if (KV == kKvBf16) {
              tma_load_2d(dst, &p.maps[src], 0, row, &b.full[s]);
              tma_load_2d(dst + 16384, &p.maps[src], 64, row, &b.full[s]);
            } else if (KV == kKvFp8) {
              tma_load_2d(dst, &p.maps[src], 0, row, &b.full[s]);
            } else {
              bulk_load(dst, static_cast<const uint8_t*>(base) +
                                 (size_t)(row / kHalfRows) * kFp4HalfBytes,
                        kFp4HalfBytes, &b.full[s]);
            }
          }
        }
        // the warp leaves with lane 0: alone, it would wait in the block's
        // last barrier for lanes that wait for it here
        if (!__shfl_sync(0xffffffffu, ok, 0)) goto out;
      } else if (warp == 1) {
        const uint32_t idesc = umma::idesc_f16(128, 16, !C::kF16, false) + ((uint32_t)(n - 16) >> 3 << 17);
        const uint32_t qb = smem_u32(smem + C::kOffQ);
        if (umma::elect_one()) {
          for (int i = 0; i < mt; ++i) {
            const uint32_t st = cnt + i;
            const int s = C::kF16 ? st & 1 : st % C::kStages;
            uint64_t* ready = C::kF16 ? &b.op_full[s] : &b.full[s];
            const uint32_t ph = C::kF16 ? (st >> 1) & 1 : (st / C::kStages) & 1;
            const int d = st & (nb - 1);
            if (!mbar_wait_or_abort(ready, ph, p.err_flag, b.abort) ||
                !mbar_wait_or_abort(&b.d_empty[d], ((st >> lnb) & 1) ^ 1, p.err_flag, b.abort))
              break;
            umma::fence_after_sync();
            const uint32_t kb =
                smem_u32(smem + (C::kF16 ? C::kOffOp + s * 32768 : C::kOffStage + s * 32768));
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t ad =
                  umma::smem_desc_sw128(kb + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
              const uint64_t bd = umma::smem_desc_sw128(
                  qb + (ks >> 2) * (uint32_t)n * 128u + (ks & 3) * 32, 16, 1024);
              umma::mma_ss(tmem + d * dcols, ad, bd, idesc, ks > 0 ? 1u : 0u);
            }
            umma::commit(C::kF16 ? &b.op_empty[s] : &b.empty[s]);
            umma::commit(&b.d_full[d]);
          }
        }
        __syncwarp();
      } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
        const int grp = (warp - kEpiWarp0) >> 2;
        float decay = v0 == 0 ? sg.decay : 1.f;
        hold(decay);
        float* plane = p.mass + (size_t)(sg.index * p.hkv + g) * p.mass_cap;
        hold(plane);
        const uint32_t tq = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int lane_key = 32 * (warp & 3) + lane;
        // A tile's entry of this lane, loaded before the tile's scores are waited
        // for (decay 0 reads none), and whether it is written (a bad page's is
        // not).  What a step needs of the segment is held in registers: an
        // indexed read of the launch's parameters costs hundreds of cycles.
        const int32_t* table = sg.page_table;
        int seq_len = sg.seq_len;
        hold(table);
        hold(seq_len);
        auto old_of = [&](int i) {
          const int key = (kt0 + i) * kTile + lane_key;
          return decay != 0.f && key < seq_len ? plane[key] : 0.f;
        };
        auto live_of = [&](int i) {
          const int key = (kt0 + i) * kTile + lane_key;
          if (key >= seq_len) return false;
          if (table && (unsigned)__ldg(table + (key >> 8)) >= (unsigned)p.num_pages) {
            flag_error(p.err_flag, kErrBadPage);
            return false;
          }
          return true;
        };
        // Tiles that are multiplied: D buffers 0, 1 go to one group and 2, 3
        // to the other, two tiles at a time (two buffers: one each).
        const uint32_t end = cnt + mt, width = nb >> 1;
        for (uint32_t at = (cnt & ~(uint32_t)(nb - 1)) + width * grp; at < end; at += nb) {
          const uint32_t st = max(at, cnt), stop = min(at + width, end);
          if (st >= stop) continue;
          const int i = st - cnt;
          const bool two = stop - st == 2;
          const float old0 = old_of(i), old1 = two ? old_of(i + 1) : 0.f;
          const int d = st & (nb - 1);
          const int key = (kt0 + i) * kTile + lane_key;
          if (!warp_wait_or_abort(&b.d_full[d], (st >> lnb) & 1, p.err_flag, b.abort)) break;
          if (two && !warp_wait_or_abort(&b.d_full[d + 1], (st >> lnb) & 1, p.err_flag, b.abort))
            break;
          umma::fence_after_sync();
          float s0 = 0.f, s1 = 0.f;
          const uint32_t td = tq + d * dcols;
          const bool masked = (kt0 + i + (two ? 2 : 1)) * kTile - 1 > minlim;
          if (two && masked)
            add_columns<true, true>(td, td + dcols, n, negs, lims, sc, key, key + kTile, &b.d_empty[d], s0, s1);
          else if (two)
            add_columns<true, false>(td, td + dcols, n, negs, lims, sc, key, key + kTile, &b.d_empty[d], s0, s1);
          else if (masked)
            add_columns<false, true>(td, td, n, negs, lims, sc, key, key, &b.d_empty[d], s0, s1);
          else
            add_columns<false, false>(td, td, n, negs, lims, sc, key, key, &b.d_empty[d], s0, s1);
          if (live_of(i)) plane[key] = __fmaf_rn(old0, decay, s0);
          if (two && live_of(i + 1)) plane[key + kTile] = __fmaf_rn(old1, decay, s1);
        }
        // the others only decay
        for (int i = mt; decay != 1.f && i < nt; ++i) {
          if ((i & 1) != grp) continue;
          const float old = old_of(i);
          if (live_of(i)) plane[(kt0 + i) * kTile + lane_key] = old * decay;
        }
      } else if (C::kF16 && warp >= kConvWarp0) {
        constexpr int kGroup = 16 * kConvWarps;          // threads of a group
        const int o = (warp - kConvWarp0) / (kConvWarps / 2);   // its tiles' parity and operand
        const int ct = (threadIdx.x - kConvWarp0 * 32) % kGroup;
        for (int i = (cnt & 1) ^ o; i < mt; i += 2) {
          const uint32_t st = cnt + i;
          const int s = st % C::kStages;
          if (!warp_wait_or_abort(&b.full[s], (st / C::kStages) & 1, p.err_flag, b.abort) ||
              !warp_wait_or_abort(&b.op_empty[o], ((st >> 1) & 1) ^ 1, p.err_flag, b.abort))
            break;
          const uint8_t* src = smem + C::kOffStage + s * C::kStageBytes;
          uint8_t* dst = smem + C::kOffOp + o * 32768;
          if (KV == kKvFp4)
            convert_tile_fp4<kGroup, 1>(src, dst, kTile, ct);
          else
            convert_tile<kGroup>(src, dst, kTile, ct);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&b.empty[s]);
            mbar_arrive(&b.op_full[o]);
          }
        }
      }
      cnt += mt;
    }
    t += nt;
  }
out:
  __syncwarp();
  if (warp == 1) {
    // every MMA and every arrival asked of them has happened
    if (umma::elect_one()) {
      umma::commit(b.drain);
      mbar_wait(b.drain, 0, p.err_flag);
    }
    __syncwarp();
  }
  umma::fence_before_sync();
  __syncthreads();
  if (*b.abort) let_copies_land();
  if (warp == 1) {
    umma::fence_after_sync();
    umma::tmem_dealloc(tmem, 512);
  }
}

template <int KV>
cudaError_t launch(const MassParams& p, int grid, cudaStream_t s) {
  static PerDeviceOnce configured;
  const cudaError_t e = configured.run([] {
    return cudaFuncSetAttribute(key_mass_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MassCfg<KV>::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(key_mass_kernel<KV>, dim3(grid), dim3(MassCfg<KV>::kThreads),
                    MassCfg<KV>::kSmem, s, p);
}

}  // namespace

cudaError_t launch_key_mass(const MassParams& p, int kv, int grid, cudaStream_t s) {
  if (grid <= 0) return cudaSuccess;
  switch (kv) {
    case kKvBf16: return launch<kKvBf16>(p, grid, s);
    case kKvFp8: return launch<kKvFp8>(p, grid, s);
    default: return launch<kKvFp4>(p, grid, s);
  }
}

}  // namespace tfpa
