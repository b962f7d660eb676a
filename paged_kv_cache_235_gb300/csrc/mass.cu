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
//   warp 1       TMEM owner and MMA issuer, two D buffers
//   warps 4-11   epilogue: two groups of four, tiles in turn
//   warps 12-19  (e4m3, 4 bits) converters: staged tiles -> f16 operand tiles
// e4m3 and 4-bit keys are exact in f16; their query vectors are scaled into
// f16 range by a power of two each.
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
  static constexpr int kStages = KV == kKvBf16 ? 4 : KV == kKvFp8 ? 5 : 9;
  static constexpr int kOps = kF16 ? 2 : 0;              // f16 operand tiles
  static constexpr int kOffQ = 0;                        // 64 KB
  static constexpr int kOffOp = 65536;
  static constexpr int kOffStage = kOffOp + kOps * 32768;
  static constexpr int kOffTab = (kOffStage + kStages * kStageBytes + 1023) & ~1023;
  static constexpr int kOffLim = kOffTab + kVec * 8;
  static constexpr int kOffBar = kOffLim + kVec * 4;
  static constexpr int kBars = 2 * kStages + 2 * 2 + 2 * 2 + 1;
  static constexpr int kSmem = kOffBar + kBars * 8 + 32 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct MassBars {
  uint64_t *full, *empty;        // [kStages]: the ring
  uint64_t *op_full, *op_empty;  // [2]: f16 operand tiles
  uint64_t *d_full, *d_empty;    // [2]: D buffers
  uint64_t* drain;
  uint32_t* tmem_slot;
  volatile int* abort;
  int* span;                     // [2][2], by pass parity: its rows' least, largest position
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

// Query vectors [v0, v0 + nv) as the B operand ([n rows][2 halves of 64],
// 128B swizzle; rows from nv on zero) with each one's score factor, -lse and
// position; all threads, 16 a vector.
template <int KV>
__device__ void stage_q(const MassParams& p, const MassSeg& sg, int g, int v0, int nv, int n,
                        uint8_t* smem, int* span) {
  using C = MassCfg<KV>;
  const uint32_t qb = smem_u32(smem + C::kOffQ);
  float2* tab = reinterpret_cast<float2*>(smem + C::kOffTab);
  int* lims = reinterpret_cast<int*>(smem + C::kOffLim);
  const int t = threadIdx.x & 15;
  for (int i = threadIdx.x >> 4; i < n; i += C::kThreads / 16) {
    uint4 w = make_uint4(0, 0, 0, 0);
    int lim = -1;
    float sc = 0.f, neg = -INFINITY;
    if (i < nv) {
      int row, head;
      find_vector(p, sg, v0 + i, row, lim, head);
      const size_t rh = (size_t)row * p.hq + g * p.group + head;
      w = __ldg(reinterpret_cast<const uint4*>(p.q + rh * kHeadDim) + t);
      sc = p.scale_log2;
      // a row without keys has lse -inf and gives no weight
      const float lse = __ldg(p.lse + rh);
      neg = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
    }
    if (C::kF16) {
      // f16, the vector's largest magnitude brought into [2^13, 2^14):
      // exact for every element within 2^28 of it
      uint32_t e[4] = {w.x, w.y, w.z, w.w};
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        amax = fmaxf(amax, fabsf(__uint_as_float(e[j] << 16)));
        amax = fmaxf(amax, fabsf(__uint_as_float(e[j] & 0xFFFF0000u)));
      }
      const unsigned lanes = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
      int ex;
      frexpf(amax, &ex);
      ex = max(min(ex, 120), -100);
      const float up = __int_as_float((127 + 14 - ex) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        e[j] = pack_f16x2(__uint_as_float(e[j] << 16) * up,
                          __uint_as_float(e[j] & 0xFFFF0000u) * up);
      w = make_uint4(e[0], e[1], e[2], e[3]);
      sc *= __int_as_float((127 - 14 + ex) << 23) * __ldg(p.k_scale + g);
    }
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                     swz128(qb + (uint32_t)(t >> 3) * (uint32_t)n * 128u, i, t & 7)),
                 "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
    if (t == 0) {
      tab[i] = make_float2(sc, neg);
      lims[i] = lim;
      if (i < nv) {
        atomicMin(&span[0], lim);
        atomicMax(&span[1], lim);
      }
    }
  }
  fence_proxy_async_smem();
}

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
  b.d_empty = b.op_full + 6;
  b.drain = b.op_full + 8;
  b.tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  b.abort = reinterpret_cast<volatile int*>(b.tmem_slot + 1);
  b.span = reinterpret_cast<int*>(b.tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], C::kF16 ? kConvWarps : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.op_full[i], kConvWarps);
      mbar_init(&b.op_empty[i], 1);
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
  const float2* tab = reinterpret_cast<const float2*>(smem + C::kOffTab);
  const int* lims = reinterpret_cast<const int*>(smem + C::kOffLim);
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
      int* span = b.span + 2 * (pass & 1);   // the other one may still be read
      if (threadIdx.x == 0) {
        span[0] = INT_MAX;
        span[1] = -1;
      }
      __syncthreads();                   // every role is done with the pass before
      if (*b.abort) goto out;
      stage_q<KV>(p, sg, g, v0, nv, n, smem, span);
      __syncthreads();
      const int minlim = span[0], maxlim = span[1];
      // tiles past the last row's position get no weight
      const int mt = max(0, min(nt, maxlim / kTile + 1 - kt0));
      if (warp == 0) {
        if (lane == 0) {
          int page_at = -1, pid = 0;
          for (int i = 0; i < mt; ++i) {
            const int key0 = (kt0 + i) * kTile;
            int row;
            if (sg.page_table) {
              const int page = key0 >> 8;
              if (page != page_at) {
                page_at = page;
                pid = __ldg(sg.page_table + page);
                if ((unsigned)pid >= (unsigned)p.num_pages) {
                  flag_error(p.err_flag, kErrBadPage);
                  pid = 0;
                }
              }
              row = (pid * p.hkv + g) * kPage + (key0 & (kPage - 1));
            } else {
              row = g * sg.slab_cap + key0;
            }
            const uint32_t st = cnt + i;
            const int s = st % C::kStages;
            if (!mbar_wait_or_abort(&b.empty[s], ((st / C::kStages) & 1) ^ 1, p.err_flag, b.abort))
              break;
            uint8_t* dst = smem + C::kOffStage + s * C::kStageBytes;
            mbar_arrive_expect_tx(&b.full[s], C::kStageBytes);
            if (KV == kKvBf16) {
              tma_load_2d(dst, &p.maps[sg.src], 0, row, &b.full[s]);
              tma_load_2d(dst + 16384, &p.maps[sg.src], 64, row, &b.full[s]);
            } else if (KV == kKvFp8) {
              tma_load_2d(dst, &p.maps[sg.src], 0, row, &b.full[s]);
            } else {
              bulk_load(dst, static_cast<const uint8_t*>(sg.k_base) +
                                 (size_t)(row / kHalfRows) * kFp4HalfBytes,
                        kFp4HalfBytes, &b.full[s]);
            }
          }
        }
        __syncwarp();
      } else if (warp == 1) {
        const uint32_t idesc = umma::idesc_f16(128, 16, !C::kF16, false) + ((uint32_t)(n - 16) >> 3 << 17);
        const uint32_t qb = smem_u32(smem + C::kOffQ);
        for (int i = 0; i < mt; ++i) {
          const uint32_t st = cnt + i;
          const int s = C::kF16 ? st & 1 : st % C::kStages;
          uint64_t* ready = C::kF16 ? &b.op_full[s] : &b.full[s];
          const uint32_t ph = C::kF16 ? (st >> 1) & 1 : (st / C::kStages) & 1;
          const int d = st & 1;
          if (!mbar_wait_or_abort(ready, ph, p.err_flag, b.abort)) break;
          if (!mbar_wait_or_abort(&b.d_empty[d], ((st >> 1) & 1) ^ 1, p.err_flag, b.abort)) break;
          __syncwarp();
          umma::fence_after_sync();
          if (lane == 0) {
            const uint32_t kb =
                smem_u32(smem + (C::kF16 ? C::kOffOp + s * 32768 : C::kOffStage + s * 32768));
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t ad =
                  umma::smem_desc_sw128(kb + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
              const uint64_t bd = umma::smem_desc_sw128(
                  qb + (ks >> 2) * (uint32_t)n * 128u + (ks & 3) * 32, 16, 1024);
              umma::mma_ss(tmem + d * 256, ad, bd, idesc, ks > 0 ? 1u : 0u);
            }
            umma::commit(C::kF16 ? &b.op_empty[s] : &b.empty[s]);
            umma::commit(&b.d_full[d]);
          }
          __syncwarp();
        }
      } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
        const int grp = (warp - kEpiWarp0) >> 2;
        const float decay = v0 == 0 ? sg.decay : 1.f;
        float* plane = p.mass + (size_t)(sg.index * p.hkv + g) * p.mass_cap;
        const uint32_t td = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + grp * 256;
        for (int i = 0; i < nt; ++i) {
          const uint32_t st = cnt + i;
          // tiles that are multiplied go to the group whose D buffer they
          // take; the others only decay
          if ((int)(st & 1) != grp) continue;
          const int key = (kt0 + i) * kTile + 32 * (warp & 3) + lane;
          bool live = key < sg.seq_len;
          if (live && sg.page_table) {
            // a bad page's keys keep their entries
            const int pid = __ldg(sg.page_table + (key >> 8));
            if ((unsigned)pid >= (unsigned)p.num_pages) {
              flag_error(p.err_flag, kErrBadPage);
              live = false;
            }
          }
          // decay 0 does not read the old entry
          const float old = live && decay != 0.f ? plane[key] * decay : 0.f;
          float sum = 0.f;
          if (i < mt) {
            if (!__all_sync(0xffffffffu, mbar_wait_or_abort(&b.d_full[grp], (st >> 1) & 1,
                                                             p.err_flag, b.abort)))
              break;
            umma::fence_after_sync();
            const bool masked = (kt0 + i + 1) * kTile - 1 > minlim;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c0 = 0; c0 < n; c0 += 16) {
              uint32_t v[16];
              umma::tmem_ld16(td + c0, v);
              umma::tmem_ld_wait();
              if (masked) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 f = tab[c0 + j];
                  const float w = fast_exp2(__fmaf_rn(__uint_as_float(v[j]), f.x, f.y));
                  acc[j & 3] += key <= lims[c0 + j] ? w : 0.f;
                }
              } else {
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  const float4 f = *reinterpret_cast<const float4*>(tab + c0 + j);
                  acc[j & 3] += fast_exp2(__fmaf_rn(__uint_as_float(v[j]), f.x, f.y));
                  acc[(j + 1) & 3] += fast_exp2(__fmaf_rn(__uint_as_float(v[j + 1]), f.z, f.w));
                }
              }
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.d_empty[grp]);
            sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
          }
          if (live && (i < mt || decay != 1.f)) plane[key] = old + sum;
        }
      } else if (C::kF16 && warp >= kConvWarp0) {
        const int ct = threadIdx.x - kConvWarp0 * 32;
        for (int i = 0; i < mt; ++i) {
          const uint32_t st = cnt + i;
          const int s = st % C::kStages, o = st & 1;
          if (!mbar_wait_or_abort(&b.full[s], (st / C::kStages) & 1, p.err_flag, b.abort)) break;
          if (!mbar_wait_or_abort(&b.op_empty[o], ((st >> 1) & 1) ^ 1, p.err_flag, b.abort)) break;
          __syncwarp();
          const uint8_t* src = smem + C::kOffStage + s * C::kStageBytes;
          uint8_t* dst = smem + C::kOffOp + o * 32768;
          if (KV == kKvFp4)
            convert_tile_fp4<32 * kConvWarps>(src, dst, kTile, ct);
          else
            convert_tile<32 * kConvWarps>(src, dst, kTile, ct);
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
  umma::fence_before_sync();
  __syncthreads();
  if (*b.abort) {
    // a wait gave up: let the MMAs and the loads in flight end
    if (warp == 1 && lane == 0) {
      umma::commit(b.drain);
      mbar_wait(b.drain, 0, p.err_flag);
    }
    if (threadIdx.x == 0) {
      const uint64_t since = global_timer_ns();
      while (global_timer_ns() - since < 1000000) {}     // 1 ms: far longer than any copy takes
    }
    __syncthreads();
  }
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
