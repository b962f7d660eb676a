// Attention of each row over its own blocks of keys (tfpa_decode_blocks).
//
// A work item is a row, a kv head and up to 8 or 16 of its query heads; its
// list of blocks is cut into up to eight equal parts.  The item's CTAs are a
// cluster, and their parts' states (running maximum, sum, unnormalised output)
// meet in distributed shared memory, so there is one launch, no scratch and no
// merge kernel.  The parts follow from the list's length alone and each has a
// state of its own, so a row's bytes do not depend on its batch; how many of them
// a CTA takes, one after the other, does (a CTA of few keys is mostly start and
// end: 32 rows' lists of 2,048 keys over 4 bits 40.3 us with a part each, 30.3 us
// with four).
// Per CTA:
//   warp 4      producer: a lane a list entry looks the entry and its page up
//               (the chain of two loads runs once a 32 entries), then blocks
//               stream in as stages of 64 keys (bf16: 32), K and V (TMA tiles
//               with 128B swizzle; a 4-bit cache's codes and scales as bulk
//               copies);
//   warps 0..3  consumers: 16 keys of a stage each (bf16: two warps a stage, the
//               pairs in turn).  Both products have the
//               keys' side as the MMA's 16 rows and the query vectors as its 8
//               columns (with the vectors as rows, 4 query heads would leave 12
//               of 16 rows empty): S^T = K Q^T, weights transposed in registers,
//               O^T = V^T P^T.  Each warp keeps its own softmax state.
// What bounds it is the stream of K and V out of memory, with the start and the
// cluster's end around it: 8 streams' lists of 4,096 bf16 keys (134 MB, a part a
// CTA) take 26.5 us, 5.1 TB/s, one stream's 5.5 us.  Over e4m3 (67 MB) they take 18.4
// us, 3.6 TB/s, over 4 bits (38 MB) 16.5 us, 2.3 TB/s: the start and the end stay, and
// the consumers issue in 37 and 46 % of the cycles.  With four draft rows a stream,
// whose lists mostly name the same blocks, it is the second-level cache's reads
// over bf16 (32 lists of 2,048 keys: 37.1 us, 7.2 TB/s) and over the narrower types
// the consumers' instructions, most of them conversions (e4m3 30.2 us, 4 bits 30.3,
// an instruction in 55 % of the cycles; folding the parts' states is 1.5 us of it).
// One stream's long list is bound by its eight parts a kv head: 65,536 bf16 keys of 2
// kv heads 109 us (16 CTAs, 0.6 TB/s), of 8 kv heads 111 us (64 CTAs, 2.4 TB/s).  The
// kernels of several parts a CTA spill 8 to 48 bytes a thread (registers for four, or
// two, CTAs a SM).
#include "cluster.cuh"
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kRow = kHeadDim + 4;   // floats of a state's row: columns in banks of their own

template <int KV>
struct Cfg {
  static constexpr bool kF16 = KV != kKvBf16;          // f16 operands, kv head scales
  // f16 weights, and with them the sums and the output before its division, are 2^7
  // times 2^(score - running maximum): scores pass the maximum by 2^8 at most
  // (kRescaleThreshold), so they stay below 2^15 of f16's 2^16, and what is far below
  // the maximum keeps 7 bits more above f16's last one, 2^-24.  (Without them weights
  // from 2^-25 down would be lost, while their keys count in the sum.)
  static constexpr float kWeightLog2 = kF16 ? 7.f : 0.f;
  static constexpr int kStageKeys = KV == kKvBf16 ? 32 : 64;
  static constexpr int kStageWarps = kStageKeys / 16;  // consumer warps that read a stage
  static constexpr int kGroups = kConsumers / kStageWarps;   // and groups of them, in turn
  static constexpr int kHalfStage =                    // K of 64 keys, or V
      kStageKeys * (KV == kKvBf16 ? 256 : KV == kKvFp8 ? 128 : kFp4CodeBytes + kFp4ScaleBytes);
  static constexpr int kStageBytes = 2 * kHalfStage;
  // four CTAs of eight vectors a SM: a batch's clusters of eight then run at once
  static constexpr int kStages = KV == kKvFp4 ? 5 : 3;
  static constexpr int kRing = kStages * kStageBytes;
};

struct Shared {
  uint64_t full[8], empty[8];
  int key0[8];                 // first key of a stage; -1: a part's end
  int lost;                    // a wait gave up
  float m[16], l[16];          // the CTA's state, read by the cluster (with the ring's start)
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// The key (of 16) in row i of a score tile.  4 bits: a lane's V rows are those
// of columns 2c and 2c + 1 of the weights; rows c and 4 + (c ^ 1) lie next to
// each other over the lanes, and neighbouring K rows, 64 bytes each, in
// different halves of the banks.
template <int KV>
__device__ __forceinline__ int key_of(int i) {
  if (KV != kKvFp4) return i;
  return (i & 8) + (i & 1 ? 4 + (((i >> 1) & 3) ^ 1) : (i >> 1) & 3);
}

// Head dim of row i (0..15) of output tile t.
template <int KV>
__device__ __forceinline__ int dim_of(int t, int i) {
  if (KV == kKvBf16) return 16 * t + i;
  if (KV == kKvFp8) return 16 * t + 2 * (i & 7) + (i >> 3);
  return 16 * (i & 7) + 2 * t + (i >> 3);
}

// K rows `row` of the stage as operand registers: the 32 dims that this lane
// (column c of its quad) holds of a row, in the order of load_q.
template <int KV>
__device__ __forceinline__ void load_k(uint32_t sb, int row, int c, uint32_t (&k)[16]) {
  if (KV == kKvBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = sb + (i >> 1) * (Cfg<KV>::kHalfStage / 2);
      const uint4 w = lds128(swz128(at, row, 2 * c + (i & 1)));
      k[4 * i] = w.x;
      k[4 * i + 1] = w.y;
      k[4 * i + 2] = w.z;
      k[4 * i + 3] = w.w;
    }
  } else if (KV == kKvFp8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 w = lds128(swz128(sb, row, 2 * c + i));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[8 * i + 2 * j] = e4m3x2_to_f16x2((uint16_t)(ws[j] & 0xFFFF));
        k[8 * i + 2 * j + 1] = e4m3x2_to_f16x2((uint16_t)(ws[j] >> 16));
      }
    }
  } else {
    const uint4 w = lds128(sb + row * kFp4CodeBytes + 16 * c);
    const uint32_t s2 = e4m3x2_to_f16x2(
        (uint16_t)lds16(sb + Cfg<KV>::kStageKeys * kFp4CodeBytes + row * kFp4ScaleBytes + 2 * c));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[4];
      e2m1x8_to_f16x8(ws[j], h);
      const uint32_t s = prmt(s2, s2, j < 2 ? 0x1010 : 0x3232);
#pragma unroll
      for (int u = 0; u < 4; ++u) k[4 * j + u] = hmul2(h[u], s);
    }
  }
}

// Query vector `h` (nullptr: none) as this lane's 32 dims in operand registers,
// and the factor of its scores.  f16 operands: scaled by a power of two into
// f16 range, exact for every element within 2^28 of the vector's largest.
template <int KV>
__device__ __forceinline__ void load_q(const __nv_bfloat16* h, int c, float scale,
                                       uint32_t (&q)[16], float& factor) {
  const uint4* qp = reinterpret_cast<const uint4*>(h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = KV == kKvBf16 ? (i >> 1) * 8 + 2 * c + (i & 1) : 4 * c + i;
    const uint4 w = h ? *(qp + at) : make_uint4(0, 0, 0, 0);
    q[4 * i] = w.x;
    q[4 * i + 1] = w.y;
    q[4 * i + 2] = w.z;
    q[4 * i + 3] = w.w;
  }
  factor = scale;
  if (!Cfg<KV>::kF16) return;
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    amax = fmaxf(amax, fabsf(__uint_as_float(q[j] << 16)));
    amax = fmaxf(amax, fabsf(__uint_as_float(q[j] & 0xFFFF0000u)));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  int ex;
  frexpf(amax, &ex);
  ex = max(min(ex, 120), -100);
  const float up = __int_as_float((127 + 14 - ex) << 23);
#pragma unroll
  for (int j = 0; j < 16; ++j)
    q[j] = pack_f16x2(__uint_as_float(q[j] << 16) * up,
                      __uint_as_float(q[j] & 0xFFFF0000u) * up);
  factor = scale * __int_as_float((127 - 14 + ex) << 23);
}

// O^T += V^T P^T over 16 keys at rows r0.. of the stage (V at sb).  keep:
// masks of a lane's keys (columns 2c, 2c + 1 and 2c + 8, 2c + 9), which zero
// what lies behind the row's position (a weight of 0 would not: 0 NaN = NaN).
// pl: what bf16 leaves of the weights (over bf16 caches).
template <int KV, int NT>
__device__ __forceinline__ void add_pv(uint32_t sb, int r0, int lane, const uint32_t (&pb)[NT][2],
                                       const uint32_t (&pl)[NT][2], uint32_t keep0, uint32_t keep1,
                                       float (&o)[NT][8][4]) {
  const int gq = lane >> 2, c = lane & 3;
  auto mma = [&](int t, const uint32_t (&a)[4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (Cfg<KV>::kF16) {
        mma_f16_free(o[n][t], a, pb[n][0], pb[n][1]);
      } else {
        mma_bf16(o[n][t], a, pb[n][0], pb[n][1]);
        mma_bf16(o[n][t], a, pl[n][0], pl[n][1]);
      }
    }
  };
  if (KV == kKvBf16) {
    // matrices: keys 0-7 and 8-15 (lane bit 4) of two chunks of 8 dims (bit 3)
    const int row = r0 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      uint32_t a[4];
      ldmatrix_x4_trans(a, swz128(sb + (t >> 2) * (Cfg<KV>::kHalfStage / 2), row,
                                  (2 * t & 7) + ((lane >> 3) & 1)));
      a[0] &= keep0;
      a[1] &= keep0;
      a[2] &= keep1;
      a[3] &= keep1;
      mma(t, a);
    }
  } else if (KV == kKvFp8) {
    // a 16-bit column holds dims 2i and 2i + 1: rows i and i + 8 of a tile
    const int row = r0 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
      uint32_t w[4];
      ldmatrix_x4_trans(w, swz128(sb, row, t + (lane >> 4)));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t x = prmt(w[2 * u] & keep0, 0, 0x3120);
        const uint32_t y = prmt(w[2 * u + 1] & keep1, 0, 0x3120);
        const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)(x & 0xFFFF)),
                               e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                               e4m3x2_to_f16x2((uint16_t)(y & 0xFFFF)),
                               e4m3x2_to_f16x2((uint16_t)(y >> 16))};
        mma(t + u, a);
      }
    }
  } else {
    // dims 16 gq .. 16 gq + 15 of four keys: one scale each
    uint2 w[4];
    uint32_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + key_of<KV>(2 * c + (i & 1) + 8 * (i >> 1));
      w[i] = lds64(sb + row * kFp4CodeBytes + 8 * gq);
      s[i] = lds8(sb + Cfg<KV>::kStageKeys * kFp4CodeBytes + row * kFp4ScaleBytes + gq);
    }
    const uint32_t s01 = e4m3x2_to_f16x2((uint16_t)((s[0] | (s[1] << 8)) & prmt(keep0, 0, 0x4420)));
    const uint32_t s23 = e4m3x2_to_f16x2((uint16_t)((s[2] | (s[3] << 8)) & prmt(keep1, 0, 0x4420)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // a byte of two keys' equal nibbles converts to a pair along the keys
      uint32_t f[2][2][4];                 // [keys 0-7, 8-15][even, odd dims][pair]
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t A = i ? w[2 * k].y : w[2 * k].x, B = i ? w[2 * k + 1].y : w[2 * k + 1].x;
        e2m1x8_to_f16x8((A & 0x0F0F0F0Fu) | ((B & 0x0F0F0F0Fu) << 4), f[k][0]);
        e2m1x8_to_f16x8(((A >> 4) & 0x0F0F0F0Fu) | (B & 0xF0F0F0F0u), f[k][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a[4] = {hmul2(f[0][0][j], s01), hmul2(f[0][1][j], s01),
                               hmul2(f[1][0][j], s23), hmul2(f[1][1][j], s23)};
        mma(4 * i + j, a);
      }
    }
  }
}

// Lanes of a waiting state.
template <int NT>
__host__ __device__ constexpr int waiting_lanes(int group) {
  return NT == 1 && group <= 4 ? 16 : 32;
}

// Two states' common maximum goes into m; the factor that this one's sums take.
__device__ __forceinline__ float toward(float& m, float other) {
  const float M = fmaxf(m, other);
  const float a = m == -INFINITY ? 0.f : fast_exp2(m - M);
  m = M;
  return a;
}

// A warp's state in shared memory, [float4 of its fragments][lane], its maxima and
// sums behind them.  `lanes`: 32, or 16 where the vectors are four at most (a
// lane's columns are vectors 2c and 2c + 1): `at` is then -1 in the others.
template <int NT>
constexpr int kStateBytes = (8 * NT + NT) * 32 * 16;
template <int NT>
__device__ __forceinline__ void put_state(float4* to, int lanes, int at,
                                          const float (&o)[NT][8][4], const float (&m)[NT][2],
                                          const float (&l)[NT][2]) {
  if (at < 0) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      to[(8 * n + t) * lanes + at] = make_float4(o[n][t][0], o[n][t][1], o[n][t][2], o[n][t][3]);
    to[(8 * NT + n) * lanes + at] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
  }
}
// The state there and this one, in this one.  (Products and sums rounded on their
// own: the result is the same whichever of the two is there.)
template <int NT>
__device__ __forceinline__ void take_state(const float4* from, int lanes, int at,
                                           float (&o)[NT][8][4], float (&m)[NT][2],
                                           float (&l)[NT][2]) {
  if (at < 0) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float4 ml = from[(8 * NT + n) * lanes + at];
    float om[2] = {ml.x, ml.y};
    const float ol[2] = {ml.z, ml.w};
    float a[2], b[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float was = m[n][e];
      a[e] = toward(m[n][e], om[e]);
      b[e] = toward(om[e], was);
      l[n][e] = __fadd_rn(__fmul_rn(l[n][e], a[e]), __fmul_rn(ol[e], b[e]));
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float4 x = from[(8 * n + t) * lanes + at];
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[n][t][j] = __fadd_rn(__fmul_rn(o[n][t][j], a[j & 1]), __fmul_rn(y[j], b[j & 1]));
    }
  }
}

// The producer warp: a part, units [u0, u1) of the list, 64 keys each (a block of
// `per` units an entry), and its end.  False if a wait gave up.
template <int KV>
__device__ bool produce(const BlocksParams& p, const BlocksRun& run, const int32_t* list, int u0,
                        int u1, int per, int pos, int g, uint8_t* ring, Shared& sh,
                        uint32_t& stage) {
  using C = Cfg<KV>;
  const int lane = threadIdx.x & 31;
  const int i1 = (u1 + per - 1) / per;
  for (int base = u0 / per; base < i1; base += 32) {
    // a lane an entry: the block, and the storage row of its first key
    int b = -1, row0 = 0;
    if (base + lane < i1) b = *(list + base + lane);
    if (b >= 0 && (int64_t)b * p.block > pos) b = -1;
    if (b >= 0) {
      const int key0 = b * p.block;
      if (run.page_table) {
        const int pid = *(run.page_table + (key0 >> 8));
        if ((unsigned)pid < (unsigned)p.num_pages) {
          row0 = (pid * p.hkv + g) * kPage + (key0 & (kPage - 1));
        } else {
          flag_error(p.err_flag, kErrBadPage);
          b = -1;
        }
      } else {
        row0 = g * run.slab_cap + key0;
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, b >= 0);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int key0 = __shfl_sync(0xffffffffu, b, l) * p.block;
      const int r0 = __shfl_sync(0xffffffffu, row0, l);
      const int first = (base + l) * per;                // the entry's first unit
      const int n = min(64 * (u1 - first), min(p.block, pos - key0 + 1));
      for (int k = 64 * max(0, u0 - first); k < n; k += C::kStageKeys, ++stage) {
        const int buf = stage % C::kStages;
        if (!warp_wait(&sh.empty[buf], ((stage / C::kStages) & 1) ^ 1, p.err_flag)) return false;
        if (lane == 0) {
          uint64_t* fb = &sh.full[buf];
          uint8_t* sk = ring + (size_t)buf * C::kStageBytes;
          uint8_t* sv = sk + C::kHalfStage;
          const int y = r0 + k;
          sh.key0[buf] = key0 + k;
          mbar_arrive_expect_tx(fb, C::kStageBytes);
          if (KV == kKvFp4) {
            const size_t codes = fp4_codes(y), scales = fp4_scales(y);
            constexpr uint32_t kCodes = C::kStageKeys * kFp4CodeBytes;
            constexpr uint32_t kScales = C::kStageKeys * kFp4ScaleBytes;
            const uint8_t* kb = static_cast<const uint8_t*>(run.k_base);
            const uint8_t* vb = static_cast<const uint8_t*>(run.v_base);
            bulk_load(sk, kb + codes, kCodes, fb);
            bulk_load(sk + kCodes, kb + scales, kScales, fb);
            bulk_load(sv, vb + codes, kCodes, fb);
            bulk_load(sv + kCodes, vb + scales, kScales, fb);
          } else {
            const KVMaps& m = p.maps[run.src];
            tma_load_2d(sk, &m.k, 0, y, fb);
            if (KV == kKvBf16) tma_load_2d(sk + C::kHalfStage / 2, &m.k, 64, y, fb);
            tma_load_2d(sv, &m.v, 0, y, fb);
            if (KV == kKvBf16) tma_load_2d(sv + C::kHalfStage / 2, &m.v, 64, y, fb);
          }
        }
      }
    }
  }
  const int buf = stage % C::kStages;
  if (!warp_wait(&sh.empty[buf], ((stage / C::kStages) & 1) ^ 1, p.err_flag)) return false;
  if (lane == 0) {
    sh.key0[buf] = -1;
    mbar_arrive(&sh.full[buf]);
  }
  ++stage;
  return true;
}

// ONE: a CTA has one part (its code apart from the other keeps its registers).
template <int KV, int NT, bool ONE>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 2)
    decode_blocks_kernel(const __grid_constant__ BlocksParams p) {
  using C = Cfg<KV>;
  constexpr int kVecs = 8 * NT;
  __shared__ Shared sh;
  extern __shared__ uint8_t ring_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(ring_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)same_in_warp((uint32_t)tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kConsumers);
    }
    sh.lost = 0;
    fence_mbar_init();
  }
  allow_next_grid();
  __syncthreads();
  wait_prior_grid();
  // ---- the item, and this CTA's parts of its list
  const int cta = blockIdx.x % p.ctas;
  int item = blockIdx.x / p.ctas;
  const int qtiles = (p.group + kVecs - 1) / kVecs;
  const int qt = item % qtiles;
  item /= qtiles;
  const int row = item / p.hkv, g = item % p.hkv;
  const BlocksRun& run = p.runs[run_holding(p.runs, p.nruns, &BlocksRun::row0, row)];
  const int pos = run.pos0 + (row - run.row0);
  const int part0 = ONE ? cta : cta * p.cta_parts;
  const int nparts = ONE ? 1 : min(p.cta_parts, p.parts - part0);
  // the states that wait, [level], behind the ring and the fold where that is there too
  constexpr bool kInStage = C::kStageBytes >= 2 * kStateBytes<NT>;
  float4* pending =
      reinterpret_cast<float4*>(ring + C::kRing + (kInStage ? 0 : 2 * kStateBytes<NT>));
  // the CTA's state, once the ring is done
  float* mine = reinterpret_cast<float*>(ring + (ONE ? 4 * kStateBytes<NT> : 0));
  const int vecs = min(kVecs, p.group - qt * kVecs);     // query vectors of this item
  const size_t head0 = (size_t)row * p.hq + (size_t)g * p.group + qt * kVecs;

  const int gq = lane >> 2, c = lane & 3;
  float o[NT][8][4], m[NT][2], l[NT][2];
  if (warp == kConsumers) {
    const int32_t* list = p.blocks + ((size_t)row * p.hkv + g) * p.nsel;
    const int per = p.block / 64;
    const int64_t units = (int64_t)p.nsel * per;
    uint32_t stage = 0;
    bool ok = true;
    for (int i = part0; ok && i < part0 + nparts; ++i)
      ok = produce<KV>(p, run, list, (int)(units * i / p.parts), (int)(units * (i + 1) / p.parts),
                       per, pos, g, ring, sh, stage);
    if (!ok) sh.lost = 1;
  } else {
    uint32_t q[NT][16];
    float sc[NT][2];
    const float scale = C::kF16 ? p.scale_log2 * *(p.k_scale + g) : p.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int v = 8 * n + gq;
      float f;
      load_q<KV>(v < vecs ? p.q + (head0 + v) * kHeadDim : nullptr, c, scale, q[n], f);
      // the factors of the vectors in this lane's columns, 2c and 2c + 1
      sc[n][0] = __shfl_sync(0xffffffffu, f, 8 * c);
      sc[n][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
    }
    const int r0 = 16 * (warp % C::kStageWarps);
    // Every warp passes every stage, also those that are the other group's: the
    // parity of a phase tells it from the next one only, so a warp must not be
    // two loads of a stage ahead of what it has seen.
    uint32_t stage = 0;
    bool live = true;                      // no wait of this warp has given up
    for (int slot = 0; slot < nparts; ++slot) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
      }
      // (counted from the part's own first stage, so that a warp's keys are the
      // same in whatever CTA the part runs)
      for (uint32_t turn = 0; live; ++stage, ++turn) {
        const int buf = stage % C::kStages;
        live = warp_wait(&sh.full[buf], (stage / C::kStages) & 1, p.err_flag);
        if (!live) break;
        const int first = sh.key0[buf];
        if (first < 0) break;              // (the marker's stage is the fold's until released)
        const int key0 = first + r0;
        if (turn % C::kGroups == (uint32_t)(warp / C::kStageWarps) && key0 <= pos) {
          const uint32_t sk = smem_u32(ring + (size_t)buf * C::kStageBytes);
          // ---- S^T = K Q^T: keys key_of(gq), key_of(gq + 8); vectors 2c, 2c + 1
          float s[NT][4];
          {
            uint32_t ka[16], kb[16];
            load_k<KV>(sk, r0 + key_of<KV>(gq), c, ka);
            load_k<KV>(sk, r0 + key_of<KV>(gq + 8), c, kb);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t a[4] = {ka[2 * ks], kb[2 * ks], ka[2 * ks + 1], kb[2 * ks + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (C::kF16)
                  mma_f16_free(s[n], a, q[n][2 * ks], q[n][2 * ks + 1]);
                else
                  mma_bf16(s[n], a, q[n][2 * ks], q[n][2 * ks + 1]);
              }
            }
          }
          const bool see0 = key0 + key_of<KV>(gq) <= pos, see1 = key0 + key_of<KV>(gq + 8) <= pos;
          // ---- online softmax over the tile's keys, a column a vector.  The running
          // maximum moves by 2^8 at least, which after a part's first keys is rare:
          // one vote asks whether some score passes it by that.
          bool passes = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[n][e] = see0 ? s[n][e] * sc[n][e] : -INFINITY;
              s[n][2 + e] = see1 ? s[n][2 + e] * sc[n][e] : -INFINITY;
              passes |= fmaxf(s[n][e], s[n][2 + e]) > m[n][e] + kRescaleThreshold;
            }
          if (__any_sync(0xffffffffu, passes)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float al[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
                for (int d = 4; d < 32; d *= 2)
                  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                al[e] = 1.f;
                if (mx > m[n][e] + kRescaleThreshold) {
                  al[e] = fast_exp2(m[n][e] - mx);
                  l[n][e] *= al[e];
                  m[n][e] = mx;
                }
              }
#pragma unroll
              for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][t][j] *= al[j & 1];
            }
          }
          uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float base = (m[n][e] == -INFINITY ? 0.f : m[n][e]) - C::kWeightLog2;
              s[n][e] = fast_exp2(s[n][e] - base);
              s[n][2 + e] = fast_exp2(s[n][2 + e] - base);
              l[n][e] += s[n][e] + s[n][2 + e];
            }
            // Weights rounded to f16's 11 bits (kWeightLog2: to multiples of 2^-31 of the
            // running maximum's weight where they are below 2^-21 of it); bf16's 8 would
            // show in out, which is rounded to them too: a weight's first 8 bits, and the
            // rest rounded to 8 more, which costs 0.2 us of a batch's 26.2.  (The rest is
            // never 0 or negative beside a weight above 2^-102: an infinite V keeps its
            // sign.)  The sums are not rounded.  Two f16 numbers a weight would bring out
            // from 0.00168 to 0.00167 of 64 bits (the output's own rounding) for 0.7 us of
            // 30.1 (32 draft rows over 4 bits), 0.9 of 16.4 (8 streams, 64 blocks) and 5 of
            // 44.5 (the same with 32 query heads a kv head).
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = s[n][2 * i], y = s[n][2 * i + 1];
              if (C::kF16) {
                pb[n][i] = transpose8x8(pack_f16x2(x, y));
              } else {
                auto rest = [](float v) {
                  return fmaxf(v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), v * 0x1p-24f);
                };
                pb[n][i] = transpose8x8(prmt(__float_as_uint(x), __float_as_uint(y), 0x7632));
                pl[n][i] = transpose8x8(pack_bf16x2(rest(x), rest(y)));
              }
            }
          }
          // ---- O^T += V^T P^T
          auto mask = [&](int i) {
            return (key0 + key_of<KV>(2 * c + i) <= pos ? 0xFFFFu : 0u) |
                   (key0 + key_of<KV>(2 * c + 1 + i) <= pos ? 0xFFFF0000u : 0u);
          };
          add_pv<KV, NT>(sk + C::kHalfStage, r0, lane, pb, pl, mask(0), mask(8), o);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[buf]);
      }
      // ---- the part's state: the warps' in pairs, (0, 2) and (1, 3), then the two.
      // (A warp that gave up comes here too: the barriers count on all four.)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
      constexpr int kState = kStateBytes<NT> / 16;
      if (ONE) {
        // the only part: the whole ring is free, and all four warps fold
        float4* all = reinterpret_cast<float4*>(ring);
        named_bar_sync(1, 32 * kConsumers);
        put_state<NT>(all + warp * kState, 32, lane, o, m, l);
        named_bar_sync(1, 32 * kConsumers);
        break;
      }
      float4* fold = reinterpret_cast<float4*>(
          kInStage ? ring + (stage % C::kStages) * C::kStageBytes
                   : ring + C::kRing);
      if (!kInStage) named_bar_sync(1, 32 * kConsumers);   // the last part's fold is read
      if (warp >= 2) put_state<NT>(fold + (warp - 2) * (kStateBytes<NT> / 16), 32, lane, o, m, l);
      named_bar_sync(1, 32 * kConsumers);
      if (warp < 2) {
        take_state<NT>(fold + warp * (kStateBytes<NT> / 16), 32, lane, o, m, l);
        if (warp == 1) put_state<NT>(fold + kStateBytes<NT> / 16, 32, lane, o, m, l);
        named_bar_sync(2, 64);
        if (warp == 0) {
          take_state<NT>(fold + kStateBytes<NT> / 16, 32, lane, o, m, l);
          // and the parts' in pairs, pairs of pairs and so on, as the cluster goes on
          // to do: the states of the levels that lack their second half wait
          const int lanes = waiting_lanes<NT>(p.group);
          const int at = lanes == 32 ? lane : c < 2 ? 2 * gq + c : -1;
          const int wait = kStateBytes<NT> / 16 / 32 * lanes;
          int level = 0;
          for (; slot >> level & 1; ++level)
            take_state<NT>(pending + level * wait, lanes, at, o, m, l);
          if (slot + 1 < nparts)
            put_state<NT>(pending + level * wait, lanes, at, o, m, l);
          else
            for (; slot >> level; ++level)
              if (slot >> level & 1)
                take_state<NT>(pending + level * wait, lanes, at, o, m, l);
        }
      }
      if (kInStage && warp > 0) fence_proxy_async_smem();  // copies overwrite the fold next
      __syncwarp();
      if (live && lane == 0) mbar_arrive(&sh.empty[stage % C::kStages]);
      ++stage;
    }
    // ---- the CTA's state, [vector][dim], for the cluster
    if (ONE) {
      float4* all = reinterpret_cast<float4*>(ring);
      constexpr int kState = kStateBytes<NT> / 16;
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int t = (i * kConsumers + warp) % 8, n = (i * kConsumers + warp) / 8;
        // the pairs (0, 2) and (1, 3), then the two, as take_state adds them
        float4 ml[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) ml[w] = all[w * kState + (8 * NT + n) * 32 + lane];
        float f[4][2], h[2][2], mm[2], ll[2];   // factors of the pairs, and of the two
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m4[4], l4[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            m4[w] = e ? ml[w].y : ml[w].x;
            l4[w] = e ? ml[w].w : ml[w].z;
          }
          float ma = m4[0], mb = m4[1], m2 = m4[2], m3 = m4[3];
          const float a0 = toward(ma, m4[2]), a2 = toward(m2, m4[0]);
          const float b1 = toward(mb, m4[3]), b3 = toward(m3, m4[1]);
          const float la = __fadd_rn(__fmul_rn(l4[0], a0), __fmul_rn(l4[2], a2));
          const float lb = __fadd_rn(__fmul_rn(l4[1], b1), __fmul_rn(l4[3], b3));
          float mt = ma, mu = mb;
          h[0][e] = toward(mt, mb);
          h[1][e] = toward(mu, ma);
          mm[e] = mt;
          ll[e] = __fadd_rn(__fmul_rn(la, h[0][e]), __fmul_rn(lb, h[1][e]));
          f[0][e] = a0;
          f[1][e] = b1;
          f[2][e] = a2;
          f[3][e] = b3;
        }
        float x[4][4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 y = all[w * kState + (8 * n + t) * 32 + lane];
          x[w][0] = y.x;
          x[w][1] = y.y;
          x[w][2] = y.z;
          x[w][3] = y.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = j & 1;
          const float xa = __fadd_rn(__fmul_rn(x[0][j], f[0][e]), __fmul_rn(x[2][j], f[2][e]));
          const float xb = __fadd_rn(__fmul_rn(x[1][j], f[1][e]), __fmul_rn(x[3][j], f[3][e]));
          mine[(8 * n + 2 * c + e) * kRow + dim_of<KV>(t, gq + 8 * (j >> 1))] =
              __fadd_rn(__fmul_rn(xa, h[0][e]), __fmul_rn(xb, h[1][e]));
        }
        if (t == 0 && gq == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sh.m[8 * n + 2 * c + e] = mm[e];
            sh.l[8 * n + 2 * c + e] = ll[e];
          }
        }
      }
    } else if (warp == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mine[(8 * n + 2 * c + (j & 1)) * kRow + dim_of<KV>(t, gq + 8 * (j >> 1))] = o[n][t][j];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (gq == 0) {
            sh.m[8 * n + 2 * c + e] = m[n][e];
            sh.l[8 * n + 2 * c + e] = l[n][e];
          }
      }
    }
    if (!live) sh.lost = 1;
  }
  __syncthreads();
  if (sh.lost) let_copies_land();
  // ---- the CTAs' states, in the cluster's shared memory: each CTA finishes its
  // share of the item's elements, eight lanes one of four dims, a CTA each, so that
  // there is one trip to the other CTAs; pairs first, like the parts
  const float vs = C::kF16 ? *(p.v_scale + g) : 1.f;
  __syncwarp();
  if (p.ctas > 1) cluster_sync();
  const int j = lane & 7;
  const int share = (vecs * (kHeadDim / 4) + p.ctas - 1) / p.ctas;
  const int e1 = min(vecs * (kHeadDim / 4), (cta + 1) * share);
  for (int e0 = cta * share + (warp * 32 + lane) / 8; e0 - (lane >> 3) < e1; e0 += kThreads / 8) {
    const int e = min(e0, e1 - 1), v = e / (kHeadDim / 4), d = e % (kHeadDim / 4) * 4;
    float M = -INFINITY, L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < p.ctas) {
      M = __uint_as_float(ld_cluster_u32(mapa_shared(smem_u32(&sh.m[v]), j)));
      L = __uint_as_float(ld_cluster_u32(mapa_shared(smem_u32(&sh.l[v]), j)));
      x = ld_cluster_f4(mapa_shared(smem_u32(mine + v * kRow + d), j));
    }
#pragma unroll
    for (int k = 1; k < 8; k *= 2) {
      const float a = toward(M, __shfl_xor_sync(0xffffffffu, M, k));
      const bool there = ((j ^ k) & ~(k - 1)) < p.ctas;    // the other half has a CTA
      auto both = [&](float y) {
        y = __fmul_rn(y, a);
        const float z = __shfl_xor_sync(0xffffffffu, y, k);
        return there ? __fadd_rn(y, z) : y;
      };
      L = both(L);
      x.x = both(x.x);
      x.y = both(x.y);
      x.z = both(x.z);
      x.w = both(x.w);
    }
    if (j != 0 || e0 >= e1) continue;
    const float f = L == 0.f ? 0.f : vs / L;         // no key: zeros
    uint2 w;
    w.x = pack_bf16x2(x.x * f, x.y * f);
    w.y = pack_bf16x2(x.z * f, x.w * f);
    *reinterpret_cast<uint2*>(p.out + (head0 + v) * kHeadDim + d) = w;
    if (d == 0 && p.lse)
      p.lse[head0 + v] =
          L == 0.f ? -INFINITY : (M - C::kWeightLog2 + log2f(L)) * 0.6931471805599453f;
  }
  __syncwarp();
  if (p.ctas > 1) cluster_sync();                    // read, before a CTA's memory goes
}

// Shared memory of a CTA that takes `parts` parts of `group` vectors: the ring, and
// the fold's two states where a stage does not hold them, and those that wait for
// their second half.
template <int KV, int NT>
constexpr int smem_of(int parts, int group) {
  const int fold = Cfg<KV>::kStageBytes >= 2 * kStateBytes<NT> ? 0 : 2 * kStateBytes<NT>;
  const int levels = parts > 4 ? 3 : parts > 2 ? 2 : parts > 1 ? 1 : 0;
  const int waits = levels * (kStateBytes<NT> / 32 * waiting_lanes<NT>(group));
  return Cfg<KV>::kRing + 1024 + (parts == 1 ? 0 : fold + waits);
}

template <int KV, int NT, bool ONE>
cudaError_t launch(const BlocksParams& p, cudaStream_t s) {
  static_assert(4 * kStateBytes<NT> + 8 * NT * kRow * 4 <= Cfg<KV>::kRing, "the states' memory");
  static_assert(smem_of<KV, NT>(8, 16) + sizeof(Shared) <= 232448, "shared memory");
  static PerDeviceOnce configured;
  const cudaError_t e = configured.run([] {
    return cudaFuncSetAttribute(decode_blocks_kernel<KV, NT, ONE>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_of<KV, NT>(ONE ? 1 : 8, 16));
  });
  if (e != cudaSuccess) return e;
  const int qtiles = (p.group + 8 * NT - 1) / (8 * NT);
  const dim3 grid(p.rows * p.hkv * qtiles * p.ctas);
  return launch_pdl_cluster(decode_blocks_kernel<KV, NT, ONE>, grid, dim3(kThreads),
                            smem_of<KV, NT>(p.cta_parts, p.group), s, p, p.ctas);
}

template <int KV>
cudaError_t launch_of(const BlocksParams& p, cudaStream_t s) {
  if (p.group <= 8)
    return p.cta_parts == 1 ? launch<KV, 1, true>(p, s) : launch<KV, 1, false>(p, s);
  return p.cta_parts == 1 ? launch<KV, 2, true>(p, s) : launch<KV, 2, false>(p, s);
}

}  // namespace

cudaError_t launch_decode_blocks(const BlocksParams& p, int kv, cudaStream_t s) {
  switch (kv) {
    case kKvBf16: return launch_of<kKvBf16>(p, s);
    case kKvFp8: return launch_of<kKvFp8>(p, s);
    default: return launch_of<kKvFp4>(p, s);
  }
}

}  // namespace tfpa
