// Eviction: of every segment and kv head the keep[s] keys of largest
// accumulated weight stay (positions among the first `sink` and the last
// `recent` before all others), packed into slots [0, keep[s]).
//
// Attention does not depend on the order of a head's keys, so nothing is
// shifted: a key that stays in a slot below keep[s] stays where it is, and
// each evicted slot below it (a hole) takes one of the keys that stay behind
// it (a mover), holes and movers both in ascending order.  Sources and
// destinations are disjoint, so all rows move at once, in place, without
// staging; about keep (L - keep) / L rows of L move.
//
// select_kernel: a cluster of one to eight blocks per (segment, kv head), each
// with an equal run of slots whose keys (the weights' order-preserving 32-bit
// form) it keeps in shared memory where they fit.  A radix select over 11, 11
// and 10 bits finds the keep[s]-th largest key: the blocks' histograms are
// added up through distributed shared memory, every block for itself.  Then
// the slots are gone through in order, a thread four of them: holes and movers
// are counted (of the keys equal to the threshold the first slots stay; where
// not all of them do, they are counted first), numbered and written.  What
// bounds it is the chain of three passes and the numbering, each ended by
// barriers of the block or the cluster (8 streams of 16,384 to 32,768 keys: 26 us,
// issue slots 47 % busy, DRAM 6 %); four keys a step shorten its links.
// A run's lists are put in rank order in shared memory and written by
// consecutive lanes (a lane writing its own slots' numbers spread each store
// over four times the sectors: 14 -> 7 us of the choice's 46).
// move_kernel: a lane per 16 bytes of a row, so that a warp moves one bf16
// pair's K and V rows at a time, two e4m3 pairs' or four 4-bit ones' (a lane per
// four bytes of a 4-bit row: 231 -> 180 us for 8 streams of 32,768 to 65,536
// keys, the choice with it); the pairs' weights and positions go with them.
#include "cluster.cuh"
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Larger weight, larger key; both zeros alike, a NaN above every number and
// a protected position above all.
__device__ __forceinline__ uint32_t order_key(float m, bool guarded) {
  if (guarded) return 0xFFFFFFFFu;
  if (m != m) return 0xFFFFFFFEu;
  const uint32_t b = __float_as_uint(m + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive prefix sum of x over the block's threads; total: the sum.
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t* warp_s, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                      // warp_s of the previous call is read
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  const uint32_t w = warp_s[lane];
  uint32_t winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += y;
  }
  total = __shfl_sync(0xffffffffu, winc, 31);
  return __shfl_sync(0xffffffffu, winc - w, warp) + inc - x;
}

struct SelectShared {
  uint32_t hist[kBins];
  uint32_t warp_s[kSelWarps];
  uint32_t pick[3];
  uint32_t count[2];                    // what the other blocks of the cluster read
};

// CLUSTER: several blocks a (segment, kv head).
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) select_kernel(
    const __grid_constant__ EvictParams p) {
  __shared__ SelectShared sh;
  extern __shared__ uint4 keys[];        // [chunk / 4] where they fit
  allow_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31;
  const int nb = CLUSTER ? p.cluster : 1, rank = CLUSTER ? (int)cluster_ctarank() : 0;
  const int plane_i = blockIdx.x / nb;
  const EvictSeg& sg = p.segs[plane_i / p.hkv];
  const int g = plane_i % p.hkv;
  const size_t plane = (size_t)sg.index * p.hkv + g;
  float* mass = p.mass + plane * p.mass_cap;
  int32_t* pos = p.key_pos ? p.key_pos + plane * p.mass_cap : nullptr;
  int32_t* moves = p.moves + plane * (p.mass_cap + 4);
  const int L = sg.seq_len, n = sg.keep;
  if (n == L) {                         // everything stays (the cluster's blocks all leave)
    if (tid == 0 && rank == 0) moves[0] = 0;
    return;
  }
  auto sync = [] {
    if (CLUSTER) {
      __syncwarp();
      cluster_sync();
    } else {
      __syncthreads();
    }
  };
  // The sum over the cluster's blocks of one's shared word, and over the
  // blocks before this one.
  auto cluster_sum = [&](const uint32_t* a, uint32_t& before) {
    before = 0;
    if (!CLUSTER) return *a;
    uint32_t s = 0;
    for (int r = 0; r < nb; ++r) {
      const uint32_t v = ld_cluster_u32(mapa_shared(smem_u32(a), r));
      s += v;
      if (r < rank) before += v;
    }
    return s;
  };
  // this block's slots; a step takes kSelThreads threads' four
  const int chunk = select_chunk(L, nb);
  const int lo = min(L, rank * chunk), hi = min(L, lo + chunk);
  const bool kept = chunk <= p.key_slots;
  int next_pos = sg.next_pos;
  if (next_pos == kNextPosHeld) {       // the largest position that a slot holds, plus one
    int most = -1;
    for (int j = lo + tid; j < hi; j += kSelThreads) most = max(most, pos[j]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) sh.warp_s[tid >> 5] = (uint32_t)most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, (int)sh.warp_s[lane]);
    if (tid == 0) sh.count[0] = (uint32_t)most;
    sync();
    for (int r = 0; CLUSTER && r < nb; ++r)
      most = max(most, (int)ld_cluster_u32(mapa_shared(smem_u32(&sh.count[0]), r)));
    sync();                             // read, before count or warp_s is written again
    next_pos = most + 1;
  }
  const int guard_from = next_pos - p.recent;
  // Keys of slots j .. j + 3 (j a multiple of 4; 0, which no key is, from hi
  // on).  mass_cap is a multiple of 4, so the reads stay within the plane.
  auto make_keys = [&](int j) {
    const float4 m = *reinterpret_cast<const float4*>(mass + j);
    int4 at = make_int4(j, j + 1, j + 2, j + 3);
    if (pos) at = *reinterpret_cast<const int4*>(pos + j);
    auto one = [&](float x, int a, int i) {
      // (a negative position, a slot whose entry is not written, is neither)
      return i < hi ? order_key(x, a >= 0 && (a < p.sink || a >= guard_from)) : 0u;
    };
    return make_uint4(one(m.x, at.x, j), one(m.y, at.y, j + 1), one(m.z, at.z, j + 2),
                      one(m.w, at.w, j + 3));
  };
  auto keys_of = [&](int j) { return kept ? keys[(j - lo) >> 2] : make_keys(j); };
  // ---- the n-th largest key: `prefix` its leading bits, `want` its rank
  // among the keys that share them, `same` their number
  uint32_t prefix = 0, want = (uint32_t)n, same = 0, unused;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t high = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
    sh.hist[tid] = 0;
    sh.hist[tid + kSelThreads] = 0;
    __syncthreads();
    auto add = [&](const uint4& k) {
      const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v[u] && (v[u] & high) == prefix) atomicAdd(&sh.hist[(v[u] >> shift) & mask], 1u);
    };
    const int step = 4 * kSelThreads;
    int j = lo + 4 * tid;
    if (pass == 0) {
      for (; j + step < hi; j += 2 * step) {   // two steps' reads on their way
        const uint4 a = make_keys(j), b = make_keys(j + step);
        if (kept) {
          keys[(j - lo) >> 2] = a;
          keys[(j + step - lo) >> 2] = b;
        }
        add(a);
        add(b);
      }
      for (; j < hi; j += step) {
        const uint4 a = make_keys(j);
        if (kept) keys[(j - lo) >> 2] = a;
        add(a);
      }
    } else {
      for (; j < hi; j += step) add(keys_of(j));
    }
    sync();
    // thread t: bins 2047 - 2 t and 2046 - 2 t, from the largest down
    const int top = kBins - 1 - 2 * tid;
    const uint32_t c0 = cluster_sum(&sh.hist[top], unused);
    const uint32_t c1 = cluster_sum(&sh.hist[top - 1], unused);
    uint32_t total;
    const uint32_t above = block_prefix(c0 + c1, sh.warp_s, total);
    if (above < want && want <= above + c0 + c1) {
      const bool second = want > above + c0;
      sh.pick[0] = (uint32_t)(second ? top - 1 : top);
      sh.pick[1] = want - above - (second ? c0 : 0u);
      sh.pick[2] = second ? c1 : c0;
    }
    sync();                             // picked, and everyone has read the histograms
    prefix |= sh.pick[0] << shift;
    want = sh.pick[1];
    same = sh.pick[2];
    __syncthreads();
  }
  // ---- holes and movers in slot order, a warp's slots consecutive: runs of
  // 128, a lane four slots
  const int runs = (hi - lo + 127) >> 7;
  const int per = (runs + kSelWarps - 1) / kSelWarps;
  const int w0 = min(hi, lo + (tid >> 5) * per * 128), w1 = min(hi, w0 + per * 128);
  auto lane_keys = [&](int j0) {
    return j0 + 4 * lane < w1 ? keys_of(j0 + 4 * lane) : make_uint4(0, 0, 0, 0);
  };
  auto equal4 = [&](const uint4& k) {   // bit u: slot u's key is the threshold
    return (k.x == prefix ? 1u : 0u) | (k.y == prefix ? 2u : 0u) | (k.z == prefix ? 4u : 0u) |
           (k.w == prefix ? 8u : 0u);
  };
  auto above4 = [&](const uint4& k) {
    return (k.x > prefix ? 1u : 0u) | (k.y > prefix ? 2u : 0u) | (k.z > prefix ? 4u : 0u) |
           (k.w > prefix ? 8u : 0u);
  };
  // exclusive sum over the lanes before, and the warp's sum
  auto warp_prefix = [&](uint32_t x, uint32_t& sum) {
    uint32_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    sum = __shfl_sync(0xffffffffu, inc, 31);
    return inc - x;
  };
  uint32_t total, eq_at = 0;            // equal keys in slots before the run
  const bool ties = want < same;        // not all of the equal keys stay
  if (ties) {
    uint32_t eq = 0;
    for (int j0 = w0; j0 < w1; j0 += 128) eq += __popc(equal4(lane_keys(j0)));
    eq = __reduce_add_sync(0xffffffffu, eq);
    uint32_t before = block_prefix(lane == 0 ? eq : 0u, sh.warp_s, total);
    eq_at = __shfl_sync(0xffffffffu, before, 0);
    if (tid == 0) sh.count[0] = total;
    sync();
    cluster_sum(&sh.count[0], before);
    eq_at += before;
    sync();
  }
  // The lane's four slots: which stay; holes (below n) and movers (from n on)
  // among them.  Moves `at_eq` on over the run.
  auto look = [&](int j0, uint32_t& at_eq, unsigned& holes, unsigned& movers) {
    const int j = j0 + 4 * lane;
    const uint4 k = lane_keys(j0);
    unsigned e = equal4(k);
    if (ties) {
      uint32_t sum, r = at_eq + warp_prefix(__popc(e), sum);
      at_eq += sum;
      unsigned first = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (e >> u & 1u) {
          if (r < want) first |= 1u << u;
          ++r;
        }
      e = first;
    }
    const unsigned stays = above4(k) | e;
    const int nl = min(max(w1 - j, 0), 4), nn = min(max(n - j, 0), 4);
    const unsigned live = (1u << nl) - 1u, low = (1u << nn) - 1u;
    holes = ~stays & live & low;
    movers = stays & live & ~low;
    return live & ~low & ~stays;        // evicted slots behind the cut
  };
  uint32_t nh = 0, nm = 0;
  {
    uint32_t at_eq = eq_at;
    for (int j0 = w0; j0 < w1; j0 += 128) {
      unsigned holes, movers;
      look(j0, at_eq, holes, movers);
      nh += __popc(holes);
      nm += __popc(movers);
    }
  }
  nh = __reduce_add_sync(0xffffffffu, nh);
  nm = __reduce_add_sync(0xffffffffu, nm);
  uint32_t th, tm, hb, mb;
  uint32_t h0 = block_prefix(lane == 0 ? nh : 0u, sh.warp_s, th);
  uint32_t m0 = block_prefix(lane == 0 ? nm : 0u, sh.warp_s, tm);
  h0 = __shfl_sync(0xffffffffu, h0, 0);
  m0 = __shfl_sync(0xffffffffu, m0, 0);
  if (tid == 0) {
    sh.count[0] = th;
    sh.count[1] = tm;
  }
  sync();
  const uint32_t all = cluster_sum(&sh.count[0], hb);
  cluster_sum(&sh.count[1], mb);
  h0 += hb;
  m0 += mb;
  if (tid == 0 && rank == 0) moves[0] = (int32_t)all;
  uint8_t* list = reinterpret_cast<uint8_t*>(sh.hist) + 256 * (tid >> 5);   // 32 warps x 256 bytes
  {
    uint32_t at_eq = eq_at;
    for (int j0 = w0; j0 < w1; j0 += 128) {
      unsigned holes, movers;
      const unsigned gone = look(j0, at_eq, holes, movers);
      const int j = j0 + 4 * lane;
      // both ranks in one scan (a run has at most 128 of each)
      uint32_t sum;
      const uint32_t r = warp_prefix(__popc(holes) | (uint32_t)__popc(movers) << 16, sum);
      // each list in rank order in the warp's part of shared memory (the slots'
      // offsets in the run), then written by consecutive lanes
      uint32_t rh = r & 0xFFFFu, rm = r >> 16;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (holes >> u & 1u) list[rh++] = (uint8_t)(4 * lane + u);
        if (movers >> u & 1u) list[128 + rm++] = (uint8_t)(4 * lane + u);
      }
      __syncwarp();
      const uint32_t nholes = sum & 0xFFFFu, nmovers = sum >> 16;
      for (uint32_t i = lane; i < nholes; i += 32) moves[4 + 2 * (h0 + i) + 1] = j0 + list[i];
      for (uint32_t i = lane; i < nmovers; i += 32) moves[4 + 2 * (m0 + i)] = j0 + list[128 + i];
      __syncwarp();
      h0 += nholes;
      m0 += nmovers;
      // the evicted slots behind the cut (a mover's is emptied when it moves);
      // the lane's other slots are written back as they are
      if (gone) {
        float4 m = *reinterpret_cast<const float4*>(mass + j);
        m = make_float4(gone & 1u ? 0.f : m.x, gone & 2u ? 0.f : m.y, gone & 4u ? 0.f : m.z,
                        gone & 8u ? 0.f : m.w);
        *reinterpret_cast<float4*>(mass + j) = m;
        if (pos) {
          int4 a = *reinterpret_cast<const int4*>(pos + j);
          a = make_int4(gone & 1u ? -1 : a.x, gone & 2u ? -1 : a.y, gone & 4u ? -1 : a.z,
                        gone & 8u ? -1 : a.w);
          *reinterpret_cast<int4*>(pos + j) = a;
        }
      }
    }
  }
  sync();                               // no block leaves while another reads its counts
}

constexpr int kMoveWarps = 8;

// Lane t's part of a stored row: 16 bytes, as many lanes as the row has (4
// bits: of its codes; lane 0 takes the scales too).  Rows are read and written
// once, and the loads and stores say so (8 streams of 32,768 to 65,536 bf16
// keys 201 -> 193 us, the choice with it).
template <int KV>
struct MoveRow {
  static constexpr int kLanes = KV == kKvBf16 ? 16 : KV == kKvFp8 ? 8 : 4;
  uint4 v;
  uint2 scales;
  __device__ __forceinline__ void load(const uint8_t* b, size_t r, int t) {
    if (KV == kKvFp4) {
      v = __ldcs(reinterpret_cast<const uint4*>(b + fp4_codes(r)) + t);
      if (t == 0) scales = __ldcs(reinterpret_cast<const uint2*>(b + fp4_scales(r)));
    } else {
      v = __ldcs(reinterpret_cast<const uint4*>(b) + r * kLanes + t);
    }
  }
  __device__ __forceinline__ void store(uint8_t* b, size_t r, int t) const {
    if (KV == kKvFp4) {
      __stcs(reinterpret_cast<uint4*>(b + fp4_codes(r)) + t, v);
      if (t == 0) __stcs(reinterpret_cast<uint2*>(b + fp4_scales(r)), scales);
    } else {
      __stcs(reinterpret_cast<uint4*>(b) + r * kLanes + t, v);
    }
  }
};

// Blocks: grid_x per (segment, kv head).  A pair on a page whose id is
// out of range is skipped and flagged: its rows stay, and its weights and
// positions with them.
template <int KV>
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(
    const __grid_constant__ EvictParams p) {
  using Row = MoveRow<KV>;
  allow_next_grid();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int plane = blockIdx.x / p.grid_x, bx = blockIdx.x - plane * p.grid_x;
  const EvictSeg& sg = p.segs[plane / p.hkv];
  const int g = plane % p.hkv;
  const size_t at = (size_t)sg.index * p.hkv + g;
  const int32_t* moves = p.moves + at * (p.mass_cap + 4);
  float* mass = p.mass + at * p.mass_cap;
  int32_t* pos = p.key_pos ? p.key_pos + at * p.mass_cap : nullptr;
  const int count = moves[0];
  // a pair takes 2 kLanes lanes, K's and V's; a warp kPairs pairs at a time
  constexpr int kPairs = 16 / Row::kLanes;
  const int sub = lane / (2 * Row::kLanes), t = lane % Row::kLanes;
  const bool is_v = lane / Row::kLanes & 1;
  uint8_t* base = static_cast<uint8_t*>(is_v ? sg.v_base : sg.k_base);
  auto page_of = [&](int slot, bool& ok) {
    const int pid = __ldg(sg.page_table + (slot >> 8));
    ok = ok && (unsigned)pid < (unsigned)p.num_pages;
    return pid;
  };
  auto row_of = [&](int slot, bool& ok) -> size_t {
    if (!sg.page_table) return (size_t)g * sg.slab_cap + slot;
    const int pid = page_of(slot, ok);
    return ((size_t)pid * p.hkv + g) * kPage + (slot & (kPage - 1));
  };
  // A warp takes pairs in batches, every one's row on its way before the
  // first is stored.
  constexpr int kSteps = 4, kBatch = kSteps * kPairs;
  for (int i0 = (bx * kMoveWarps + (threadIdx.x >> 5)) * kBatch; i0 < count;
       i0 += p.grid_x * kMoveWarps * kBatch) {
    if (lane < kBatch && i0 + lane < count) {   // weights and positions: a lane a pair
      const int2 m = *reinterpret_cast<const int2*>(moves + 4 + 2 * (i0 + lane));
      bool ok = true;
      if (sg.page_table) {
        page_of(m.x, ok);
        page_of(m.y, ok);
      }
      if (ok) {
        mass[m.y] = mass[m.x];
        mass[m.x] = 0.f;
        if (pos) {
          pos[m.y] = pos[m.x];
          pos[m.x] = -1;
        }
      }
    }
    Row row[kSteps];
    size_t dst[kSteps];
    bool ok[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int i = i0 + u * kPairs + sub;
      ok[u] = i < count;
      if (!ok[u]) continue;
      const int2 m = *reinterpret_cast<const int2*>(moves + 4 + 2 * i);
      const size_t src = row_of(m.x, ok[u]);
      dst[u] = row_of(m.y, ok[u]);
      if (ok[u])
        row[u].load(base, src, t);
      else if (t == 0)
        flag_error(p.err_flag, kErrBadPage);
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (ok[u]) row[u].store(base, dst[u], t);
  }
}

}  // namespace

// The blocks keep their keys in shared memory if the longest segment's share
// fits (key_slots); a longer one's are formed anew each pass.
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  static PerDeviceOnce configured;
  const cudaError_t e = configured.run([] {
    const cudaError_t r = cudaFuncSetAttribute(
        select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectKeys * 4);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSelectKeys * 4);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(p.nsegs * p.hkv * p.cluster), block(kSelThreads);
  const size_t smem = (size_t)p.key_slots * 4;
  return p.cluster > 1 ? launch_pdl_cluster(select_kernel<true>, grid, block, smem, s, p, p.cluster)
                       : launch_pdl(select_kernel<false>, grid, block, smem, s, p);
}

cudaError_t launch_evict_move(const EvictParams& p, int kv, cudaStream_t s) {
  if (p.grid_x <= 0) return cudaSuccess;
  const dim3 grid(p.grid_x * p.nsegs * p.hkv), block(32 * kMoveWarps);
  switch (kv) {
    case kKvBf16: return launch_pdl(move_kernel<kKvBf16>, grid, block, 0, s, p);
    case kKvFp8: return launch_pdl(move_kernel<kKvFp8>, grid, block, 0, s, p);
    default: return launch_pdl(move_kernel<kKvFp4>, grid, block, 0, s, p);
  }
}

}  // namespace tfpa
