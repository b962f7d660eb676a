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
// select_kernel: one block per (segment, kv head).  A radix select over the
// weights' order-preserving 32-bit keys, eight bits a pass, finds the
// keep[s]-th largest; one ordered pass over the slots then numbers holes and
// movers (ties at the threshold stay lowest slot first), writes the pairs and
// moves the weights and positions.
// move_kernel: a warp per pair, 16 lanes a K row and 16 a V row.
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// Larger weight, larger key; both zeros alike, a NaN above every number and
// a protected position above all.
__device__ __forceinline__ uint32_t order_key(float m, bool guarded) {
  if (guarded) return 0xFFFFFFFFu;
  if (m != m) return 0xFFFFFFFEu;
  const uint32_t b = __float_as_uint(m + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive prefix sums over the block of two 16-bit counts packed in x (the
// block's totals stay below 2^16); total: their sums.
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
  uint32_t w = warp_s[lane];
  uint32_t winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += y;
  }
  total = __shfl_sync(0xffffffffu, winc, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, winc - w, warp);
  return before + inc - x;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(
    const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_s[kSelWarps];
  __shared__ uint32_t pick[2];
  allow_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x;
  const EvictSeg& sg = p.segs[blockIdx.x / p.hkv];
  const int g = blockIdx.x % p.hkv;
  const size_t plane = (size_t)sg.index * p.hkv + g;
  float* mass = p.mass + plane * p.mass_cap;
  int32_t* pos = p.key_pos ? p.key_pos + plane * p.mass_cap : nullptr;
  int32_t* moves = p.moves + plane * (p.mass_cap + 4);
  const int L = sg.seq_len, n = sg.keep;
  if (n == L) {                         // everything stays
    if (tid == 0) moves[0] = 0;
    return;
  }
  const int guard_from = sg.next_pos - p.recent;
  auto key_of = [&](int j) {
    const int at = pos ? pos[j] : j;
    return order_key(mass[j], at < p.sink || at >= guard_from);
  };
  // ---- the n-th largest key: `prefix` its leading bits, `want` its rank
  // among the keys that share them
  uint32_t prefix = 0, want = (uint32_t)n;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t hi = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int j = tid; j < L; j += kSelThreads) {
      const uint32_t k = key_of(j);
      if ((k & hi) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 32) {                     // lane i: digits 255 - 8 i down to 248 - 8 i
      uint32_t own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += hist[255 - (8 * tid + i)];
      uint32_t inc = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += y;
      }
      uint32_t above = inc - own;
      if (above < want && want <= inc) {
        int d = 255 - 8 * tid;
        while (above + hist[d] < want) above += hist[d--];
        pick[0] = (uint32_t)d;
        pick[1] = want - above;
      }
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    want = pick[1];
  }
  // ---- holes and movers, in slot order.  Of the keys equal to the
  // threshold the first `want` stay.
  uint32_t equal_before = 0, holes = 0, movers = 0;
  for (int base = 0; base < L; base += kSelThreads) {
    const int j = base + tid;
    const uint32_t k = j < L ? key_of(j) : 0u;
    const bool eq = j < L && k == prefix;
    uint32_t total;
    const uint32_t er = block_prefix(eq ? 1u : 0u, warp_s, total) + equal_before;
    equal_before += total;
    const bool stays = j < L && (k > prefix || (eq && er < want));
    const bool hole = j < n && !stays, mover = j >= n && stays;
    const uint32_t r = block_prefix((hole ? 1u : 0u) | (mover ? 0x10000u : 0u), warp_s, total);
    if (hole) moves[4 + 2 * (holes + (r & 0xFFFFu)) + 1] = j;
    if (mover) moves[4 + 2 * (movers + (r >> 16))] = j;
    holes += total & 0xFFFFu;
    movers += total >> 16;
  }
  if (tid == 0) moves[0] = (int32_t)holes;
  __syncthreads();
  // ---- weights and positions follow their keys; the slots behind are empty
  for (uint32_t i = tid; i < holes; i += kSelThreads) {
    const int src = moves[4 + 2 * i], dst = moves[4 + 2 * i + 1];
    mass[dst] = mass[src];
    if (pos) pos[dst] = pos[src];
  }
  __syncthreads();
  for (int j = n + tid; j < L; j += kSelThreads) {
    mass[j] = 0.f;
    if (pos) pos[j] = -1;
  }
}

constexpr int kMoveWarps = 8;

// Blocks: grid_x per (segment, kv head).  A pair on a page whose id is
// out of range is skipped and flagged.
template <int KV>
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(
    const __grid_constant__ EvictParams p) {
  allow_next_grid();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int plane = blockIdx.x / p.grid_x, bx = blockIdx.x - plane * p.grid_x;
  const EvictSeg& sg = p.segs[plane / p.hkv];
  const int g = plane % p.hkv;
  const int32_t* moves = p.moves + ((size_t)sg.index * p.hkv + g) * (p.mass_cap + 4);
  const int count = moves[0];
  const bool is_v = lane >= 16;
  const int t = lane & 15;
  uint8_t* base = static_cast<uint8_t*>(is_v ? sg.v_base : sg.k_base);
  auto row_of = [&](int slot, bool& ok) -> size_t {
    if (!sg.page_table) return (size_t)g * sg.slab_cap + slot;
    const int pid = __ldg(sg.page_table + (slot >> 8));
    ok = ok && (unsigned)pid < (unsigned)p.num_pages;
    return ((size_t)pid * p.hkv + g) * kPage + (slot & (kPage - 1));
  };
  for (int i = bx * kMoveWarps + (threadIdx.x >> 5); i < count; i += p.grid_x * kMoveWarps) {
    const int2 m = *reinterpret_cast<const int2*>(moves + 4 + 2 * i);
    bool ok = true;
    const size_t src = row_of(m.x, ok), dst = row_of(m.y, ok);
    if (!ok) {
      if (lane == 0) flag_error(p.err_flag, kErrBadPage);
      continue;
    }
    if (KV == kKvBf16) {
      reinterpret_cast<uint4*>(base)[dst * 16 + t] = reinterpret_cast<const uint4*>(base)[src * 16 + t];
    } else if (KV == kKvFp8) {
      reinterpret_cast<uint2*>(base)[dst * 16 + t] = reinterpret_cast<const uint2*>(base)[src * 16 + t];
    } else {
      *reinterpret_cast<uint32_t*>(base + fp4_codes(dst) + 4 * t) =
          *reinterpret_cast<const uint32_t*>(base + fp4_codes(src) + 4 * t);
      if (t < 2)
        *reinterpret_cast<uint32_t*>(base + fp4_scales(dst) + 4 * t) =
            *reinterpret_cast<const uint32_t*>(base + fp4_scales(src) + 4 * t);
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  return launch_pdl(select_kernel, dim3(p.nsegs * p.hkv), dim3(kSelThreads), 0, s, p);
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
