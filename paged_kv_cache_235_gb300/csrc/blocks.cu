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
#include "cluster.cuh"
#include "common.cuh"
#include "kvstore.cuh"
#include "params.h"

namespace tfpa {
namespace {

// ---------------------------------------------------------------- bounds
constexpr int kBoundThreads = 128;

// One CTA a (block, kv head): 16 lanes a row, 8 head dims a lane, 8 rows at a
// time.  Bound by the read of the keys: 32,768 bf16 keys of 8 kv heads (67 MB) in
// 13.4 us, 5.2 TB/s.  Over e4m3 (36 MB, 10.7 us) and 4 bits (21 MB, 12.9 us), of which a
// lane loads 8 and 4 bytes a row, it is the integer pipe, busy in 65 and 72 % of the
// cycles with conversions and comparisons.  A step's few blocks take 2.6 us, the launch
// and one read's latency.
template <int KV>
__global__ void __launch_bounds__(kBoundThreads)
    key_bounds_kernel(const __grid_constant__ BoundsParams p) {
  __shared__ uint4 part[2][kBoundThreads];
  allow_next_grid();
  wait_prior_grid();
  const int g = blockIdx.x % p.hkv;
  const int item = blockIdx.x / p.hkv;
  const BoundsRun& run = p.runs[run_holding(p.runs, p.nruns, &BoundsRun::item0, item)];
  const int block = run.block0 + (item - run.item0);
  const int64_t key0 = (int64_t)block * p.block;
  const int n = (int)min((int64_t)p.block, run.seq_len - key0);
  const int page = (int)(key0 >> 8);
  const int per_page = kPage / p.block, in_page = block % per_page;
  size_t row0, at;
  if (run.page_table) {
    const int pid = *(run.page_table + page);
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
  // lowest and highest so far, two dims a word: bf16 (a bf16 cache) or f16, which
  // hold every stored value
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = KV == kKvBf16 ? 0x7F807F80u : 0x7C007C00u;
    hi[i] = lo[i] | 0x80008000u;
  }
  constexpr int kRows = kBoundThreads / 16;          // rows at a time
  constexpr int kStep = 8;                           // and of those, loads in flight
  for (int r0 = threadIdx.x >> 4; r0 < n; r0 += kRows * kStep) {
    Raw8<KV> raw[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u)
      if (r0 + u * kRows < n) raw[u].load(run.k_base, row0 + r0 + u * kRows, t);
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      if (r0 + u * kRows >= n) break;
      uint32_t x[4];
      raw[u].words(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] &= number_mask<KV>(x[i]);               // a NaN counts as 0
        lo[i] = min2<KV>(lo[i], x[i]);
        hi[i] = max2<KV>(hi[i], x[i]);
      }
    }
  }
  part[0][threadIdx.x] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  part[1][threadIdx.x] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int which = threadIdx.x >> 4;        // lanes 0-15 the smallest, 16-31 the largest
  uint4 m = part[which][t];
  for (int r = 1; r < kRows; ++r) {
    const uint4 x = part[which][r * 16 + t];
    m.x = which ? max2<KV>(m.x, x.x) : min2<KV>(m.x, x.x);
    m.y = which ? max2<KV>(m.y, x.y) : min2<KV>(m.y, x.y);
    m.z = which ? max2<KV>(m.z, x.z) : min2<KV>(m.z, x.z);
    m.w = which ? max2<KV>(m.w, x.w) : min2<KV>(m.w, x.w);
  }
  if (KV != kKvBf16) {                       // f16 to bf16: at most six bits, exact
    m.x = bf16x2_of_f16x2(m.x);
    m.y = bf16x2_of_f16x2(m.y);
    m.z = bf16x2_of_f16x2(m.z);
    m.w = bf16x2_of_f16x2(m.w);
  }
  reinterpret_cast<uint4*>(run.bounds)[(at * 2 + which) * 16 + t] = m;
}

// ---------------------------------------------------------------- selection
// A cluster of one to eight CTAs takes a kv head and up to four consecutive rows
// of a stream.  Its CTAs share the blocks: a warp reads eight blocks' bounds at a
// time (16 bytes a lane, so the reads of a page are one run), forms all rows'
// scores from them and leaves them in the shared memory of the CTA that chooses
// for the row (rank r for row r).  What bounds that part is the read of the
// bounds, once for the rows together.
// The choice: the scores' leading bits that all of them share are passed over,
// a histogram of the next 11 finds the bin of the border, and few keys in it are
// ranked one against all (else 11 bits more).  Barriers and their latencies are
// what it costs, not work: of 8 streams' 2,048 blocks (67 MB of bounds, 20.2 us) 5 us,
// of one stream's 313 (6.4 us) half; 32 rows' 512 blocks, four rows a stream, 13.7 us.
// A choice that comes down to exact scores takes 2 us more.
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
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
__device__ __forceinline__ bool is_score(uint32_t k) { return k != kTaken && k != kAbsent; }
// The same of a float64 score; a NaN above every number.
__device__ __forceinline__ uint64_t order64(double s) {
  if (s != s) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

struct SelShared {
  union {
    uint32_t hist[kBins];
    double q64[256];         // sum_h min(q, 0) (0..127), sum_h max(q, 0) (128..255), for exact
                             // scores, between two uses of the histogram
    float q32[4][256];       // and before its first use, of each row
  };
  uint4 seen[kMaxCluster * kSelWarps];      // what every warp of the cluster has seen: the largest
                                            // |bound| (bf16 bits; ~0: a score was no number), the
                                            // smallest and largest key, taken << 16 | free blocks
  uint32_t warp_s[kSelWarps];
  uint32_t pick[3];
  uint32_t count;
  uint32_t border;
  int near_i[kNear];
  uint64_t near_k[kNear];
};
constexpr size_t kSelectSmem = (size_t)kSelectBlocks * 12;
static_assert(sizeof(SelShared) + kSelectSmem <= 232448, "shared memory");

// Exclusive prefix sum of x over the block's threads; total: the sum.
__device__ __forceinline__ uint32_t sel_prefix(uint32_t x, uint32_t* warp_s, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                       // warp_s of the previous call is read
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t v = warp_s[w];
    before += w < warp ? v : 0u;
    total += v;
  }
  return before + inc - x;
}

// Index (in blocks' bounds) of block b, or -1 on a page out of range.
__device__ __forceinline__ int bound_at(const SelectParams& p, const SelRun& run, int g, int b) {
  const int per_page = kPage / p.block;
  if (!run.page_table) return g * (run.slab_cap / p.block) + b;
  const int pid = *(run.page_table + b / per_page);
  if ((unsigned)pid >= (unsigned)p.num_pages) return -1;
  return (pid * p.hkv + g) * per_page + b % per_page;
}
// This lane's 16 bytes of it: lanes 0-15 the smallest, 16-31 the largest.
__device__ __forceinline__ uint4 bound_load(const SelRun& run, int at, int lane) {
  return *(static_cast<const uint4*>(run.bounds) + (size_t)at * 32 + lane);
}

// The query heads' negative parts of head dim d, and the positive ones, summed as
// float64 would: in float32 where no sum rounds, which heads of like size see to
// (64-bit adds are a sixty-fourth of the rate).
__device__ __forceinline__ void sum_heads64(const __nv_bfloat16* q, int group, int d,
                                            SelShared& sh) {
  float down = 0.f, up = 0.f;
  bool exact = true;
  // of one sign, so a sum that does not round gives both back
  auto add = [&](float& a, float x) {
    const float t = a + x;
    exact = exact && t - a == x && t - x == a;
    a = t;
  };
  for (int h0 = 0; h0 < group; h0 += 4) {
    float x[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      x[h] = h0 + h < group ? __bfloat162float(q[(size_t)(h0 + h) * kHeadDim + d]) : 0.f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      add(down, x[h] > 0.f ? 0.f : x[h]);
      add(up, x[h] < 0.f ? 0.f : x[h]);
    }
  }
  double a = down, b = up;
  if (!exact) {
    a = b = 0.0;
    for (int h = 0; h < group; ++h) {
      const float x = __bfloat162float(q[(size_t)h * kHeadDim + d]);
      a += x > 0.f ? 0.f : x;
      b += x < 0.f ? 0.f : x;
    }
  }
  sh.q64[d] = a;
  sh.q64[128 + d] = b;
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

// Sums over the warp's lanes of eight values a lane: lane l gets value l / 4's.
__device__ __forceinline__ float reduce8(const float (&v)[8], int lane) {
  float a[4], b[2], c;
  const bool u4 = lane & 16, u3 = lane & 8, u2 = lane & 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    a[j] = (u4 ? v[j + 4] : v[j]) + __shfl_xor_sync(0xffffffffu, u4 ? v[j] : v[j + 4], 16);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    b[j] = (u3 ? a[j + 2] : a[j]) + __shfl_xor_sync(0xffffffffu, u3 ? a[j] : a[j + 2], 8);
  c = (u2 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, u2 ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// The rows' blocks from the keys in this CTA's shared memory: the want-th
// largest, what is near it, and the list.  A thread takes eight consecutive keys
// of a round of 2,048, and keeps them in registers where one round is all.
__device__ void choose(const SelectParams& p, const SelRun& run, const __nv_bfloat16* q, int g,
                       int n, bool every, int ranks, float q1, uint32_t* key32,
                       uint64_t* key64, SelShared& sh, int32_t* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)same_in_warp((uint32_t)tid >> 5);
  constexpr int kRound = 8 * kSelThreads;
  const bool one = n <= kRound;
  bool loaded = false;
  uint32_t k[8];
  // fn(first block, its eight keys), round by round
  auto rounds = [&](auto&& fn) {
    for (int base = 0; base < n; base += kRound) {
      const int b = base + 8 * tid;
      if (!one || !loaded) {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = kAbsent;
        if (b < n) {                     // (the keys' memory is whole eights)
          const uint4 u = *reinterpret_cast<const uint4*>(key32 + b);
          const uint4 v = *reinterpret_cast<const uint4*>(key32 + b + 4);
          const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (b + i < n) k[i] = w[i];
        }
      }
      fn(b);
    }
    loaded = true;
  };
  auto clear = [&] {
    reinterpret_cast<uint4*>(sh.hist)[tid] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(sh.hist)[tid + kSelThreads] = make_uint4(0, 0, 0, 0);
  };
  static_assert(kBins == 8 * kSelThreads, "histogram");
  // ---- how many are free to choose from, and their range
  uint32_t ntaken = 0, nfree = 0, kmin = 0xFFFFFFFFu, kmax = 0, most = 0;
  if (!every) {
    clear();
    if (tid == 0) sh.count = 0;
    uint32_t counts = 0;                 // taken << 16 | free (18,432 at most)
    for (int i = lane; i < ranks * kSelWarps; i += 32) {
      const uint4 v = sh.seen[i];
      most = max(most, v.x);
      kmin = min(kmin, v.y);
      kmax = max(kmax, v.z);
      counts += v.w;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    counts = __reduce_add_sync(0xffffffffu, counts);
    ntaken = counts >> 16;
    nfree = counts & 0xFFFFu;
    __syncthreads();
  }
  const uint32_t want = min(nfree, p.nsel > (int)ntaken ? p.nsel - ntaken : 0u);
  uint32_t in_from = 0;                  // keys from here on are in, but for near ones
  float low = 0.f, top = 0.f;
  bool all = false;                      // every score is near
  if (want == 0) {
    in_from = kTaken;
  } else if (want < nfree) {
    // ---- how far a float32 score may be off: its roundings' sum |q| |bound|, the
    // sums over G heads (all of one sign), 8 products and sums of a lane, 5 of the
    // reduction, 2^-24 each; e is twice that and more.  The exact want-th largest
    // score is within half of e of the one found in float32, so a score beyond that
    // by more than e (and a sixteenth, for the roundings here) is decided; the others
    // are near.
    const float e = (float)(16 + p.group) * 0x1p-23f * q1 * __uint_as_float(most << 16) + 1e-40f;
    all = most >= 0x7F80u || !(e < INFINITY);
    bool decided = false, listed = false;  // no near one to tell; the near ones are in near_i
    // ---- the want-th largest key
    const uint32_t differ = kmin ^ kmax;
    int shift = differ ? 32 - __clz(differ) : 0;         // bits that are not the same in all
    uint32_t prefix = shift == 32 ? 0u : kmin >> shift << shift;
    const uint32_t first_high = shift == 32 ? 0u : ~0u << shift;
    uint32_t rest = want;
    while (shift > 0) {
      const int bits = min(shift, 11);
      const uint32_t high = shift == 32 ? 0u : ~0u << shift;
      shift -= bits;
      rounds([&](int) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (is_score(k[i]) && (k[i] & high) == prefix)
            atomicAdd(&sh.hist[(k[i] >> shift) & ((1u << bits) - 1)], 1u);
      });
      __syncthreads();
      // thread t: the eight bins from 2047 - 8 t down
      const uint4 u = reinterpret_cast<const uint4*>(sh.hist)[kBins / 4 - 1 - 2 * tid];
      const uint4 v = reinterpret_cast<const uint4*>(sh.hist)[kBins / 4 - 2 - 2 * tid];
      const uint32_t c[8] = {u.w, u.z, u.y, u.x, v.w, v.z, v.y, v.x};
      uint32_t sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i];
      uint32_t total, above = sel_prefix(sum, sh.warp_s, total);
      if (above < rest && rest <= above + sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < rest && rest <= above + c[i]) {
            sh.pick[0] = kBins - 1 - 8 * tid - i;
            sh.pick[1] = rest - above;
            sh.pick[2] = c[i];
          }
          above += c[i];
        }
      }
      __syncthreads();
      const int bin = (int)same_in_warp(sh.pick[0]);
      prefix |= (uint32_t)bin << shift;
      rest = same_in_warp(sh.pick[1]);
      const uint32_t same = same_in_warp(sh.pick[2]);
      // Few keys in the border's bin and the two beside it, and the near ones among
      // them: one warp settles it.
      const uint32_t up = bin + 1 < kBins ? same_in_warp(sh.hist[bin + 1]) : 0u;
      const uint32_t down = bin > 0 ? same_in_warp(sh.hist[bin - 1]) : 0u;
      if (high == first_high && shift > 0 && !all && same + up + down <= 32) {
        rounds([&](int b) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (int)((k[i] >> shift) & (kBins - 1)) - bin;
            if (is_score(k[i]) && at >= -1 && at <= 1) {
              const uint32_t to = atomicAdd(&sh.count, 1u);
              sh.near_k[to] = k[i];
              sh.near_i[to] = b + i;
            }
          }
        });
        __syncthreads();
        if (warp == 0) {
          const uint32_t cnt = same + up + down, nth = rest + up;
          const bool there = (uint32_t)lane < cnt;
          const uint32_t mine = there ? (uint32_t)sh.near_k[lane] : 0u;
          const int block = there ? sh.near_i[lane] : 0;
          uint32_t more = 0, equal = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {       // (0 behind the last: below every key)
            const uint32_t other = __shfl_sync(0xffffffffu, mine, i);
            more += other > mine;
            equal += other == mine;
          }
          const unsigned who =
              __ballot_sync(0xffffffffu, there && more < nth && nth <= more + equal);
          const uint32_t border = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
          const float at = value32(border), s = value32(mine);
          const float t = at + 1.0625f * e, l = at - 1.0625f * e;
          const uint32_t in = __popc(__ballot_sync(0xffffffffu, there && s > t));
          const bool is_near = there && s <= t && s >= l;
          const unsigned nears = __ballot_sync(0xffffffffu, is_near);
          // (bins beyond the first and the last of the range are empty)
          const uint32_t edge = prefix;
          const bool inside = (bin == 0 || order32(l) >= edge - (1u << shift)) &&
                              (bin == kBins - 1 || order32(t) - edge < (2u << shift));
          if (is_near) sh.near_i[__popc(nears & ((1u << lane) - 1))] = block;
          if (lane == 0) {
            const bool plain = (uint32_t)__popc(nears) == nth - in;
            sh.border = border;
            sh.pick[0] = !inside ? 0u : plain ? 1u : 2u;
            sh.pick[1] = plain ? order32(l) : order32(t) + 1;
            sh.pick[2] = nth - in;
            sh.count = inside ? __popc(nears) : 0;
          }
        } else if (warp >= kSelWarps / 2) {
          sum_heads64(q, p.group, tid - kSelThreads / 2, sh);   // in case; the histogram is read
        }
        __syncthreads();
        const uint32_t how = same_in_warp(sh.pick[0]);
        prefix = sh.border;
        decided = how == 1;
        listed = how == 2;
        in_from = sh.pick[1];
        break;
      }
      if (shift > 0 && same <= kNear) {
        // few share the leading bits: the rest-th largest of them directly
        const uint32_t lead = ~0u << shift;
        rounds([&](int) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (is_score(k[i]) && (k[i] & lead) == prefix)
              sh.near_k[atomicAdd(&sh.count, 1u)] = k[i];
        });
        __syncthreads();
        if (tid < (int)same) {
          const uint32_t mine = (uint32_t)sh.near_k[tid];
          uint32_t more = 0, equal = 0;
#pragma unroll 4
          for (uint32_t i = 0; i < same; ++i) {
            const uint32_t other = (uint32_t)sh.near_k[i];
            more += other > mine;
            equal += other == mine;
          }
          if (more < rest && rest <= more + equal) sh.border = mine;
        }
        __syncthreads();
        prefix = sh.border;
        break;
      }
      if (shift > 0) {
        clear();
        __syncthreads();
      }
    }
    // ---- else who is in, who is out, and who is too near to tell
    const float at = value32(prefix);
    top = at + 1.0625f * e;
    low = at - 1.0625f * e;
    auto is_near = [&](uint32_t x) {
      if (!is_score(x)) return false;
      const float s = value32(x);
      return all || (s >= low && s <= top);
    };
    // the first `need` of the near ones in near_i, by their exact scores
    auto settle = [&](uint32_t near, uint32_t need) {
      for (uint32_t i = warp; i < near; i += kSelWarps) {
        const uint4 w = bound_load(run, bound_at(p, run, g, sh.near_i[i]), lane);
        const double s = score64(sh, w, lane);
        if (lane == 0) sh.near_k[i] = order64(s);
      }
      __syncthreads();
      if (tid < (int)near) {
        const uint64_t mine = sh.near_k[tid];
        const int b = sh.near_i[tid];
        uint32_t before = 0;
        for (uint32_t i = 0; i < near; ++i)
          before += sh.near_k[i] > mine || (sh.near_k[i] == mine && sh.near_i[i] < b);
        if (before < need) key32[b] = kTaken;
      }
    };
    uint32_t both = 0;                   // in << 16 | near
    if (!decided && !listed) rounds([&](int) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        both += is_near(k[i]) ? 1u : is_score(k[i]) && value32(k[i]) > top ? 0x10000u : 0u;
    });
    uint32_t total = want << 16;
    if (!decided && !listed) sel_prefix(both, sh.warp_s, total);
    total = same_in_warp(total);
    const uint32_t near = total & 0xFFFFu, need = want - (total >> 16);
    if (decided) {
      // in_from says it
    } else if (listed) {
      settle(same_in_warp(sh.count), sh.pick[2]);
      __syncthreads();
      loaded = false;                    // the near ones that are in say so now
    } else if (near == need) {
      in_from = order32(low);
    } else {
      // ---- the near ones' exact scores
      if (tid < 128) sum_heads64(q, p.group, tid, sh);
      if (tid == 0) sh.count = 0;
      __syncthreads();
      if (near <= kNear) {
        rounds([&](int b) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (is_near(k[i])) {
              sh.near_i[atomicAdd(&sh.count, 1u)] = b + i;
              key32[b + i] = kAbsent;
            } else if (is_score(k[i])) {
              key32[b + i] = value32(k[i]) > top ? kTaken : kAbsent;
            }
          }
        });
        __syncthreads();
        settle(near, need);
      } else {
        // many (equal blocks, scores that are no numbers): the need-th largest of
        // their exact keys, 8 bits at a time
        for (int b = warp; b < n; b += kSelWarps) {
          const uint32_t x = key32[b];
          const bool mine = is_near(x);
          uint64_t exact = 0;            // 0 marks a block that is not near
          if (mine) {
            const uint4 w = bound_load(run, bound_at(p, run, g, b), lane);
            exact = max(order64(score64(sh, w, lane)), (uint64_t)1);
          }
          __syncwarp();
          if (lane == 0) {
            key64[b] = exact;
            if (!mine && is_score(x)) key32[b] = value32(x) > top ? kTaken : kAbsent;
          }
        }
        uint64_t prefix64 = 0;
        uint32_t left = need;
        for (int shift64 = 56; shift64 >= 0; shift64 -= 8) {
          __syncthreads();
          sh.hist[tid] = 0;
          __syncthreads();
          for (int b = tid; b < n; b += kSelThreads) {
            const uint64_t x = key64[b];
            if (x && (shift64 == 56 || (x >> (shift64 + 8)) == (prefix64 >> (shift64 + 8))))
              atomicAdd(&sh.hist[(x >> shift64) & 255], 1u);
          }
          __syncthreads();
          const uint32_t c = sh.hist[255 - tid];
          uint32_t sum;
          const uint32_t above = sel_prefix(c, sh.warp_s, sum);
          if (above < left && left <= above + c) {
            sh.pick[0] = 255 - tid;
            sh.pick[1] = left - above;
          }
          __syncthreads();
          prefix64 |= (uint64_t)sh.pick[0] << shift64;
          left = sh.pick[1];
        }
        // those above the need-th, and of the ones equal to it the first `left`
        uint32_t seen = 0;
        for (int b0 = 0; b0 < n; b0 += kSelThreads) {
          const int b = b0 + tid;
          const uint64_t x = b < n ? key64[b] : 0;
          uint32_t sum;
          const uint32_t before = seen + sel_prefix(x == prefix64, sh.warp_s, sum);
          if (x) key32[b] = x > prefix64 || (x == prefix64 && before < left) ? kTaken : kAbsent;
          seen += sum;
        }
      }
      __syncthreads();
      loaded = false;                    // the keys say it all now
      in_from = kTaken;
    }
  }
  // ---- the chosen blocks, ascending.  (Every key but kAbsent is at least 1.)
  in_from = max(in_from, 1u);
  uint32_t filled = 0;
  rounds([&](int b) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += k[i] >= in_from;
    uint32_t total, at = filled + sel_prefix(mine, sh.warp_s, total);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k[i] >= in_from) out[at++] = b + i;
    filled += total;
  });
  for (uint32_t i = filled + tid; i < (uint32_t)p.nsel; i += kSelThreads) out[i] = -1;
}

// R: rows of a cluster at most.  The grid: clusters of p.cluster CTAs, one for
// each (row group, kv head).
template <int R>
__global__ void __launch_bounds__(kSelThreads, R == 1 ? 4 : 2)
    select_blocks_kernel(const __grid_constant__ SelectParams p) {
  __shared__ SelShared sh;
  extern __shared__ uint64_t dyn[];          // [cap] exact keys, then [cap] keys
  uint64_t* key64 = dyn;
  uint32_t* key32 = reinterpret_cast<uint32_t*>(dyn + p.cap);
  const int nc = p.cluster;
  if (nc > 1) cluster_arrive();              // every CTA has to run before its memory is written
  allow_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)same_in_warp((uint32_t)tid >> 5);
  const int rank = nc > 1 ? (int)cluster_ctarank() : 0;
  const int item = blockIdx.x / nc, g = item % p.hkv, group = item / p.hkv;
  const SelRun& run = p.runs[run_holding(p.runs, p.nruns, &SelRun::group0, group)];
  const int in_run = (group - run.group0) * R;           // first row of the group, in its run
  const int rows = min(R, run.nrows - in_run);
  const int row0 = run.row0 + in_run, pos0 = run.pos0 + in_run;
  const int n = (pos0 + rows - 1) / p.block + 1;         // blocks that its last row sees
  const bool every = n <= p.nsel;                        // every block is in: no scores
  const bool waits = nc > 1;
  float qf[R][8];
  if (every) {
    if (rank < rows) {
      const int last = (pos0 + rank) / p.block;
      for (int b = tid; b <= last; b += kSelThreads) {
        const bool there = bound_at(p, run, g, b) >= 0;
        if (!there) flag_error(p.err_flag, kErrBadPage);
        key32[b] = there ? kTaken : kAbsent;
      }
    }
  } else {
    // ---- this CTA's blocks, eight a warp and step
    const int chunk = ((n + nc - 1) / nc + 7) & ~7;
    const int lo = min(n, rank * chunk), hi = min(n, lo + chunk);
    uint32_t most = 0;
    uint32_t kmin = 0xFFFFFFFFu, kmax = 0, counts = 0;     // of this lane's row
    bool nonfinite = false, may_write = !waits;
    auto find = [&](int b) { return b < hi ? bound_at(p, run, g, b) : -1; };
    int b0 = lo + warp * 8;
    int at = find(b0 + (lane & 7));
    uint4 w[8];
    auto load = [&] {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int a = __shfl_sync(0xffffffffu, at, j);
        w[j] = a >= 0 ? bound_load(run, a, lane) : make_uint4(0, 0, 0, 0);
      }
    };
    load();                                  // under way while the queries are summed
    // ---- the query heads' negative parts (threads 0-127) and positive ones,
    // summed: a head dim a thread, four heads of all rows on their way at once
    static_assert(kSelThreads == 256, "a thread a sum");
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] = 0.f;
    const __nv_bfloat16* qp =
        p.q + ((size_t)row0 * p.hq + (size_t)g * p.group) * kHeadDim + (tid & 127);
    for (int h0 = 0; h0 < p.group; h0 += 4) {
      float x[R][4];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          x[r][h] = r < rows && h0 + h < p.group
                        ? __bfloat162float(qp[((size_t)r * p.hq + h0 + h) * kHeadDim])
                        : 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          sum[r] += tid < 128 ? (x[r][h] > 0.f ? 0.f : x[r][h]) : (x[r][h] < 0.f ? 0.f : x[r][h]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) sh.q32[r][tid] = sum[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 u = *reinterpret_cast<const float4*>(&sh.q32[r < rows ? r : 0][lane * 8]);
      const float4 v = *reinterpret_cast<const float4*>(&sh.q32[r < rows ? r : 0][lane * 8 + 4]);
      qf[r][0] = u.x; qf[r][1] = u.y; qf[r][2] = u.z; qf[r][3] = u.w;
      qf[r][4] = v.x; qf[r][5] = v.y; qf[r][6] = v.z; qf[r][7] = v.w;
    }
    for (; b0 < hi; b0 += kSelWarps * 8) {
      const int here = __shfl_sync(0xffffffffu, at, lane >> 2);   // the block this lane answers for
      at = find(b0 + kSelWarps * 8 + (lane & 7));
      float s[R][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[8];
        unpack8(w[j], x);
        most = __vmaxu2(most, w[j].x & 0x7FFF7FFFu);
        most = __vmaxu2(most, w[j].y & 0x7FFF7FFFu);
        most = __vmaxu2(most, w[j].z & 0x7FFF7FFFu);
        most = __vmaxu2(most, w[j].w & 0x7FFF7FFFu);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r][j] = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s[r][j] = fmaf(qf[r][i], x[i], s[r][j]);
        }
      }
      const int b = b0 + (lane >> 2);
      float mine = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float v = reduce8(s[r], lane);
        if ((lane & 3) == r) mine = v;
      }
      load();
      const int r = lane & 3;                            // and the row
      if (!may_write) {
        __syncwarp();
        cluster_wait();
        may_write = true;
      }
      if (r < rows && b < hi) {
        const int last = (pos0 + r) / p.block;
        if (b <= last) {
          uint32_t key;
          if (here < 0) {
            key = kAbsent;
            flag_error(p.err_flag, kErrBadPage);
          } else if (b < p.sink || b > last - p.recent) {
            key = kTaken;
            counts += 0x10000u;
          } else {
            const bool number = fabsf(mine) < INFINITY;
            nonfinite |= !number;
            key = order32(number ? mine : 0.f);
            kmin = min(kmin, key);
            kmax = max(kmax, key);
            ++counts;
          }
          if (waits)
            st_cluster_u32(mapa_shared(smem_u32(key32 + b), r), key);
          else
            key32[b] = key;
        }
      }
    }
    __syncwarp();
    if (!may_write) cluster_wait();
    most = max(most & 0xFFFFu, most >> 16);
    most = __reduce_max_sync(0xffffffffu, nonfinite ? 0xFFFFu : most);
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {        // the lanes of one row
      kmin = min(kmin, __shfl_xor_sync(0xffffffffu, kmin, d));
      kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, d));
      counts += __shfl_xor_sync(0xffffffffu, counts, d);
    }
    if (lane < rows) {
      uint4* slot = &sh.seen[rank * kSelWarps + warp];
      if (waits)
        st_cluster128(mapa_shared(smem_u32(slot), lane), most, kmin, kmax, counts);
      else
        *slot = make_uint4(most, kmin, kmax, counts);
    }
  }
  __syncwarp();
  if (waits) {
    if (every) cluster_wait();
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (rank >= rows) return;
  // ---- this CTA's row
  float q1 = 0.f;
  if (!every) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r == rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q1 += fabsf(qf[r][i]);
      }
#pragma unroll
    for (int d = 16; d; d >>= 1) q1 += __shfl_xor_sync(0xffffffffu, q1, d);
  }
  const int row = row0 + rank;
  choose(p, run, p.q + ((size_t)row * p.hq + (size_t)g * p.group) * kHeadDim, g,
         (pos0 + rank) / p.block + 1, every, nc, q1, key32, key64, sh,
         p.blocks + ((size_t)row * p.hkv + g) * p.nsel);
}

template <int R>
cudaError_t launch_select(const SelectParams& p, cudaStream_t s) {
  static PerDeviceOnce configured;
  const cudaError_t e = configured.run([] {
    return cudaFuncSetAttribute(select_blocks_kernel<R>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(select_blocks_kernel<R>, dim3(p.groups * p.hkv * p.cluster),
                            dim3(kSelThreads), (size_t)p.cap * 12, s, p, p.cluster);
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
  return p.rows_per == 1   ? launch_select<1>(p, s)
         : p.rows_per == 2 ? launch_select<2>(p, s)
                           : launch_select<4>(p, s);
}

}  // namespace tfpa
