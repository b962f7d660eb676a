// C-ABI entry points: argument checks, row grouping, slicing, TMA
// descriptors and launches.  No allocation, no stream synchronisation.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <cmath>
#include <cstring>
#include <unordered_map>
#include <vector>

#include "params.h"
#include "tfpa.h"

using namespace tfpa;

namespace {

// ------------------------------------------------------------ launch hook
// Set from one thread while no other call runs (a test facility); read by
// every call without a lock.
std::atomic<tfpa_launch_hook> g_hook_fn{nullptr};
std::atomic<void*> g_hook_user{nullptr};
std::atomic<int> g_hook_dry{0};

bool dry_run() {
  return g_hook_dry.load(std::memory_order_relaxed) != 0 &&
         g_hook_fn.load(std::memory_order_relaxed) != nullptr;
}

void record(int kind, int row0, int rows, int runs, int items, int grid, int64_t qoff,
            int64_t ooff) {
  const tfpa_launch_hook fn = g_hook_fn.load(std::memory_order_acquire);
  if (!fn) return;
  tfpa_launch_record r;
  r.kind = kind;
  r.row0 = row0;
  r.rows = rows;
  r.runs = runs;
  r.items = items;
  r.grid = grid;
  r.q_offset = qoff;
  r.out_offset = ooff;
  fn(&r, g_hook_user.load(std::memory_order_relaxed));
}

// ------------------------------------------------------------ device info
// SM count and compute capability of each device, read once per device.
struct DeviceInfo {
  std::atomic<int> ready{0};
  int sm_count = 0;
  int major = 0;
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];

// The current device's info, or nullptr if a CUDA call fails.
const DeviceInfo* device_info() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  DeviceInfo& d = g_dev[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    int n = 0, major = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
      return nullptr;
    d.sm_count = n;     // two threads may both get here: they store the same values
    d.major = major;
    d.ready.store(1, std::memory_order_release);
  }
  return &d;
}

int sm_count() {
  if (dry_run()) return 152;
  const DeviceInfo* d = device_info();
  return d ? d->sm_count : 0;
}

int check_device() {
  if (dry_run()) return TFPA_OK;
  const DeviceInfo* d = device_info();
  if (!d) return TFPA_ECUDA;
  return d->major == 10 ? TFPA_OK : TFPA_EDEVICE;
}

// ------------------------------------------------------------ tensor maps
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

struct MapKey {
  const void* ptr;
  uint64_t rows;
  int fp8, box_inner, box_rows;
  bool operator==(const MapKey& o) const {
    return ptr == o.ptr && rows == o.rows && fp8 == o.fp8 && box_inner == o.box_inner &&
           box_rows == o.box_rows;
  }
};
struct MapKeyHash {
  size_t operator()(const MapKey& k) const {
    size_t h = std::hash<const void*>()(k.ptr);
    h ^= std::hash<uint64_t>()(k.rows) + 0x9e3779b97f4a7c15ull + (h << 6) + (h >> 2);
    h ^= (size_t)(k.fp8 * 131 + k.box_inner * 7 + k.box_rows);
    return h;
  }
};
// Each host thread keeps its own cache of encoded maps, so calls from
// several threads share no lock.  A map only describes an address range and
// a box, so it stays valid for any buffer later placed at the same address
// with the same extent.
thread_local std::unordered_map<MapKey, CUtensorMap, MapKeyHash> t_maps;

// A 2D view [rows][128] of a K or V buffer, 128B swizzle, box
// [box_inner elements][box_rows rows].
int get_map(const void* ptr, uint64_t rows, bool fp8, int box_inner, int box_rows,
            CUtensorMap* out) {
  if (dry_run()) {
    std::memset(out, 0, sizeof(*out));
    return TFPA_OK;
  }
  MapKey key{ptr, rows, fp8 ? 1 : 0, box_inner, box_rows};
  auto it = t_maps.find(key);
  if (it != t_maps.end()) {
    *out = it->second;
    return TFPA_OK;
  }
  auto fn = encode_fn();
  if (!fn) return TFPA_ECUDA;
  const uint64_t esz = fp8 ? 1 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(kHeadDim * esz)};
  cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUtensorMap m;
  CUresult r = fn(&m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return TFPA_ECUDA;
  if (t_maps.size() > 4096) t_maps.clear();
  t_maps.emplace(key, m);
  *out = m;
  return TFPA_OK;
}

// q of one launch as a 3D tensor [rows][hq][128] bf16, 128B swizzle; box
// 64 x 1 x 128 (prefill: one head's 128-row tile, half the head dim) or
// 64 x G x 128 / G (verify: a kv head's query vectors of 128 / G rows).
int get_qmap(const void* q, int hq, int rows, int box_heads, int box_rows, CUtensorMap* out) {
  if (dry_run()) {
    std::memset(out, 0, sizeof(*out));
    return TFPA_OK;
  }
  auto fn = encode_fn();
  if (!fn) return TFPA_ECUDA;
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)hq, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)hq * kHeadDim * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TFPA_OK : TFPA_ECUDA;
}

// ------------------------------------------------------------ validation
// Q tiles of the prompt and verify paths are loaded by TMA, from device (or
// managed) memory only: pinned host memory, which the decode path takes for
// q, is refused for them before anything is enqueued.
int check_tma_source(const void* q) {
  if (dry_run()) return TFPA_OK;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, q) != cudaSuccess) {
    cudaGetLastError();   // the failed query's error stays with this call
    return TFPA_EINVAL;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged ? TFPA_OK
                                                                              : TFPA_EINVAL;
}

int32_t pages_of(int32_t L) { return L / kPage + (L % kPage != 0); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache(const tfpa_cache* c) {
  if (!c) return TFPA_EINVAL;
  if (c->dtype != TFPA_BF16 && c->dtype != TFPA_FP8_E4M3 && c->dtype != TFPA_FP4_E2M1)
    return TFPA_EINVAL;
  if (c->head_dim != kHeadDim || c->hkv < 1 || c->hq < 1 || c->hq % c->hkv) return TFPA_EINVAL;
  if (c->dtype != TFPA_BF16 && (!c->k_scale || !c->v_scale)) return TFPA_EINVAL;
  if ((c->k_pool && !aligned(c->k_pool, 16)) || (c->v_pool && !aligned(c->v_pool, 16)))
    return TFPA_EINVAL;
  return TFPA_OK;
}

int check_segs(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg) {
  if (nseg < 0 || (nseg > 0 && !segs)) return TFPA_EINVAL;
  for (int32_t s = 0; s < nseg; ++s) {
    const tfpa_seg& g = segs[s];
    if (g.seq_len < 1) return TFPA_EINVAL;
    if (g.page_table) {
      if (!c->k_pool || !c->v_pool || c->num_pages < 1) return TFPA_EINVAL;
      if ((int64_t)c->num_pages * c->hkv * kPage > INT32_MAX) return TFPA_EINVAL;
      if (g.page_table_host) {
        const int32_t n = pages_of(g.seq_len);
        for (int32_t i = 0; i < n; ++i)
          if (g.page_table_host[i] < 0 || g.page_table_host[i] >= c->num_pages)
            return TFPA_ERANGE;
      }
    } else {
      if (!g.k_slab || !g.v_slab) return TFPA_EINVAL;
      if (!aligned(g.k_slab, 16) || !aligned(g.v_slab, 16)) return TFPA_EINVAL;
      // (a multiple of the page, so it holds the stream's last page whole)
      if (g.slab_cap % kPage || g.slab_cap < g.seq_len) return TFPA_EINVAL;
      if ((int64_t)c->hkv * g.slab_cap > INT32_MAX) return TFPA_EINVAL;
    }
  }
  return TFPA_OK;
}

// A run: consecutive rows of one segment at consecutive positions.
struct Run {
  int32_t seg, row0, nrows, pos0;
};

int build_runs(const tfpa_seg* segs, int32_t nseg, const int32_t* row_seg,
               const int32_t* row_pos, int32_t rows, std::vector<Run>& out) {
  out.clear();
  if (rows < 0 || (rows > 0 && (!row_seg || !row_pos))) return TFPA_EINVAL;
  for (int32_t r = 0; r < rows;) {
    const int32_t s = row_seg[r], p = row_pos[r];
    if (s < 0 || s >= nseg) return TFPA_ERANGE;
    if (p < 0 || p >= segs[s].seq_len) return TFPA_ERANGE;
    // the rows that go on from this one, within the segment
    const int32_t most = std::min(rows - r, segs[s].seq_len - p);
    // blocks without an exit, which the compiler vectorises (32,768 rows: 6 us in
    // blocks of 64, 12 in blocks of 16 alone)
    int32_t n = 1;
    const auto differs = [&](int32_t m) {
      int32_t differ = 0;
      for (int32_t i = 0; i < m; ++i)
        differ |= (row_seg[r + n + i] ^ s) | (row_pos[r + n + i] ^ (p + n + i));
      return differ != 0;
    };
    if (most > 1 && !differs(1)) {
      while (n + 64 <= most && !differs(64)) n += 64;
      while (n + 16 <= most && !differs(16)) n += 16;
    }
    while (n < most && row_seg[r + n] == s && row_pos[r + n] == p + n) ++n;
    out.push_back(Run{s, r, n, p});
    r += n;
  }
  return TFPA_OK;
}

// Runs of four or more m-tiles (16 query vectors each, so at least 49
// vectors per kv head) are dense enough for the tensor cores: they take the
// prefill kernel in verify mode, when a tile holds the group's heads.
// Over a 4-bit cache, whose decode kernel spends most of its time on turning
// codes into operands, already runs of two or more (more than 16 vectors: 8
// streams of 65,536 keys, 20 vectors, 265 us on tiles and 330 us as items).
constexpr int kFp4VerifyVectors = 16;
bool on_verify_path(const Run& r, int G, int kv) {
  if (kv == kKvFp4) return G <= kVerifyVectors && r.nrows * G > kFp4VerifyVectors;
  return G <= kVerifyVectors && (r.nrows * G + 15) / 16 >= 4;
}

// Stored bytes of one row of one kv head, K or V.
int row_bytes_of(const tfpa_cache* c) {
  return c->dtype == TFPA_BF16       ? 2 * kHeadDim
         : c->dtype == TFPA_FP8_E4M3 ? kHeadDim
                                     : kFp4CodeBytes + kFp4ScaleBytes;
}

// A C entry's work; host memory that runs out (for a call's row groups, a
// plan's launches, a map) is an error code, not an exception.
template <typename F>
int no_throw(F&& fn) {
  try {
    return fn();
  } catch (const std::bad_alloc&) {
    return TFPA_ENOMEM;
  }
}

// Runs of more than eight query vectors per kv head over a 4-bit cache take
// the decode kernel of 16-vector items, the others that of eight (8 streams of
// 65,536 keys: 16 vectors 161 us in one item, 240 us as two of eight; eight
// vectors 123 us in an item of eight, 165 us in one of 16).
bool on_wide_path(const Run& r, int G, int kv) { return kv == kKvFp4 && r.nrows * G > 8; }

int to_err(cudaError_t e) { return e == cudaSuccess ? TFPA_OK : TFPA_ECUDA; }

}  // namespace

// A call's launches, planned and kept by value for a later tfpa_plan_launch.
// In device mode (dyn_base set) each decode, merge and write launch owns a
// 16-byte aligned slot of the caller's device buffer at dyn_base, from which
// it reads its dynamic data; the plan keeps the host image in the launch's
// parameters (`d`) for tfpa_plan_dyn_pack.
struct tfpa_plan {
  enum Kind : int { kDecode, kVerify, kMerge, kWrite };
  struct Entry {
    Kind kind;
    int kv;         // KvType
    int grid;
    size_t index;   // into the vector of its kind
  };
  std::vector<Entry> entries;
  std::vector<DecodeParams> decode;
  std::vector<PrefillParams> verify;
  std::vector<MergeParams> merge;
  std::vector<WriteParams> write;
  uint8_t* dyn_base = nullptr;   // DEVICE, or nullptr: parameter mode
  size_t dyn_cap = 0;
  size_t dyn_used = 0;           // bytes of dyn_base handed out
  cudaGraphExec_t exec = nullptr;   // tfpa_plan_capture's graph
  uint64_t exec_shape = 0;          // the plan's shape when it was captured
  uint64_t shape = 0;               // the shape of the launches held now
  bool captured = false;
  ~tfpa_plan() {
    if (exec) cudaGraphExecDestroy(exec);
  }
};

namespace {

// Where a call's launches go: enqueued on a stream now, or appended to a
// plan.  A planning call that fails takes back what it appended (Mark).
struct Sink {
  cudaStream_t stream = nullptr;
  tfpa_plan* plan = nullptr;
  struct Mark {
    size_t e, d, v, m, w, dyn;
  };
  // Device mode: launch shapes must not depend on the streams' lengths.
  bool device() const { return plan && plan->dyn_base; }
  Mark mark() const {
    return plan ? Mark{plan->entries.size(), plan->decode.size(), plan->verify.size(),
                       plan->merge.size(), plan->write.size(), plan->dyn_used}
                : Mark{0, 0, 0, 0, 0, 0};
  }
  void rollback(const Mark& k) const {
    if (!plan) return;
    plan->entries.resize(k.e);
    plan->decode.resize(k.d);
    plan->verify.resize(k.v);
    plan->merge.resize(k.m);
    plan->write.resize(k.w);
    plan->dyn_used = k.dyn;
  }
  template <typename P>
  int keep(tfpa_plan::Kind kind, std::vector<P>& v, const P& p, int kv, int grid) const {
    v.push_back(p);
    plan->entries.push_back(tfpa_plan::Entry{kind, kv, grid, v.size() - 1});
    return TFPA_OK;
  }
  // keep() for a launch with dynamic data: in device mode the launch takes
  // the next slot of the plan's device buffer.
  template <typename P>
  int keep_dyn(tfpa_plan::Kind kind, std::vector<P>& v, const P& p, int kv, int grid) const {
    const size_t off = plan->dyn_used;
    if (plan->dyn_base) {
      const size_t end = (off + sizeof(p.d) + 15) & ~size_t(15);
      if (end > plan->dyn_cap) return TFPA_ECAPACITY;
      plan->dyn_used = end;
    }
    keep(kind, v, p, kv, grid);
    v.back().dyn = plan->dyn_base
                       ? reinterpret_cast<decltype(p.dyn)>(plan->dyn_base + off)
                       : nullptr;
    return TFPA_OK;
  }
  int decode(const DecodeParams& p, int kv, int grid) const {
    if (plan) return keep_dyn(tfpa_plan::kDecode, plan->decode, p, kv, grid);
    return dry_run() ? TFPA_OK : to_err(launch_decode_partial(p, kv, grid, stream));
  }
  int verify(const PrefillParams& p, int kv, int tiles) const {
    // the tensor-core verify launch's grid follows the streams' lengths
    if (device()) return TFPA_EINVAL;
    if (plan) return keep(tfpa_plan::kVerify, plan->verify, p, kv, tiles);
    return dry_run() ? TFPA_OK : to_err(launch_verify(p, kv, tiles, stream));
  }
  int merge(const MergeParams& p) const {
    if (plan) return keep_dyn(tfpa_plan::kMerge, plan->merge, p, 0, 0);
    return dry_run() ? TFPA_OK : to_err(launch_merge(p, stream));
  }
  int write(const WriteParams& p) const {
    if (plan) return keep_dyn(tfpa_plan::kWrite, plan->write, p, 0, 0);
    return dry_run() ? TFPA_OK : to_err(launch_write_kv(p, stream));
  }
};

}  // namespace

// One page per split up to 16 pages (a short stream's keys spread over as
// many CTAs as it has pages), then at least two.
extern "C" int32_t tfpa_pages_per_split(int32_t seq_len) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  if (np <= 16) return 1;
  return std::max<int32_t>(2, (np + kMaxSplits - 1) / kMaxSplits);
}

extern "C" int32_t tfpa_num_splits(int32_t seq_len) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  const int32_t pps = tfpa_pages_per_split(seq_len);
  return (np + pps - 1) / pps;
}

namespace {

// Splits of a run on the tensor-core verify path: at least 24 pages and at
// most 7 a stream.  A verify tile carries a fixed cost (set-up, its first
// loads, a cold first softmax step and the epilogue: about a quarter of a
// 24-page tile), so a long stream takes a few long tiles.  A function of the
// stream's length only, like the decode splits, so a stream's bytes do not
// depend on its batch.  On 65,536-key streams (7 splits of 37 pages), 8
// streams x 8 kv heads make 448 tiles, 2.95 waves of 152 SMs; 16-node trees
// took 294 / 345 us (e4m3 / bf16 cache) with 11 splits of 24 pages, 279 /
// 331 with 9 of 29, 263 / 325 with 7 of 37 and 295 / 348 with 6 of 43.
// Other batches fill the waves differently.  Never more splits than the
// decode path's, so a scratch sized for decode holds them.
// Over a 4-bit cache at least 16 pages: 16-node trees of 32,761 keys 218 us
// with six splits of 24 (384 tiles, 2.53 waves), 183 us with seven of 19.
int32_t verify_pages_per_split(int32_t seq_len, int kv) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  return std::max<int32_t>(kv == kKvFp4 ? 16 : 24, (np + 6) / 7);
}
int32_t verify_num_splits(int32_t seq_len, int kv) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  const int32_t pps = verify_pages_per_split(seq_len, kv);
  return (np + pps - 1) / pps;
}

// Splits of a run of a 4-bit cache.  An item's end (sixteen warps' states
// handed over and folded) costs as much as about 500 of its keys, and a key
// arrives in half an e4m3 key's time, so the items are longer than the other
// types': at least four pages (two where fewer than eight kv heads make few
// items), and at most 16 (32) splits a stream.  A function of the stream's
// length and the cache's kv heads only; never more than tfpa_num_splits.
int32_t fp4_pages_per_split(int32_t seq_len, int32_t hkv) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  if (np <= 8) return 1;
  if (np <= 16) return 2;
  return hkv >= 8 ? std::max<int32_t>(4, (np + 15) / 16) : std::max<int32_t>(2, (np + 31) / 32);
}
int32_t fp4_num_splits(int32_t seq_len, int32_t hkv) {
  const int32_t np = pages_of(std::max(seq_len, 1));
  const int32_t pps = fp4_pages_per_split(seq_len, hkv);
  return (np + pps - 1) / pps;
}
// Splits of a run that the decode partial kernel takes.
int32_t decode_num_splits(int kv, int32_t seq_len, int32_t hkv) {
  return kv == kKvFp4 ? fp4_num_splits(seq_len, hkv) : tfpa_num_splits(seq_len);
}

// K/V sources of one launch: source 0 is the pool, 1.. are slab streams.
struct SourceSet {
  int slab_seg[kMaxSlabs];
  int nslab = 0;
  bool pool = false;
  // Source index for segment `s`, or -1 if the set is full.
  int add(const tfpa_seg* segs, int s) {
    if (segs[s].page_table) {
      pool = true;
      return 0;
    }
    for (int i = 0; i < nslab; ++i)
      if (slab_seg[i] == s) return i + 1;
    if (nslab == kMaxSlabs) return -1;
    slab_seg[nslab] = s;
    return ++nslab;
  }
};

int fill_maps(const tfpa_cache* c, const tfpa_seg* segs, const SourceSet& ss, bool fp8,
              int box_inner, int box_rows, KVMaps* maps, int32_t& nsrc) {
  int e;
  if (ss.pool) {
    const uint64_t rows = (uint64_t)c->num_pages * c->hkv * kPage;
    if ((e = get_map(c->k_pool, rows, fp8, box_inner, box_rows, &maps[0].k))) return e;
    if ((e = get_map(c->v_pool, rows, fp8, box_inner, box_rows, &maps[0].v))) return e;
  }
  for (int i = 0; i < ss.nslab; ++i) {
    const tfpa_seg& g = segs[ss.slab_seg[i]];
    const uint64_t rows = (uint64_t)c->hkv * g.slab_cap;
    if ((e = get_map(g.k_slab, rows, fp8, box_inner, box_rows, &maps[i + 1].k))) return e;
    if ((e = get_map(g.v_slab, rows, fp8, box_inner, box_rows, &maps[i + 1].v))) return e;
  }
  nsrc = 1 + ss.nslab;
  return TFPA_OK;
}

// Where each source's rows are: the pool, then the slabs in source order.
// Returns the number of sources.
template <typename P>
int32_t fill_bases(const tfpa_cache* c, const tfpa_seg* segs, const SourceSet& ss, P* k, P* v) {
  k[0] = c->k_pool;
  v[0] = c->v_pool;
  for (int i = 0; i < ss.nslab; ++i) {
    k[i + 1] = segs[ss.slab_seg[i]].k_slab;
    v[i + 1] = segs[ss.slab_seg[i]].v_slab;
  }
  return 1 + ss.nslab;
}

void fill_run(RunInfo& ri, const tfpa_seg& g, int src, int row0, int nrows, int pos0) {
  ri.page_table = g.page_table;
  ri.src = src;
  ri.seq_len = g.seq_len;
  ri.row0 = row0;
  ri.nrows = nrows;
  ri.pos0 = pos0;
  ri.nsplit = tfpa_num_splits(g.seq_len);
  ri.pps = tfpa_pages_per_split(g.seq_len);
  ri.item0 = 0;
  ri.slab_cap = g.page_table ? 0 : g.slab_cap;
  ri.pad_ = 0;
}

// Query vectors of a decode work item (an m-tile of the decode kernels).
int item_vectors(int kv) { return kv == kKvFp4 ? 8 : 16; }

// Key stages of decode work item (m-tile mt, split sigma) of a run: its
// split's keys, cut at the stream's end and at the last position of the
// item's rows (the kernel's item key range, in units of the kernel's chunk).
int item_stages(const RunInfo& ri, int G, int mt, int sigma, int chunk, int vecs) {
  const int nq = ri.nrows * G;
  const int last_qv = std::min(vecs * (mt + 1), nq) - 1;
  const int maxpos = ri.pos0 + last_qv / G;
  const int klo = sigma * ri.pps * kPage;
  const int khi = std::min(std::min(klo + ri.pps * kPage, ri.seq_len), maxpos + 1);
  return khi > klo ? (khi - klo + chunk - 1) / chunk : 0;
}

// Per-CTA item ranges of a decode partial launch, balanced by work: an item
// weighs its key stages plus a fixed cost (its query load and combine), and
// CTA b starts at the first item whose prefix weight reaches b / grid of the
// total.  Items are walked in the kernel's order: run, kv head, m-tile,
// split.  An item's weight does not depend on its kv head, so each run's
// (m-tile, split) prefix weights are computed once, and each CTA boundary is
// found by a binary search in the block of the kv head that holds it.
void plan_cta_ranges(DecodeParams& p, int nr, int G, int kv, int grid) {
  const int chunk = kv == kKvBf16 ? 128 : 256;
  const int vecs = item_vectors(kv);
  // The fixed cost, in key stages, was measured on the overcommitted pool
  // (17 streams of 1k-262k keys, e4m3): 0 -> 380 us, 1 -> 341 us, 2 -> 348 us,
  // 4 -> 377 us, 8 -> 444 us; uniform batches do not depend on it.  A 4-bit
  // item's end is nearer two stages (fp4_pages_per_split); others than 1 have
  // not been measured there.
  constexpr int64_t kItemCost = 1;
  thread_local std::vector<int64_t> cum;     // per run: 0, w0, w0 + w1, ...
  int32_t blk[kMaxRuns + 1];                 // run r's prefix weights: cum[blk[r] .. blk[r + 1]]
  cum.clear();
  int64_t total = 0;
  for (int r = 0; r < nr; ++r) {
    const RunInfo& ri = p.d.runs[r];
    const int mtiles = (ri.nrows * G + vecs - 1) / vecs;
    blk[r] = (int32_t)cum.size();
    int64_t sum = 0;
    cum.push_back(0);
    // splits fastest, or (4 bits) a split's m-tiles
    const bool by_split = kv == kKvFp4 || kv == kKvFp4Wide;
    const int n = mtiles * ri.nsplit, inner = by_split ? mtiles : ri.nsplit;
    for (int i = 0; i < n; ++i) {
      const int a = i / inner, b = i - a * inner;
      sum += item_stages(ri, G, by_split ? b : a, by_split ? a : b, chunk, vecs) + kItemCost;
      cum.push_back(sum);
    }
    total += sum * p.hkv;
  }
  blk[nr] = (int32_t)cum.size();
  int b = 1, item = 0;
  int64_t prefix = 0;   // weight of the items before the current block
  p.d.cta_item0[0] = 0;
  for (int r = 0; r < nr && b < grid; ++r) {
    const int64_t* c = cum.data() + blk[r];
    const int32_t n = blk[r + 1] - blk[r] - 1;   // items of one kv head's block
    for (int g = 0; g < p.hkv && b < grid; ++g) {
      // CTA b starts at the first item whose prefix weight P satisfies
      // P * grid >= total * b, i.e. P >= ceil(total * b / grid)
      while (b < grid) {
        const int64_t need = (total * b + grid - 1) / grid - prefix;
        const int32_t i = (int32_t)(std::lower_bound(c, c + n, need) - c);
        if (i >= n) break;
        p.d.cta_item0[b++] = item + i;
      }
      prefix += c[n];
      item += n;
    }
  }
  // CTAs past the last boundary get empty ranges at the end
  int n_items = 0;
  for (int r = 0; r < nr; ++r) n_items += (blk[r + 1] - blk[r] - 1) * p.hkv;
  while (b <= grid) p.d.cta_item0[b++] = n_items;
}

// Streams of at most this many splits (1,024 positions) are merged inside
// the partial kernel when the scratch has arrival counters.
constexpr int kFusedMergeMaxSplits = 4;

struct RopeArgs {
  const int32_t* pos;   // DEVICE [rows] or nullptr (the storage positions)
  const float* cos;     // DEVICE [n][64] or nullptr (plain store)
  const float* sin;
  int32_t n;
};
int write_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* k_rows,
               const void* v_rows, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
               const RopeArgs& rope, const Sink& sink, bool read = false);

// Partial (and optionally merge) launches over the call's rows.  With
// `sliced`, each launch's partials start at scratch row 0 and are merged
// before the next launch; otherwise partials land at the call's own row and
// no merge runs.
// With k_rows / v_rows (append), the rows' K and V are stored as well: by
// the decode partial kernel itself when every run takes it and no segment
// has two runs (a run's CTAs store the new rows they read before reading
// them), else by a KV write launch ahead of the decode launches.
int decode_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* q,
                const int32_t* row_seg, const int32_t* row_pos, const uint64_t* anc,
                int32_t rows, float scale, const tfpa_scratch* sc, void* out, float* lse,
                const Sink& sink, bool sliced, const void* k_rows = nullptr,
                const void* v_rows = nullptr) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (!sc || !sc->part_o || !sc->part_ml || sc->cap_rows < 1 || sc->max_splits < 1)
    return TFPA_EINVAL;
  if (rows > 0 && (!q || !aligned(q, 16))) return TFPA_EINVAL;
  if (sliced && rows > 0 && (!out || !aligned(out, 8))) return TFPA_EINVAL;
  if (anc && !aligned(anc, 8)) return TFPA_EINVAL;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TFPA_EINVAL;
  if (!sliced && rows > sc->cap_rows) return TFPA_ECAPACITY;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  for (const Run& r : runs)
    if (tfpa_num_splits(segs[r.seg].seq_len) > sc->max_splits) return TFPA_ECAPACITY;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int kv = c->dtype;
  const bool fp8 = kv == kKvFp8;
  const int G = c->hq / c->hkv;
  for (const Run& r : runs)
    if (on_verify_path(r, G, kv)) {
      if ((e = check_tma_source(q))) return e;
      break;
    }
  if (k_rows || v_rows) {
    if (!k_rows || !v_rows || !aligned(k_rows, 16) || !aligned(v_rows, 16)) return TFPA_EINVAL;
    bool fuse = true;
    for (size_t i = 0; fuse && i < runs.size(); ++i) {
      fuse = !on_verify_path(runs[i], G, kv);   // the decode partial path
      for (size_t j = 0; fuse && j < i; ++j) fuse = runs[j].seg != runs[i].seg;
    }
    if (!fuse) {
      if ((e = write_impl(c, segs, nseg, k_rows, v_rows, row_seg, row_pos, rows,
                          RopeArgs{nullptr, nullptr, nullptr, 0}, sink)))
        return e;
      k_rows = v_rows = nullptr;
    }
  }
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  const size_t hd = (size_t)c->hq * kHeadDim;

  size_t ri = 0;
  int32_t taken = 0;  // rows of runs[ri] already launched
  // Launch parameters are large (kernel arguments by value): each host
  // thread builds them in its own buffers.
  thread_local DecodeParams pd[2];   // [1]: a 4-bit cache's runs of more than eight vectors
  thread_local PrefillParams pv;     // the tensor-core verify launch of the same rows
  thread_local MergeParams mp;
  // Runs of four or more m-tiles (16 query vectors each, so at least 49
  // vectors per kv head) are dense enough for the tensor cores: they go to
  // the prefill kernel in verify mode (128 / G rows x the group's G heads
  // per tile), the rest to the decode partial kernel.  Decided on the
  // call's whole run, so every slice of it computes its rows with the same
  // arithmetic (slices give the same bytes as one launch).  A group wider
  // than a tile (more than 128 query heads per kv head) stays on the decode
  // kernel (on_verify_path).
  const int vrows = G <= kVerifyVectors ? kVerifyVectors / G : 1;   // rows of a verify tile
  while (ri < runs.size()) {
    SourceSet ss;
    const int32_t base = runs[ri].row0 + taken;  // first call row of this launch
    int32_t nrows = 0, items[2] = {0, 0}, tiles = 0;
    int nr = 0, nd[2] = {0, 0}, nv = 0;  // runs of the slice: all, decode, verify
    while (ri < runs.size() && nr < kMaxRuns && nrows < sc->cap_rows) {
      const Run& r = runs[ri];
      const int src = ss.add(segs, r.seg);
      if (src < 0) break;
      const int32_t take = std::min(r.nrows - taken, sc->cap_rows - nrows);
      const tfpa_seg& g = segs[r.seg];
      if (on_verify_path(r, G, kv)) {
        if (nv == 0) std::memset(&pv, 0, sizeof(pv));   // only launches that run are built
        RunInfo& info = pv.runs[nv++];
        fill_run(info, g, src, nrows, take, r.pos0 + taken);
        info.pps = verify_pages_per_split(g.seq_len, kv);
        info.nsplit = verify_num_splits(g.seq_len, kv);
        info.item0 = tiles;
        tiles += c->hkv * ((take + vrows - 1) / vrows) * info.nsplit;
        mp.d.runs[nr] = MergeRun{nrows, take, info.nsplit, 0};
      } else {
        // decided on the call's whole run, like the verify path
        const int w = on_wide_path(r, G, kv) ? 1 : 0;
        DecodeParams& p = pd[w];
        if (nd[w] == 0) std::memset(&p, 0, sizeof(p));
        RunInfo& info = p.d.runs[nd[w]++];
        fill_run(info, g, src, nrows, take, r.pos0 + taken);
        if (kv == kKvFp4) {
          info.pps = fp4_pages_per_split(g.seq_len, c->hkv);
          info.nsplit = fp4_num_splits(g.seq_len, c->hkv);
        }
        info.item0 = items[w];
        const int vecs = item_vectors(w ? kKvFp4Wide : kv);
        items[w] += c->hkv * ((take * G + vecs - 1) / vecs) * info.nsplit;
        mp.d.runs[nr] = MergeRun{nrows, take, info.nsplit, 0};
      }
      ++nr;
      nrows += take;
      taken += take;
      if (taken == r.nrows) {
        ++ri;
        taken = 0;
      }
    }
    const int32_t srow = sliced ? 0 : base;  // scratch row of this launch's first row
    const size_t srow_elems = (size_t)srow * c->hq * sc->max_splits;
    float* part_o = sc->part_o + srow_elems * kHeadDim;
    float* part_ml = sc->part_ml + srow_elems * 2;
    // With arrival counters, plain causal rows in parameter mode, no rows on
    // the verify path and few splits per stream, the partial kernel merges
    // the slice itself.  A group's merge runs on the one SM that finished
    // its last split, reading every split's partial: cheap for a few splits,
    // slower than a separate grid-wide merge for many.
    bool fused = sliced && nv == 0 && sc->arrive && !anc && !sink.device();
    for (int w = 0; w < 2; ++w)
      for (int r = 0; fused && r < nd[w]; ++r)
        fused = pd[w].d.runs[r].nsplit <= kFusedMergeMaxSplits;
    for (int w = 0; w < 2; ++w) {
      if (nd[w] == 0) continue;
      DecodeParams& p = pd[w];
      const int wkv = w ? kKvFp4Wide : kv;
      if (kv != kKvFp4 &&
          (e = fill_maps(c, segs, ss, fp8, fp8 ? 128 : 64, 128, p.maps, p.nsrc)))
        return e;
      p.q = static_cast<const __nv_bfloat16*>(q) + (size_t)base * hd;
      p.anc = anc ? anc + base : nullptr;   // the ancestor table shifts with the rows
      p.part_o = part_o;
      p.part_ml = part_ml;
      p.k_scale = c->k_scale;
      p.v_scale = c->v_scale;
      p.err_flag = c->err_flag;
      const size_t rd = (size_t)c->hkv * kHeadDim;
      p.k_rows = k_rows ? static_cast<const __nv_bfloat16*>(k_rows) + (size_t)base * rd : nullptr;
      p.v_rows = v_rows ? static_cast<const __nv_bfloat16*>(v_rows) + (size_t)base * rd : nullptr;
      if (k_rows || kv == kKvFp4) p.nsrc = fill_bases(c, segs, ss, p.k_base, p.v_base);
      p.arrive = fused ? sc->arrive + (size_t)srow * c->hq : nullptr;
      p.out = fused ? static_cast<__nv_bfloat16*>(out) + (size_t)base * hd : nullptr;
      p.lse = fused && lse ? lse + (size_t)base * c->hq : nullptr;
      p.d.nruns = nd[w];
      p.d.n_items = items[w];
      p.hq = c->hq;
      p.hkv = c->hkv;
      p.group = G;
      p.max_splits = sc->max_splits;
      p.num_pages = c->num_pages;
      p.rows = nrows;
      p.scale_log2 = scale * 1.4426950408889634f;
      // In device mode the grid is one CTA per SM whatever the work, so
      // that the launch can be replayed as the streams grow.
      const int grid = std::min(sink.device() ? nsm : std::min(items[w], nsm), kMaxDecodeGrid);
      plan_cta_ranges(p, nd[w], G, wkv, grid);
      record(1, base, nrows, nd[w], items[w], grid, (int64_t)base * hd, 0);
      if ((e = sink.decode(p, wkv, grid))) return e;
    }
    if (nv > 0) {
      if (kv == kKvFp4)
        pv.nsrc = fill_bases(c, segs, ss, pv.k_base, pv.v_base);
      else if ((e = fill_maps(c, segs, ss, fp8, fp8 ? 128 : 64, 128, pv.maps, pv.nsrc)))
        return e;
      // The kernel loads a verify tile's Q as two boxes of 64 query vectors
      // when G divides 64 (so that a tile of at most 64 vectors can hold
      // them twice, one copy per MMA slot), else as one box.
      const int qbox = 64 % G == 0 ? 64 / G : vrows;
      if ((e = get_qmap(static_cast<const __nv_bfloat16*>(q) + (size_t)base * hd, c->hq, nrows,
                        G, qbox, &pv.qmap)))
        return e;
      pv.q = static_cast<const __nv_bfloat16*>(q) + (size_t)base * hd;
      pv.anc = anc ? anc + base : nullptr;
      pv.part_o = part_o;
      pv.part_ml = part_ml;
      pv.k_scale = c->k_scale;
      pv.v_scale = c->v_scale;
      pv.err_flag = c->err_flag;
      pv.nruns = nv;
      pv.n_tiles = tiles;
      pv.hq = c->hq;
      pv.hkv = c->hkv;
      pv.group = G;
      pv.num_pages = c->num_pages;
      pv.rows = nrows;
      pv.max_splits = sc->max_splits;
      pv.scale_log2 = scale * 1.4426950408889634f;
      record(8, base, nrows, nv, tiles, tiles, (int64_t)base * hd, 0);
      if ((e = sink.verify(pv, kv, tiles))) return e;
    }
    if (sliced && !fused) {
      mp.part_o = part_o;
      mp.part_ml = part_ml;
      mp.out = static_cast<__nv_bfloat16*>(out) + (size_t)base * hd;
      mp.lse = lse ? lse + (size_t)base * c->hq : nullptr;
      mp.d.nruns = nr;
      mp.d.rows = nrows;
      mp.hq = c->hq;
      mp.max_splits = sc->max_splits;
      record(2, base, nrows, nr, nrows * c->hq, (nrows * c->hq + 7) / 8, 0, (int64_t)base * hd);
      if ((e = sink.merge(mp))) return e;
    }
  }
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_decode_partial(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                                   const void* q, const int32_t* row_seg, const int32_t* row_pos,
                                   int32_t rows, float softmax_scale, const tfpa_scratch* scratch,
                                   cudaStream_t stream) {
  return no_throw([&] {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, nullptr, rows, softmax_scale,
                       scratch, nullptr, nullptr, Sink{stream, nullptr}, false);
  });
}

extern "C" int tfpa_decode(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                           const void* q, const int32_t* row_seg, const int32_t* row_pos,
                           int32_t rows, float softmax_scale, const tfpa_scratch* scratch,
                           void* out, float* lse, cudaStream_t stream) {
  return no_throw([&] {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, nullptr, rows, softmax_scale,
                       scratch, out, lse, Sink{stream, nullptr}, true);
  });
}

extern "C" int tfpa_row_splits(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                               const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                               int32_t* nsplit) {
  int e;
  if ((e = check_cache(cache)) || (e = check_segs(cache, segs, nseg))) return e;
  if (rows > 0 && !nsplit) return TFPA_EINVAL;
  thread_local std::vector<Run> runs;
  if ((e = no_throw([&] { return build_runs(segs, nseg, row_seg, row_pos, rows, runs); })))
    return e;
  // the same choice of kernel as decode_impl: runs of four or more m-tiles
  // take the tensor-core verify path and its splits
  const int G = cache->hq / cache->hkv;
  for (const Run& r : runs) {
    const int32_t L = segs[r.seg].seq_len;
    const int32_t n = on_verify_path(r, G, cache->dtype)
                          ? verify_num_splits(L, cache->dtype)
                          : decode_num_splits(cache->dtype, L, cache->hkv);
    for (int32_t i = 0; i < r.nrows; ++i) nsplit[r.row0 + i] = n;
  }
  return TFPA_OK;
}

extern "C" int tfpa_decode_tree(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                                const void* q, const int32_t* row_seg, const int32_t* row_pos,
                                const uint64_t* row_anc, int32_t rows, float softmax_scale,
                                const tfpa_scratch* scratch, void* out, float* lse,
                                cudaStream_t stream) {
  if (rows > 0 && !row_anc) return TFPA_EINVAL;
  return no_throw([&] {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, row_anc, rows, softmax_scale,
                       scratch, out, lse, Sink{stream, nullptr}, true);
  });
}

extern "C" int tfpa_decode_append(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                                  const void* k_rows, const void* v_rows, const void* q,
                                  const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                                  float softmax_scale, const tfpa_scratch* scratch, void* out,
                                  float* lse, cudaStream_t stream) {
  if (rows > 0 && (!k_rows || !v_rows)) return TFPA_EINVAL;
  return no_throw([&] {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, nullptr, rows, softmax_scale,
                       scratch, out, lse, Sink{stream, nullptr}, true, k_rows, v_rows);
  });
}

extern "C" int tfpa_merge(const tfpa_scratch* sc, int32_t hq, int32_t rows,
                          const int32_t* nsplit, void* out, float* lse, cudaStream_t stream) {
  if (!sc || !sc->part_o || !sc->part_ml || hq < 1 || rows < 0) return TFPA_EINVAL;
  if (rows > sc->cap_rows) return TFPA_ECAPACITY;
  if (rows == 0) return TFPA_OK;
  if (!nsplit || !out || !aligned(out, 8)) return TFPA_EINVAL;
  for (int32_t r = 0; r < rows; ++r)
    if (nsplit[r] < 1 || nsplit[r] > std::min(sc->max_splits, kMaxSplits)) return TFPA_ECAPACITY;
  int e;
  if ((e = check_device())) return e;
  thread_local MergeParams mp;
  int32_t r = 0;
  while (r < rows) {
    std::memset(&mp, 0, sizeof(mp));
    const int32_t base = r;
    int nr = 0;
    while (r < rows && nr < (int)(sizeof(mp.d.runs) / sizeof(mp.d.runs[0]))) {
      int32_t n = 1;
      while (r + n < rows && nsplit[r + n] == nsplit[r]) ++n;
      mp.d.runs[nr++] = MergeRun{r - base, n, nsplit[r], 0};
      r += n;
    }
    const size_t srow = (size_t)base * hq * sc->max_splits;
    mp.part_o = sc->part_o + srow * kHeadDim;
    mp.part_ml = sc->part_ml + srow * 2;
    mp.out = static_cast<__nv_bfloat16*>(out) + (size_t)base * hq * kHeadDim;
    mp.lse = lse ? lse + (size_t)base * hq : nullptr;
    mp.d.nruns = nr;
    mp.d.rows = r - base;
    mp.hq = hq;
    mp.max_splits = sc->max_splits;
    record(2, base, r - base, nr, (r - base) * hq, ((r - base) * hq + 7) / 8, 0,
           (int64_t)base * hq * kHeadDim);
    if (!dry_run())
      if ((e = to_err(launch_merge(mp, stream)))) return e;
  }
  return TFPA_OK;
}

namespace {

int write_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* k_rows,
               const void* v_rows, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
               const RopeArgs& rope, const Sink& sink, bool read) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (rows > 0 && (!k_rows || !v_rows || !aligned(k_rows, 16) || !aligned(v_rows, 16)))
    return TFPA_EINVAL;
  if (rope.cos) {
    if (!rope.sin || rope.n < 1 || !aligned(rope.cos, 16) || !aligned(rope.sin, 16) ||
        (rope.pos && !aligned(rope.pos, 4)))
      return TFPA_EINVAL;
  }
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  if (rope.cos && !rope.pos)
    for (const Run& r : runs)
      if (r.pos0 + r.nrows > rope.n) return TFPA_ERANGE;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const size_t rd = (size_t)c->hkv * kHeadDim;
  thread_local WriteParams p;
  size_t ri = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    const int32_t base = runs[ri].row0;
    int nr = 0;
    int32_t nrows = 0;
    while (ri < runs.size() && nr < kMaxRuns) {
      const Run& r = runs[ri++];
      const tfpa_seg& g = segs[r.seg];
      WriteRun& w = p.d.runs[nr++];
      w.page_table = g.page_table;
      w.k_dst = g.page_table ? c->k_pool : g.k_slab;
      w.v_dst = g.page_table ? c->v_pool : g.v_slab;
      w.row0 = r.row0 - base;
      w.nrows = r.nrows;
      w.pos0 = r.pos0;
      w.slab_cap = g.slab_cap;
      w.seq_len = g.seq_len;
      nrows = r.row0 + r.nrows - base;
    }
    p.k_rows = static_cast<const __nv_bfloat16*>(k_rows) + (size_t)base * rd;
    p.v_rows = static_cast<const __nv_bfloat16*>(v_rows) + (size_t)base * rd;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.err_flag = c->err_flag;
    p.rope_cos = rope.cos;
    p.rope_sin = rope.sin;
    p.rope_pos = rope.pos ? rope.pos + base : nullptr;   // shifts with the rows
    p.rope_n = rope.n;
    p.d.nruns = nr;
    p.d.rows = nrows;
    p.hkv = c->hkv;
    p.num_pages = c->num_pages;
    p.kv = c->dtype;
    record(read ? 9 : 0, base, nrows, nr, nrows * c->hkv, (nrows * c->hkv + 15) / 16, 0, 0);
    if (read)
      e = dry_run() ? TFPA_OK : to_err(launch_read_kv(p, sink.stream));
    else
      e = sink.write(p);
    if (e) return e;
  }
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_write_kv(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                             const void* k_rows, const void* v_rows, const int32_t* row_seg,
                             const int32_t* row_pos, int32_t rows, cudaStream_t stream) {
  return no_throw([&] {
    return write_impl(c, segs, nseg, k_rows, v_rows, row_seg, row_pos, rows,
                      RopeArgs{nullptr, nullptr, nullptr, 0}, Sink{stream, nullptr});
  });
}

// The write's launches with the rows as the destination (const cast back by
// the kernel: they are the caller's output).
extern "C" int tfpa_read_kv(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, void* k_rows,
                            void* v_rows, const int32_t* row_seg, const int32_t* row_pos,
                            int32_t rows, cudaStream_t stream) {
  return no_throw([&] {
    return write_impl(c, segs, nseg, k_rows, v_rows, row_seg, row_pos, rows,
                      RopeArgs{nullptr, nullptr, nullptr, 0}, Sink{stream, nullptr}, true);
  });
}

extern "C" int tfpa_write_kv_rope(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                                  const void* k_rows, const void* v_rows,
                                  const int32_t* row_seg, const int32_t* row_pos,
                                  const int32_t* rope_pos, const float* rope_cos,
                                  const float* rope_sin, int32_t rope_n, int32_t rows,
                                  cudaStream_t stream) {
  if (!rope_cos) return TFPA_EINVAL;
  return no_throw([&] {
    return write_impl(c, segs, nseg, k_rows, v_rows, row_seg, row_pos, rows,
                      RopeArgs{rope_pos, rope_cos, rope_sin, rope_n}, Sink{stream, nullptr});
  });
}

// ------------------------------------------------------------ plans
namespace {
uint64_t compute_shape(const tfpa_plan* plan);
}  // namespace

extern "C" tfpa_plan* tfpa_plan_create(void) {
  tfpa_plan* plan = new (std::nothrow) tfpa_plan();
  if (plan) plan->shape = compute_shape(plan);
  return plan;
}

extern "C" void tfpa_plan_destroy(tfpa_plan* plan) { delete plan; }

extern "C" void tfpa_plan_clear(tfpa_plan* plan) {
  if (!plan) return;
  plan->entries.clear();
  plan->decode.clear();
  plan->verify.clear();
  plan->merge.clear();
  plan->write.clear();
  plan->dyn_used = 0;
  plan->shape = compute_shape(plan);
}

extern "C" int32_t tfpa_plan_launches(const tfpa_plan* plan) {
  return plan ? (int32_t)plan->entries.size() : 0;
}

extern "C" int tfpa_plan_set_device(tfpa_plan* plan, void* dyn, size_t bytes) {
  if (!plan || !plan->entries.empty()) return TFPA_EINVAL;
  if (dyn && (!aligned(dyn, 16) || bytes < 16)) return TFPA_EINVAL;
  plan->dyn_base = static_cast<uint8_t*>(dyn);
  plan->dyn_cap = dyn ? bytes : 0;
  plan->dyn_used = 0;
  plan->shape = compute_shape(plan);
  return TFPA_OK;
}

extern "C" size_t tfpa_plan_dyn_bytes(const tfpa_plan* plan) {
  return plan ? plan->dyn_used : 0;
}

extern "C" int tfpa_plan_dyn_pack(const tfpa_plan* plan, void* host, size_t bytes) {
  if (!plan || !plan->dyn_base) return TFPA_EINVAL;
  if (plan->dyn_used == 0) return TFPA_OK;
  if (!host) return TFPA_EINVAL;
  if (bytes < plan->dyn_used) return TFPA_ECAPACITY;
  uint8_t* dst = static_cast<uint8_t*>(host);
  auto put = [&](const void* slot, const void* d, size_t n) {
    std::memcpy(dst + (static_cast<const uint8_t*>(slot) - plan->dyn_base), d, n);
  };
  for (const DecodeParams& p : plan->decode) put(p.dyn, &p.d, sizeof(p.d));
  for (const MergeParams& p : plan->merge) put(p.dyn, &p.d, sizeof(p.d));
  for (const WriteParams& p : plan->write) put(p.dyn, &p.d, sizeof(p.d));
  return TFPA_OK;
}

namespace {
// A 64-bit hash of a byte range, eight bytes a step (multiply and
// xor-shift; FNV-1a for the tail).
uint64_t fnv1a(uint64_t h, const void* data, size_t n) {
  const uint8_t* b = static_cast<const uint8_t*>(data);
  size_t i = 0;
  for (; i + 8 <= n; i += 8) {
    uint64_t w;
    std::memcpy(&w, b + i, 8);
    h = (h ^ w) * 0x9E3779B97F4A7C15ull;
    h ^= h >> 29;
  }
  for (; i < n; ++i) h = (h ^ b[i]) * 1099511628211ull;
  return h;
}
// A launch's parameters without its dynamic data.
template <typename P>
uint64_t hash_static(uint64_t h, const P& p) {
  const uint8_t* b = reinterpret_cast<const uint8_t*>(&p);
  const size_t d0 = reinterpret_cast<const uint8_t*>(&p.d) - b;
  h = fnv1a(h, b, d0);
  return fnv1a(h, b + d0 + sizeof(p.d), sizeof(P) - d0 - sizeof(p.d));
}
}  // namespace

namespace {
uint64_t compute_shape(const tfpa_plan* plan) {
  uint64_t h = 14695981039346656037ull;
  for (const tfpa_plan::Entry& en : plan->entries) {
    const int32_t head[3] = {(int32_t)en.kind, (int32_t)en.kv, en.grid};
    h = fnv1a(h, head, sizeof(head));
    switch (en.kind) {
      case tfpa_plan::kDecode: h = hash_static(h, plan->decode[en.index]); break;
      case tfpa_plan::kVerify: h = fnv1a(h, &plan->verify[en.index], sizeof(PrefillParams)); break;
      case tfpa_plan::kMerge: h = hash_static(h, plan->merge[en.index]); break;
      case tfpa_plan::kWrite: h = hash_static(h, plan->write[en.index]); break;
    }
  }
  return h;
}
}  // namespace

// The shape is recomputed after each planning call (while the GPU is busy
// with the previous step), so that a replay only compares two numbers.
extern "C" uint64_t tfpa_plan_shape(const tfpa_plan* plan) { return plan ? plan->shape : 0; }

extern "C" int tfpa_plan_capture(tfpa_plan* plan, const tfpa_copy* before, int32_t nbefore,
                                 const tfpa_copy* after, int32_t nafter, cudaStream_t stream) {
  if (!plan || plan->entries.empty() || nbefore < 0 || nafter < 0 ||
      (nbefore > 0 && !before) || (nafter > 0 && !after))
    return TFPA_EINVAL;
  for (int32_t i = 0; i < nbefore; ++i)
    if (before[i].bytes && (!before[i].dst || !before[i].src)) return TFPA_EINVAL;
  for (int32_t i = 0; i < nafter; ++i)
    if (after[i].bytes && (!after[i].dst || !after[i].src)) return TFPA_EINVAL;
  const uint64_t shape = tfpa_plan_shape(plan);
  if (dry_run()) {
    plan->exec_shape = shape;
    plan->captured = true;
    return TFPA_OK;
  }
  int e;
  if ((e = check_device())) return e;
  if (stream == nullptr || stream == cudaStreamLegacy) return TFPA_EINVAL;   // not capturable
  if (cudaStreamBeginCapture(stream, cudaStreamCaptureModeThreadLocal) != cudaSuccess)
    return TFPA_ECUDA;
  bool ok = true;
  for (int32_t i = 0; ok && i < nbefore; ++i)
    if (before[i].bytes)
      ok = cudaMemcpyAsync(before[i].dst, before[i].src, before[i].bytes, cudaMemcpyDefault,
                           stream) == cudaSuccess;
  if (ok) ok = tfpa_plan_launch(plan, stream) == TFPA_OK;
  for (int32_t i = 0; ok && i < nafter; ++i)
    if (after[i].bytes)
      ok = cudaMemcpyAsync(after[i].dst, after[i].src, after[i].bytes, cudaMemcpyDefault,
                           stream) == cudaSuccess;
  cudaGraph_t graph = nullptr;
  const bool ended = cudaStreamEndCapture(stream, &graph) == cudaSuccess;
  cudaGraphExec_t exec = nullptr;
  ok = ok && ended && graph && cudaGraphInstantiate(&exec, graph, 0ull) == cudaSuccess;
  if (graph) cudaGraphDestroy(graph);
  if (!ok) {
    cudaGetLastError();   // the failed call's error stays with this call
    return TFPA_ECUDA;
  }
  if (plan->exec) cudaGraphExecDestroy(plan->exec);
  plan->exec = exec;
  plan->exec_shape = shape;
  plan->captured = true;
  return TFPA_OK;
}

extern "C" int tfpa_plan_replay(const tfpa_plan* plan, cudaStream_t stream) {
  if (!plan || !plan->captured) return TFPA_EINVAL;
  if (tfpa_plan_shape(plan) != plan->exec_shape) return TFPA_EINVAL;
  if (dry_run()) return TFPA_OK;
  return to_err(cudaGraphLaunch(plan->exec, stream));
}

namespace {
// Runs a planning call into `plan`; on failure the plan is left as it was.
template <typename F>
int plan_call(tfpa_plan* plan, F&& fn) {
  if (!plan) return TFPA_EINVAL;
  const Sink sink{nullptr, plan};
  const Sink::Mark m = sink.mark();
  const int e = no_throw([&] { return fn(sink); });
  if (e != TFPA_OK)
    sink.rollback(m);   // the plan, and so its shape, as before the call
  else
    plan->shape = compute_shape(plan);
  return e;
}
}  // namespace

extern "C" int tfpa_plan_write_kv(tfpa_plan* plan, const tfpa_cache* c, const tfpa_seg* segs,
                                  int32_t nseg, const void* k_rows, const void* v_rows,
                                  const int32_t* row_seg, const int32_t* row_pos,
                                  int32_t rows) {
  return plan_call(plan, [&](const Sink& sink) {
    return write_impl(c, segs, nseg, k_rows, v_rows, row_seg, row_pos, rows,
                      RopeArgs{nullptr, nullptr, nullptr, 0}, sink);
  });
}

extern "C" int tfpa_plan_decode(tfpa_plan* plan, const tfpa_cache* cache, const tfpa_seg* segs,
                                int32_t nseg, const void* q, const int32_t* row_seg,
                                const int32_t* row_pos, int32_t rows, float softmax_scale,
                                const tfpa_scratch* scratch, void* out, float* lse) {
  return plan_call(plan, [&](const Sink& sink) {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, nullptr, rows, softmax_scale,
                       scratch, out, lse, sink, true);
  });
}

extern "C" int tfpa_plan_decode_append(tfpa_plan* plan, const tfpa_cache* cache,
                                       const tfpa_seg* segs, int32_t nseg, const void* k_rows,
                                       const void* v_rows, const void* q, const int32_t* row_seg,
                                       const int32_t* row_pos, int32_t rows, float softmax_scale,
                                       const tfpa_scratch* scratch, void* out, float* lse) {
  if (rows > 0 && (!k_rows || !v_rows)) return TFPA_EINVAL;
  return plan_call(plan, [&](const Sink& sink) {
    return decode_impl(cache, segs, nseg, q, row_seg, row_pos, nullptr, rows, softmax_scale,
                       scratch, out, lse, sink, true, k_rows, v_rows);
  });
}

extern "C" int tfpa_plan_launch(const tfpa_plan* plan, cudaStream_t stream) {
  if (!plan) return TFPA_EINVAL;
  if (dry_run()) return TFPA_OK;
  for (const tfpa_plan::Entry& en : plan->entries) {
    cudaError_t r = cudaSuccess;
    switch (en.kind) {
      case tfpa_plan::kDecode:
        r = launch_decode_partial(plan->decode[en.index], en.kv, en.grid, stream);
        break;
      case tfpa_plan::kVerify:
        r = launch_verify(plan->verify[en.index], en.kv, en.grid, stream);
        break;
      case tfpa_plan::kMerge:
        r = launch_merge(plan->merge[en.index], stream);
        break;
      case tfpa_plan::kWrite:
        r = launch_write_kv(plan->write[en.index], stream);
        break;
    }
    if (r != cudaSuccess) return TFPA_ECUDA;
  }
  return TFPA_OK;
}

extern "C" int tfpa_keep_kv(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                            const int32_t* keep_seg, const int32_t* keep_src,
                            const int32_t* keep_dst, int32_t n, cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (n < 0 || (n > 0 && (!keep_seg || !keep_src || !keep_dst))) return TFPA_EINVAL;
  if (n > kMaxKeep) return TFPA_ECAPACITY;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t sg = keep_seg[i];
    if (sg < 0 || sg >= nseg) return TFPA_ERANGE;
    const tfpa_seg& g = segs[sg];
    if (keep_src[i] < 0 || keep_src[i] >= g.seq_len || keep_dst[i] < 0 ||
        keep_dst[i] >= g.seq_len)
      return TFPA_ERANGE;
    for (int32_t j = 0; j < i; ++j)          // one writer per destination row
      if (keep_seg[j] == sg && keep_dst[j] == keep_dst[i]) return TFPA_EINVAL;
  }
  if (n == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  thread_local KeepParams p;
  std::memset(&p, 0, sizeof(p));
  for (int32_t i = 0; i < n; ++i) {
    const tfpa_seg& g = segs[keep_seg[i]];
    KeepPair& kp = p.pairs[i];
    kp.page_table = g.page_table;
    kp.k_slab = g.page_table ? nullptr : g.k_slab;
    kp.v_slab = g.page_table ? nullptr : g.v_slab;
    kp.slab_cap = g.page_table ? 0 : g.slab_cap;
    kp.src = keep_src[i];
    kp.dst = keep_dst[i];
  }
  p.k_pool = c->k_pool;
  p.v_pool = c->v_pool;
  p.err_flag = c->err_flag;
  p.n = n;
  p.hkv = c->hkv;
  p.num_pages = c->num_pages;
  p.row_bytes = row_bytes_of(c);
  record(4, 0, n, 0, n * c->hkv, c->hkv, 0, 0);
  if (!dry_run())
    if ((e = to_err(launch_keep(p, stream)))) return e;
  return TFPA_OK;
}

extern "C" int tfpa_stage_pages(int32_t* page_table, int32_t first, const int32_t* pages,
                                int32_t n, cudaStream_t stream) {
  if (!page_table || first < 0 || n < 0 || (n > 0 && !pages)) return TFPA_EINVAL;
  if (n == 0) return TFPA_OK;
  int e;
  if (!dry_run() && (e = check_device())) return e;
  thread_local StageParams p;
  for (int32_t done = 0; done < n; done += kMaxStage) {
    const int32_t m = std::min<int32_t>(kMaxStage, n - done);
    p.table = page_table;
    p.first = first + done;
    p.n = m;
    std::memcpy(p.ids, pages + done, sizeof(int32_t) * m);
    record(5, done, m, 0, m, 1, 0, 0);
    if (!dry_run())
      if ((e = to_err(launch_stage(p, stream)))) return e;
  }
  return TFPA_OK;
}

namespace {

int copy_impl(const tfpa_cache* c, const tfpa_seg* seg, int32_t p0, int32_t p1, const void* image,
              bool restore, cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, seg, 1))) return e;
  if (!image || !aligned(image, 16)) return TFPA_EINVAL;
  if (p0 < 0 || p0 > p1 || p1 > seg->seq_len) return TFPA_ERANGE;
  if (p0 == p1) return TFPA_OK;
  if (!dry_run() && (e = check_device())) return e;
  CopyParams p{};
  p.page_table = seg->page_table;
  p.k_base = seg->page_table ? c->k_pool : seg->k_slab;
  p.v_base = seg->page_table ? c->v_pool : seg->v_slab;
  p.image = static_cast<uint8_t*>(const_cast<void*>(image));
  p.err_flag = c->err_flag;
  p.slab_cap = seg->page_table ? 0 : seg->slab_cap;
  p.p0 = p0;
  p.p1 = p1;
  p.page0 = p0 / kPage;
  p.hkv = c->hkv;
  p.num_pages = c->num_pages;
  p.row_bytes = row_bytes_of(c);
  p.restore = restore ? 1 : 0;
  const int npages = (p1 - 1) / kPage - p0 / kPage + 1;
  record(restore ? 7 : 6, p0, p1 - p0, 0, npages * c->hkv * 2, npages * c->hkv * 2, 0, 0);
  if (!dry_run())
    if ((e = to_err(launch_copy(p, npages, stream)))) return e;
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_save_kv(const tfpa_cache* cache, const tfpa_seg* seg, int32_t p0, int32_t p1,
                            void* image, cudaStream_t stream) {
  return copy_impl(cache, seg, p0, p1, image, false, stream);
}

extern "C" int tfpa_restore_kv(const tfpa_cache* cache, const tfpa_seg* seg, int32_t p0,
                               int32_t p1, const void* image, cudaStream_t stream) {
  return copy_impl(cache, seg, p0, p1, image, true, stream);
}

// ------------------------------------------------------------ eviction
namespace {
constexpr int kMassKeys = 128;   // keys of a tile of the weight kernel

int mass_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* q,
              const float* lse, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
              float scale, float decay, float* mass, int32_t mass_cap, cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (rows > 0 && (!q || !aligned(q, 16) || !lse || !aligned(lse, 4) || !mass ||
                   !aligned(mass, 4)))
    return TFPA_EINVAL;
  if (!std::isfinite(scale) || !(scale > 0.f) || !std::isfinite(decay) || decay < 0.f)
    return TFPA_EINVAL;
  if (mass_cap < 1) return TFPA_EINVAL;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  // what a launch could not number is refused before the first one
  auto blocks_of = [&](int32_t s) {
    return (int64_t)c->hkv * (((int64_t)segs[s].seq_len + kMassKeys - 1) / kMassKeys);
  };
  for (const Run& r : runs)
    if (segs[r.seg].seq_len > mass_cap || blocks_of(r.seg) > INT32_MAX) return TFPA_ECAPACITY;
  if ((int64_t)rows * (c->hq / c->hkv) > INT32_MAX) return TFPA_EINVAL;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  // A segment's runs one after the other, in the call's order, so that one
  // block sums all of its rows and the order of a sum is fixed.
  std::stable_sort(runs.begin(), runs.end(),
                   [](const Run& a, const Run& b) { return a.seg < b.seg; });
  const int kv = c->dtype;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  thread_local MassParams p;
  size_t ri = 0;
  int32_t last_seg = -1;                // the segment of the previous launch's last run
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    int32_t nrows = 0, nr = 0;
    int64_t items = 0;
    SourceSet ss;
    const int32_t first_row = runs[ri].row0;
    while (ri < runs.size() && nr < kMaxRuns) {
      const Run& r = runs[ri];
      if (p.nsegs == 0 || p.segs[p.nsegs - 1].index != r.seg) {
        const tfpa_seg& g = segs[r.seg];
        const int64_t blocks = blocks_of(r.seg);
        if (items + blocks > INT32_MAX) break;  // the next launch's
        const int src = ss.add(segs, r.seg);
        if (src < 0) break;
        MassSeg& m = p.segs[p.nsegs++];
        m.page_table = g.page_table;
        m.k_base = g.page_table ? c->k_pool : g.k_slab;
        m.index = r.seg;
        m.seq_len = g.seq_len;
        m.slab_cap = g.slab_cap;
        m.item0 = (int32_t)items;
        m.run0 = nr;
        m.decay = r.seg == last_seg ? 1.f : decay;
        m.src = src;
        items += blocks;
        last_seg = r.seg;
      }
      ++p.segs[p.nsegs - 1].nruns;
      p.runs[nr++] = MassRun{r.row0, r.nrows, r.pos0};
      nrows += r.nrows;
      ++ri;
    }
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.lse = lse;
    p.mass = mass;
    p.k_scale = c->k_scale;
    p.err_flag = c->err_flag;
    p.hq = c->hq;
    p.hkv = c->hkv;
    p.group = c->hq / c->hkv;
    p.num_pages = c->num_pages;
    p.mass_cap = mass_cap;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.tiles = (int32_t)items;
    p.dbufs = 4;
    for (int i = 0; i < p.nsegs; ++i) {
      int64_t vecs = 0;
      for (int r = 0; r < p.segs[i].nruns; ++r)
        vecs += (int64_t)p.runs[p.segs[i].run0 + r].nrows * (c->hq / c->hkv);
      if (vecs > 128) p.dbufs = 2;
    }
    if (kv != kKvFp4) {
      const bool fp8 = kv == kKvFp8;
      const int inner = fp8 ? 128 : 64;
      if (ss.pool && (e = get_map(c->k_pool, (uint64_t)c->num_pages * c->hkv * kPage, fp8, inner,
                                  kMassKeys, &p.maps[0])))
        return e;
      for (int i = 0; i < ss.nslab; ++i) {
        const tfpa_seg& g = segs[ss.slab_seg[i]];
        if ((e = get_map(g.k_slab, (uint64_t)c->hkv * g.slab_cap, fp8, inner, kMassKeys,
                         &p.maps[i + 1])))
          return e;
      }
    }
    const int grid = (int)std::min<int64_t>(items, nsm);
    record(10, first_row, nrows, nr, (int32_t)items, grid, 0, 0);
    if (!dry_run())
      if ((e = to_err(launch_key_mass(p, kv, grid, stream)))) return e;
  }
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_key_mass(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                             const void* q, const float* lse, const int32_t* row_seg,
                             const int32_t* row_pos, int32_t rows, float scale, float decay,
                             float* mass, int32_t mass_cap, cudaStream_t stream) {
  return no_throw([&] {
    return mass_impl(c, segs, nseg, q, lse, row_seg, row_pos, rows, scale, decay, mass, mass_cap,
                     stream);
  });
}

extern "C" int tfpa_evict_kv(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                             const int32_t* keep, const int32_t* next_pos, int32_t sink,
                             int32_t recent, float* mass, int32_t* key_pos, int32_t mass_cap,
                             int32_t* moves, cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (sink < 0 || recent < 0 || mass_cap < 4 || mass_cap % 4) return TFPA_EINVAL;
  if (nseg > 0 && (!keep || !mass || !aligned(mass, 16) || !moves || !aligned(moves, 16) ||
                   (key_pos && !aligned(key_pos, 16))))
    return TFPA_EINVAL;
  for (int32_t s = 0; s < nseg; ++s) {
    if (keep[s] < 1 || keep[s] > segs[s].seq_len) return TFPA_ERANGE;
    // seq_len keys at positions of their own, all below the next
    if (next_pos && next_pos[s] < segs[s].seq_len) return TFPA_ERANGE;
    if (segs[s].seq_len > mass_cap) return TFPA_ECAPACITY;
    if (keep[s] < segs[s].seq_len && (int64_t)sink + recent > keep[s]) return TFPA_EINVAL;
  }
  if (nseg == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  thread_local EvictParams p;
  for (int32_t s0 = 0; s0 < nseg; s0 += kMaxEvictSegs) {
    std::memset(&p, 0, sizeof(p));
    p.nsegs = std::min<int32_t>(kMaxEvictSegs, nseg - s0);
    int32_t most = 0;                   // pairs of one (segment, kv head), at most
    int32_t longest = 0;
    for (int32_t i = 0; i < p.nsegs; ++i) {
      const tfpa_seg& g = segs[s0 + i];
      EvictSeg& v = p.segs[i];
      v.page_table = g.page_table;
      v.k_base = g.page_table ? c->k_pool : g.k_slab;
      v.v_base = g.page_table ? c->v_pool : g.v_slab;
      v.index = s0 + i;
      v.seq_len = g.seq_len;
      v.keep = keep[s0 + i];
      v.next_pos = next_pos ? next_pos[s0 + i] : key_pos ? kNextPosHeld : g.seq_len;
      v.slab_cap = g.slab_cap;
      most = std::max(most, std::min(v.keep, v.seq_len - v.keep));
      if (v.keep < v.seq_len) longest = std::max(longest, v.seq_len);
    }
    p.mass = mass;
    p.key_pos = key_pos;
    p.moves = moves;
    p.err_flag = c->err_flag;
    p.hkv = c->hkv;
    p.num_pages = c->num_pages;
    p.mass_cap = mass_cap;
    p.sink = sink;
    p.recent = recent;
    const int planes = p.nsegs * c->hkv;
    // Blocks of one (segment, kv head): more while the GPU holds them (one a
    // SM) and each has 4,096 slots, a step of its threads.
    p.cluster = 1;
    while (p.cluster < 8 && (int64_t)planes * p.cluster * 2 <= nsm &&
           longest / (p.cluster * 2) >= 4096)
      p.cluster *= 2;
    while (p.cluster < 8 && select_chunk(longest, p.cluster) > kSelectKeys) p.cluster *= 2;
    p.key_slots = std::min(select_chunk(longest, p.cluster), kSelectKeys);
    record(11, s0, p.nsegs, 0, planes, planes, 0, 0);
    if (!dry_run())
      if ((e = to_err(launch_evict_select(p, stream)))) return e;
    if (most == 0) continue;
    // 32 pairs a block and round (64 and 128 of the narrower types); several
    // blocks' worth of rounds where there are many, so that planes of few pairs
    // leave early
    p.grid_x = std::min((most + 31) / 32, std::max(1, 64 * nsm / planes));
    record(12, s0, p.nsegs, 0, planes, p.grid_x * planes, 0, 0);
    if (!dry_run())
      if ((e = to_err(launch_evict_move(p, c->dtype, stream)))) return e;
  }
  return TFPA_OK;
}

// ------------------------------------------------------------ rotary tables
namespace {
constexpr double kTwoPi = 6.283185307179586476925;
constexpr int64_t kMaxRopePos = int64_t(1) << 31;

// A frequency (radians a position, at most 1) as a fraction of a turn, times
// 2^64 and rounded: its 53 bits times 1 / 2 pi to 128 bits.
uint64_t turns_of(double f) {
  int ex;
  const uint64_t mant = (uint64_t)std::ldexp(std::frexp(f, &ex), 53);   // f = mant 2^(ex - 53)
  typedef unsigned __int128 u128;
  const u128 hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;    // 2^128 / 2 pi
  const u128 prod = mant * hi + ((mant * lo) >> 64);
  const int shift = 53 - ex;
  return shift >= 127 ? 0 : (uint64_t)((prod + ((u128)1 << (shift - 1))) >> shift);
}

// The frequencies (radians a position) of a table's columns.
int rope_freqs(const tfpa_rope_spec* r, double* freq) {
  if (!r || r->rot_dim < 16 || r->rot_dim > kHeadDim || r->rot_dim % 16) return TFPA_EINVAL;
  if (!std::isfinite(r->base) || !(r->base > 1.0) || !std::isfinite(r->attn_scale) ||
      !((float)r->attn_scale > 0.f) || !std::isfinite((float)r->attn_scale))
    return TFPA_EINVAL;
  const int n = r->rot_dim / 2;
  const double d = r->rot_dim, f = r->factor;
  if (r->scaling < TFPA_ROPE_NONE || r->scaling > TFPA_ROPE_RAMP) return TFPA_EINVAL;
  if (r->scaling != TFPA_ROPE_NONE && (!std::isfinite(f) || !(f >= 1.0))) return TFPA_EINVAL;
  const bool parts = r->scaling == TFPA_ROPE_BANDS || r->scaling == TFPA_ROPE_RAMP;
  if (parts && (r->orig_len < 1 || !std::isfinite(r->low) || !std::isfinite(r->high) ||
                !(r->low > 0.0) || !(r->high > r->low)))
    return TFPA_EINVAL;
  const double base =
      r->scaling == TFPA_ROPE_BASE ? r->base * std::pow(f, d / (d - 2.0)) : r->base;
  if (!std::isfinite(base)) return TFPA_EINVAL;
  // TFPA_ROPE_RAMP: the dims that turn `high` and `low` times in orig_len positions
  double first = 0.0, end = 0.0;
  if (r->scaling == TFPA_ROPE_RAMP) {
    const auto where = [&](double turns) {
      return d * std::log(r->orig_len / (kTwoPi * turns)) / (2.0 * std::log(r->base));
    };
    first = std::max(std::floor(where(r->high)), 0.0);
    end = std::min(std::ceil(where(r->low)), d - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double w = std::pow(base, -2.0 * i / d);
    double keep = 1.0;                       // share of the frequency that is not stretched
    switch (r->scaling) {
      case TFPA_ROPE_LINEAR: keep = 0.0; break;
      case TFPA_ROPE_BANDS:
        keep = (r->orig_len * w / kTwoPi - r->low) / (r->high - r->low);
        break;
      case TFPA_ROPE_RAMP: keep = 1.0 - (i - first) / std::max(end - first, 0.001); break;
      default: break;
    }
    keep = std::min(1.0, std::max(0.0, keep));
    if (r->scaling == TFPA_ROPE_LINEAR || parts) w = w * keep + w / f * (1.0 - keep);
    freq[i] = w;
  }
  return TFPA_OK;
}
}  // namespace

extern "C" int tfpa_rope_table(const tfpa_rope_spec* spec, int64_t first, int32_t n, float* cos,
                               float* sin, cudaStream_t stream) {
  double freq[kHeadDim / 2];
  int e;
  if ((e = rope_freqs(spec, freq))) return e;
  if (n < 0 || (n > 0 && (!cos || !sin || !aligned(cos, 16) || !aligned(sin, 16))))
    return TFPA_EINVAL;
  if (first < 0 || first > kMaxRopePos - n) return TFPA_ERANGE;
  if (n == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  TableParams p{};
  p.cos = cos;
  p.sin = sin;
  p.half = spec->rot_dim / 2;
  for (int i = 0; i < p.half; ++i) p.turns[i] = turns_of(freq[i]);
  p.first = first;
  p.n = n;
  p.attn_scale = (float)spec->attn_scale;
  p.attn_rest = (float)(spec->attn_scale - (double)p.attn_scale);
  record(13, 0, n, 0, n, 0, 0, 0);
  return dry_run() ? TFPA_OK : to_err(launch_rope_table(p, nsm, stream));
}

// ------------------------------------------------------------ a projection's rows
namespace {

// Do [a, a + na) and [b, b + nb) share a byte?
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uint64_t)nb && y < x + (uint64_t)na;
}

// From this many heads on a thread group takes several: one a group then no
// longer has all of them on the GPU at once.
constexpr int32_t kWideHeads = 8192;

int qkv_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const tfpa_qkv* in,
             const int32_t* row_seg, const int32_t* row_pos, int32_t rows, void* q_out,
             cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (!in || !q_out != !in->q) return TFPA_EINVAL;
  const int64_t hd = kHeadDim;
  const int q_heads = in->q ? c->hq : 0;
  if (rows > 0) {
    const auto bad = [&](const void* p, int64_t stride, int64_t heads) {
      return !p || !aligned(p, 16) || stride % 8 || stride < heads * hd || stride > INT32_MAX;
    };
    if ((in->q && (bad(in->q, in->q_stride, c->hq) || !aligned(q_out, 16))) ||
        bad(in->k, in->k_stride, c->hkv) || bad(in->v, in->v_stride, c->hkv))
      return TFPA_EINVAL;
  }
  if ((in->q_weight && !aligned(in->q_weight, 16)) || (in->k_weight && !aligned(in->k_weight, 16)))
    return TFPA_EINVAL;
  if ((in->q_weight || in->k_weight) && (!std::isfinite(in->eps) || !(in->eps > 0.f)))
    return TFPA_EINVAL;
  if (in->rope_cos &&
      (!in->rope_sin || in->rope_n < 1 || !aligned(in->rope_cos, 16) ||
       !aligned(in->rope_sin, 16) || (in->rope_pos && !aligned(in->rope_pos, 4)) ||
       in->rot_dim < 16 || in->rot_dim > kHeadDim || in->rot_dim % 16))
    return TFPA_EINVAL;
  if ((int64_t)rows * (q_heads + c->hkv) > INT32_MAX - 16) return TFPA_EINVAL;
  if (in->q && rows > 0) {
    // q_out may be q itself, row for row; else it shares no memory with an input
    const int64_t out_bytes = (int64_t)rows * c->hq * hd * 2;
    const auto shares = [&](const void* p, int64_t bytes) {
      return p && overlap(q_out, out_bytes, p, bytes);
    };
    const auto shares_rows = [&](const void* p, int64_t stride, int64_t heads) {
      return shares(p, ((rows - 1) * stride + heads * hd) * 2);
    };
    const bool in_place = q_out == in->q && in->q_stride == c->hq * hd;
    if ((!in_place && shares_rows(in->q, in->q_stride, c->hq)) ||
        shares_rows(in->k, in->k_stride, c->hkv) || shares_rows(in->v, in->v_stride, c->hkv) ||
        shares(in->q_weight, hd * 4) || shares(in->k_weight, hd * 4))
      return TFPA_EINVAL;
    const int64_t table = in->rope_cos ? (int64_t)in->rope_n * (in->rot_dim / 2) * 4 : 0;
    if (in->rope_cos && (shares(in->rope_cos, table) || shares(in->rope_sin, table) ||
                         shares(in->rope_pos, (int64_t)rows * 4)))
      return TFPA_EINVAL;
  }
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  if (in->rope_cos && !in->rope_pos)
    for (const Run& r : runs)
      if (r.pos0 + r.nrows > in->rope_n) return TFPA_ERANGE;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  thread_local QkvParams p;
  size_t ri = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    const int32_t base = runs[ri].row0;
    int nr = 0;
    int32_t nrows = 0;
    while (ri < runs.size() && nr < kMaxRuns) {
      const Run& r = runs[ri++];
      const tfpa_seg& g = segs[r.seg];
      WriteRun& w = p.runs[nr++];
      w.page_table = g.page_table;
      w.k_dst = g.page_table ? c->k_pool : g.k_slab;
      w.v_dst = g.page_table ? c->v_pool : g.v_slab;
      w.row0 = r.row0 - base;
      w.nrows = r.nrows;
      w.pos0 = r.pos0;
      w.slab_cap = g.slab_cap;
      w.seq_len = g.seq_len;
      nrows = r.row0 + r.nrows - base;
    }
    if (in->q) {
      p.q = static_cast<const __nv_bfloat16*>(in->q) + base * in->q_stride;
      p.q_out = static_cast<__nv_bfloat16*>(q_out) + (int64_t)base * c->hq * hd;
    }
    p.k = static_cast<const __nv_bfloat16*>(in->k) + base * in->k_stride;
    p.v = static_cast<const __nv_bfloat16*>(in->v) + base * in->v_stride;
    p.q_stride = in->q_stride;
    p.k_stride = in->k_stride;
    p.v_stride = in->v_stride;
    p.q_weight = in->q_weight;
    p.k_weight = in->k_weight;
    p.eps = in->eps;
    p.rope_cos = in->rope_cos;
    p.rope_sin = in->rope_sin;
    p.rope_pos = in->rope_cos && in->rope_pos ? in->rope_pos + base : nullptr;
    p.rope_n = in->rope_n;
    p.rot_dim = in->rot_dim;
    p.interleaved = in->interleaved;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.err_flag = c->err_flag;
    p.nruns = nr;
    p.rows = nrows;
    p.q_heads = q_heads;
    p.hkv = c->hkv;
    p.num_pages = c->num_pages;
    const int32_t heads = nrows * (q_heads + c->hkv);
    p.wide = heads >= kWideHeads;
    const int32_t step = p.wide ? 4 : 1, kv_step = p.wide ? 2 : 1;   // heads of half a unit
    const int64_t units = (int64_t)nrows * ((q_heads + 2 * step - 1) / (2 * step) +
                                            (c->hkv + 2 * kv_step - 1) / (2 * kv_step));
    // one unit a warp, or what the GPU holds at once: two blocks of eight a SM
    p.warps = p.wide ? (int32_t)std::min<int64_t>(units, 16 * (int64_t)nsm) : (int32_t)units;
    record(14, base, nrows, nr, heads, p.warps, in->q ? base * in->q_stride : 0,
           in->q ? (int64_t)base * c->hq * hd : 0);
    if (!dry_run())
      if ((e = to_err(launch_write_qkv(p, c->dtype, stream)))) return e;
  }
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_write_qkv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                              const tfpa_qkv* in, const int32_t* row_seg, const int32_t* row_pos,
                              int32_t rows, void* q_out, cudaStream_t stream) {
  return no_throw([&] {
    return qkv_impl(cache, segs, nseg, in, row_seg, row_pos, rows, q_out, stream);
  });
}

// ------------------------------------------------------------ attention over selected blocks
namespace {

bool is_block(int32_t block) { return block == 64 || block == 128 || block == 256; }

// The bounds of the segments that a call's runs use.
int check_bounds(const tfpa_bounds* b, const tfpa_seg* segs, const std::vector<Run>& runs) {
  if (!b || !is_block(b->block)) return TFPA_EINVAL;
  for (const Run& r : runs) {
    const void* at = segs[r.seg].page_table ? b->pool : b->slabs ? b->slabs[r.seg] : nullptr;
    if (!at || !aligned(at, 16)) return TFPA_EINVAL;
  }
  return TFPA_OK;
}

void* bounds_of(const tfpa_bounds* b, const tfpa_seg* segs, int32_t seg) {
  return segs[seg].page_table ? b->pool : b->slabs[seg];
}

int bounds_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const tfpa_bounds* b,
                const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  if ((e = check_bounds(b, segs, runs))) return e;
  if (rows == 0) return TFPA_OK;
  int64_t all = 0;
  for (const Run& r : runs)
    all += (int64_t)c->hkv * ((r.pos0 + r.nrows - 1) / b->block - r.pos0 / b->block + 1);
  if (all > INT32_MAX) return TFPA_EINVAL;
  if ((e = check_device())) return e;
  thread_local BoundsParams p;
  size_t ri = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    const int32_t base = runs[ri].row0;
    int nr = 0;
    int32_t nrows = 0, items = 0;
    while (ri < runs.size() && nr < kMaxRuns) {
      const Run& r = runs[ri++];
      const tfpa_seg& g = segs[r.seg];
      BoundsRun& w = p.runs[nr++];
      w.page_table = g.page_table;
      w.k_base = g.page_table ? c->k_pool : g.k_slab;
      w.bounds = bounds_of(b, segs, r.seg);
      w.seq_len = g.seq_len;
      w.slab_cap = g.slab_cap;
      w.block0 = r.pos0 / b->block;
      w.item0 = items;
      items += (r.pos0 + r.nrows - 1) / b->block - w.block0 + 1;
      nrows = r.row0 + r.nrows - base;
    }
    p.err_flag = c->err_flag;
    p.nruns = nr;
    p.items = items;
    p.hkv = c->hkv;
    p.num_pages = c->num_pages;
    p.block = b->block;
    record(15, base, nrows, nr, items * c->hkv, items * c->hkv, 0, 0);
    if (!dry_run())
      if ((e = to_err(launch_key_bounds(p, c->dtype, stream)))) return e;
  }
  return TFPA_OK;
}

int select_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const tfpa_bounds* b,
                const void* q, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                int32_t nsel, int32_t sink, int32_t recent, int32_t* blocks,
                cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (rows > 0 && (!q || !aligned(q, 16) || !blocks || !aligned(blocks, 4))) return TFPA_EINVAL;
  if (nsel < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > nsel) return TFPA_EINVAL;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  if ((e = check_bounds(b, segs, runs))) return e;
  if ((int64_t)rows * c->hkv * 8 > INT32_MAX) return TFPA_EINVAL;
  for (const Run& r : runs)
    if ((r.pos0 + r.nrows - 1) / b->block + 1 > kSelectBlocks) return TFPA_ECAPACITY;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  thread_local SelectParams p;
  size_t ri = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    const int32_t base = runs[ri].row0;
    int nr = 0;
    int32_t nrows = 0, longest = 1;
    while (ri < runs.size() && nr < kMaxRuns) {
      const Run& r = runs[ri++];
      const tfpa_seg& g = segs[r.seg];
      SelRun& w = p.runs[nr++];
      longest = std::max(longest, r.nrows);
      w.page_table = g.page_table;
      w.bounds = bounds_of(b, segs, r.seg);
      w.row0 = r.row0 - base;
      w.nrows = r.nrows;
      w.pos0 = r.pos0;
      w.slab_cap = g.slab_cap;
      p.cap = std::max(p.cap, (r.pos0 + r.nrows - 1) / b->block + 1);
      nrows = r.row0 + r.nrows - base;
    }
    p.q = static_cast<const __nv_bfloat16*>(q) + (int64_t)base * c->hq * kHeadDim;
    p.blocks = blocks + (int64_t)base * c->hkv * nsel;
    p.err_flag = c->err_flag;
    p.nruns = nr;
    p.rows = nrows;
    p.hq = c->hq;
    p.hkv = c->hkv;
    p.group = c->hq / c->hkv;
    p.num_pages = c->num_pages;
    p.block = b->block;
    p.nsel = nsel;
    p.sink = sink;
    p.recent = recent;
    // Up to four rows of a run share the reads of the bounds; a cluster has a CTA
    // for each of them to choose in.  More CTAs while the GPU holds them (four a
    // SM, two with four rows, by their registers) and each has 32 blocks, eight a
    // warp of four (313 blocks: eight CTAs 7.6 us, four 8.8).
    p.rows_per = longest >= 3 ? 4 : longest;
    for (int i = 0; i < nr; ++i) {
      p.runs[i].group0 = p.groups;
      p.groups += (p.runs[i].nrows + p.rows_per - 1) / p.rows_per;
    }
    p.cap = (p.cap + 7) & ~7;           // whole eights of keys
    p.cluster = p.rows_per;
    const int64_t at_once = (p.rows_per == 1 ? 4 : 2) * nsm;
    while (p.cluster < 8 && (int64_t)p.groups * c->hkv * p.cluster * 2 <= at_once &&
           p.cap / (p.cluster * 2) >= 32)
      p.cluster *= 2;
    record(16, base, nrows, nr, p.groups * c->hkv, p.groups * c->hkv * p.cluster,
           (int64_t)base * c->hq * kHeadDim, (int64_t)base * c->hkv * nsel);
    if (!dry_run())
      if ((e = to_err(launch_select_blocks(p, stream)))) return e;
  }
  return TFPA_OK;
}

// Parts of a row's list: one for every 128 keys, up to eight.  A function of the
// list's length only, so a row's bytes do not depend on its batch.
int32_t block_parts(int32_t block, int32_t nsel) {
  return (int32_t)std::min<int64_t>(8, ((int64_t)nsel * (block / 64) + 1) / 2);
}

// Parts that a CTA takes one after the other: as few as let the launch have as many
// CTAs a SM as the kernel is built for, four with up to eight query vectors and two
// with more (by their registers; the states that wait take the fourth's shared memory
// over bf16 and e4m3 from four parts of five to eight vectors on, and at eight parts of
// fewer).  A part each, two, four and eight, in us, the rule's choice starred:
//   32 lists of 2,048 keys of 8 kv heads, 4 heads each (256 items):
//     bf16 48.6  42.8  37.2*  52.4;  e4m3 40.0  33.3  30.0*  42.3;  4 bits 40.3  33.1  30.1*  47.0
//   8 lists of 4,096 keys of 8 kv heads (64 items), 4 heads each:
//     bf16 26.6*  32.2  42.8  69.1;  e4m3 18.5*  23.8  30.6  46.0;  4 bits 16.4*  23.8  30.6  46.2
//   8 heads each: bf16 27.6*  33.3  45.7;  e4m3 19.3*  25.1  34.4;  4 bits 17.6*  24.7  32.0
//   16 heads each: bf16 38.0  33.0*  51.3;  e4m3 28.6  23.5*  38.2;  4 bits 28.4  23.2*  39.2
//   32 heads each (128 items): bf16 65.1  56.4  51.9*;  e4m3 52.2  43.7  39.3*;  4 bits 54.8  45.0  40.7*
int32_t cta_parts(int64_t items, int32_t parts, int32_t group, int nsm) {
  const int64_t at_once = (group <= 8 ? 4 : 2) * (int64_t)nsm;
  int32_t k = 1;
  while (k < parts && items * ((parts + k - 1) / k) > at_once) k *= 2;
  return std::min(k, parts);
}

constexpr int32_t kMaxListed = 1 << 24;   // entries of a list, at most

int blocks_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* q,
                const int32_t* row_seg, const int32_t* row_pos, int32_t rows, int32_t block,
                int32_t nsel, const int32_t* blocks, float scale, void* out, float* lse,
                cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (rows > 0 && (!q || !aligned(q, 16) || !blocks || !aligned(blocks, 4) || !out ||
                   !aligned(out, 16) || (lse && !aligned(lse, 4))))
    return TFPA_EINVAL;
  if (!is_block(block) || nsel < 1 || nsel > kMaxListed || !std::isfinite(scale) ||
      !(scale > 0.f))
    return TFPA_EINVAL;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  const int32_t parts = block_parts(block, nsel);
  const int G = c->hq / c->hkv;
  const int64_t qtiles = G <= 8 ? 1 : (G + 15) / 16;
  if ((int64_t)rows * c->hkv * qtiles * parts > INT32_MAX) return TFPA_EINVAL;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device())) return e;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  thread_local BlocksParams p;
  size_t ri = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    const int32_t base = runs[ri].row0;
    int nr = 0;
    int32_t nrows = 0;
    SourceSet ss;
    while (ri < runs.size() && nr < kMaxRuns) {
      const int src = ss.add(segs, runs[ri].seg);
      if (src < 0) break;
      const Run& r = runs[ri++];
      const tfpa_seg& g = segs[r.seg];
      BlocksRun& w = p.runs[nr++];
      w.src = src;
      w.page_table = g.page_table;
      w.k_base = g.page_table ? c->k_pool : g.k_slab;
      w.v_base = g.page_table ? c->v_pool : g.v_slab;
      w.row0 = r.row0 - base;
      w.nrows = r.nrows;
      w.pos0 = r.pos0;
      w.slab_cap = g.slab_cap;
      nrows = r.row0 + r.nrows - base;
    }
    const int64_t hd = (int64_t)c->hq * kHeadDim;
    p.q = static_cast<const __nv_bfloat16*>(q) + base * hd;
    p.blocks = blocks + (int64_t)base * c->hkv * nsel;
    p.out = static_cast<__nv_bfloat16*>(out) + base * hd;
    p.lse = lse ? lse + (int64_t)base * c->hq : nullptr;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.err_flag = c->err_flag;
    p.nruns = nr;
    p.rows = nrows;
    p.hq = c->hq;
    p.hkv = c->hkv;
    p.group = G;
    p.num_pages = c->num_pages;
    p.block = block;
    p.nsel = nsel;
    p.parts = parts;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (c->dtype != TFPA_FP4_E2M1) {
      const bool fp8 = c->dtype == TFPA_FP8_E4M3;
      int32_t nsrc;
      if ((e = fill_maps(c, segs, ss, fp8, fp8 ? 128 : 64, fp8 ? 64 : 32, p.maps, nsrc))) return e;
    }
    const int32_t items = (int32_t)(nrows * c->hkv * qtiles);
    p.cta_parts = cta_parts(items, parts, G, nsm);
    p.ctas = (parts + p.cta_parts - 1) / p.cta_parts;
    record(17, base, nrows, nr, items, items * p.ctas, base * hd, base * hd);
    if (!dry_run())
      if ((e = to_err(launch_decode_blocks(p, c->dtype, stream)))) return e;
  }
  return TFPA_OK;
}

}  // namespace

extern "C" int tfpa_key_bounds(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                               const tfpa_bounds* bounds, const int32_t* row_seg,
                               const int32_t* row_pos, int32_t rows, cudaStream_t stream) {
  return no_throw(
      [&] { return bounds_impl(cache, segs, nseg, bounds, row_seg, row_pos, rows, stream); });
}

extern "C" int tfpa_select_blocks(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                                  const tfpa_bounds* bounds, const void* q,
                                  const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                                  int32_t nsel, int32_t sink, int32_t recent, int32_t* blocks,
                                  cudaStream_t stream) {
  return no_throw([&] {
    return select_impl(cache, segs, nseg, bounds, q, row_seg, row_pos, rows, nsel, sink, recent,
                       blocks, stream);
  });
}

extern "C" int tfpa_decode_blocks(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                                  const void* q, const int32_t* row_seg, const int32_t* row_pos,
                                  int32_t rows, int32_t block, int32_t nsel,
                                  const int32_t* blocks, float softmax_scale, void* out,
                                  float* lse, cudaStream_t stream) {
  return no_throw([&] {
    return blocks_impl(cache, segs, nseg, q, row_seg, row_pos, rows, block, nsel, blocks,
                       softmax_scale, out, lse, stream);
  });
}

extern "C" int tfpa_call(const tfpa_call_args* c) {
  if (!c) return TFPA_EINVAL;
  switch (c->op) {
    case TFPA_OP_ROPE_TABLE:
      return tfpa_rope_table(c->u.rope.spec, c->u.rope.first, c->rows, c->u.rope.cos,
                             c->u.rope.sin, c->stream);
    case TFPA_OP_WRITE_QKV:
      return tfpa_write_qkv(c->cache, c->segs, c->nseg, &c->u.qkv, c->row_seg, c->row_pos,
                            c->rows, c->out, c->stream);
    case TFPA_OP_KEY_BOUNDS:
      return tfpa_key_bounds(c->cache, c->segs, c->nseg, c->bounds, c->row_seg, c->row_pos,
                             c->rows, c->stream);
    case TFPA_OP_SELECT_BLOCKS:
      return tfpa_select_blocks(c->cache, c->segs, c->nseg, c->bounds, c->q, c->row_seg,
                                c->row_pos, c->rows, c->nsel, c->sink, c->recent, c->blocks,
                                c->stream);
    case TFPA_OP_DECODE_BLOCKS:
      return tfpa_decode_blocks(c->cache, c->segs, c->nseg, c->q, c->row_seg, c->row_pos,
                                c->rows, c->block, c->nsel, c->blocks, (float)c->softmax_scale,
                                c->out, c->lse, c->stream);
    default:
      return TFPA_EINVAL;
  }
}

extern "C" void tfpa_set_launch_hook(tfpa_launch_hook hook, void* user, int dry_run_flag) {
  g_hook_user.store(user, std::memory_order_relaxed);
  g_hook_dry.store(hook ? dry_run_flag : 0, std::memory_order_relaxed);
  g_hook_fn.store(hook, std::memory_order_release);
}

extern "C" const char* tfpa_strerror(int code) {
  switch (code) {
    case TFPA_OK: return "ok";
    case TFPA_EINVAL: return "invalid argument (dims, dtype, null pointer or alignment)";
    case TFPA_ERANGE: return "segment, position or page id out of range";
    case TFPA_ECAPACITY: return "scratch capacity exceeded (rows or splits)";
    case TFPA_ECUDA: return "CUDA call or launch failed";
    case TFPA_EDEVICE: return "current device is not sm_100-family";
    case TFPA_ELANEMEM: return "the page pool cannot hold the claim now (wait for releases)";
    case TFPA_ENOMEM: return "host memory ran out inside the call";
    default: return "unknown error";
  }
}

extern "C" const char* tfpa_version(void) { return "tfpa 0.1 (sm_103a)"; }

// ------------------------------------------------------------ prefill
namespace {
constexpr int kPrefillTileRows = 128;

int prefill_impl(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg, const void* q,
                 const int32_t* row_seg, const int32_t* row_pos, int32_t rows, float scale,
                 int32_t max_rows_per_launch, void* out, float* lse, cudaStream_t stream) {
  int e;
  if ((e = check_cache(c)) || (e = check_segs(c, segs, nseg))) return e;
  if (rows > 0 && (!q || !aligned(q, 16) || !out || !aligned(out, 16))) return TFPA_EINVAL;
  if (max_rows_per_launch < 0 || !std::isfinite(scale) || !(scale > 0.f)) return TFPA_EINVAL;
  thread_local std::vector<Run> runs;   // reused by every call of this thread
  if ((e = build_runs(segs, nseg, row_seg, row_pos, rows, runs))) return e;
  if (rows == 0) return TFPA_OK;
  if ((e = check_device()) || (e = check_tma_source(q))) return e;
  const int kv = c->dtype;
  const bool fp8 = kv == kKvFp8;
  const int G = c->hq / c->hkv;
  const int npairs = (G + 1) / 2;
  const int32_t cap = max_rows_per_launch > 0 ? max_rows_per_launch : INT32_MAX;
  const int nsm = sm_count();
  if (nsm < 1) return TFPA_ECUDA;
  const size_t hd = (size_t)c->hq * kHeadDim;
  thread_local PrefillParams p;
  size_t ri = 0;
  int32_t taken = 0;
  while (ri < runs.size()) {
    std::memset(&p, 0, sizeof(p));
    SourceSet ss;
    const int32_t base = runs[ri].row0 + taken;
    int32_t nrows = 0, tiles = 0;
    int nr = 0;
    while (ri < runs.size() && nr < kMaxRuns && nrows < cap) {
      const Run& r = runs[ri];
      const int src = ss.add(segs, r.seg);
      if (src < 0) break;
      const int32_t take = std::min(r.nrows - taken, cap - nrows);
      RunInfo& info = p.runs[nr++];
      fill_run(info, segs[r.seg], src, nrows, take, r.pos0 + taken);
      info.item0 = tiles;
      tiles += c->hkv * npairs * ((take + kPrefillTileRows - 1) / kPrefillTileRows);
      nrows += take;
      taken += take;
      if (taken == r.nrows) {
        ++ri;
        taken = 0;
      }
    }
    if (kv == kKvFp4)
      p.nsrc = fill_bases(c, segs, ss, p.k_base, p.v_base);
    else if ((e = fill_maps(c, segs, ss, fp8, fp8 ? 128 : 64, 128, p.maps, p.nsrc)))
      return e;
    if ((e = get_qmap(static_cast<const __nv_bfloat16*>(q) + (size_t)base * hd, c->hq, nrows, 1,
                      kPrefillTileRows,
                      &p.qmap)))
      return e;
    p.q = static_cast<const __nv_bfloat16*>(q) + (size_t)base * hd;
    p.out = static_cast<__nv_bfloat16*>(out) + (size_t)base * hd;
    p.lse = lse ? lse + (size_t)base * c->hq : nullptr;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.err_flag = c->err_flag;
    p.nruns = nr;
    p.n_tiles = tiles;
    p.hq = c->hq;
    p.hkv = c->hkv;
    p.group = G;
    p.num_pages = c->num_pages;
    p.rows = nrows;
    p.scale_log2 = scale * 1.4426950408889634f;
    // A cluster of two CTAs per tile (each takes half of the tile's key
    // tiles), heaviest tiles first.
    record(3, base, nrows, nr, tiles, 2 * tiles, (int64_t)base * hd, (int64_t)base * hd);
    if (!dry_run())
      if ((e = to_err(launch_prefill(p, kv, tiles, stream)))) return e;
  }
  return TFPA_OK;
}
}  // namespace

extern "C" int tfpa_prefill(const tfpa_cache* c, const tfpa_seg* segs, int32_t nseg,
                            const void* q, const int32_t* row_seg, const int32_t* row_pos,
                            int32_t rows, float scale, int32_t max_rows_per_launch, void* out,
                            float* lse, cudaStream_t stream) {
  return no_throw([&] {
    return prefill_impl(c, segs, nseg, q, row_seg, row_pos, rows, scale, max_rows_per_launch, out,
                        lse, stream);
  });
}
