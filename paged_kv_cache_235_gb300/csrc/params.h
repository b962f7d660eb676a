// Kernel launch parameters shared by the host planner and the kernels.
//
// A call's rows are grouped into runs: consecutive rows of one segment at
// consecutive positions.  Everything a kernel needs about a run travels in
// the launch parameters (passed by value, so a launch captured in a graph
// keeps them); only the bulk data (pages, tables, q, out, scratch) is in
// device memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace tfpa {

constexpr int kPage = 256;          // positions per page
constexpr int kHeadDim = 128;       // head size
constexpr int kMaxSplits = 32;      // split-K partials per (row, head), at most
constexpr int kMaxRuns = 64;        // runs per launch
constexpr int kMaxSlabs = 15;       // slab streams per launch (+1 source for the pool)
constexpr int kMaxSources = kMaxSlabs + 1;
constexpr int kMaxDecodeGrid = 256;  // CTAs of one decode partial launch, at most

// Element type of a cache (the values of tfpa_kv_dtype).
enum KvType : int { kKvBf16 = 0, kKvFp8 = 1, kKvFp4 = 2 };
// A decode partial launch over a 4-bit cache whose runs have more than eight
// query vectors per kv head.
constexpr int kKvFp4Wide = 3;

// A 4-bit cache: storage row R (pool: (page * hkv + g) * 256 + position %
// 256; slab: g * slab_cap + position) lies in half-block R / 128, which
// holds its 128 rows' codes ([128][64] bytes) and then their scales
// ([128][8] bytes): one aligned run of 9,216 bytes that a single bulk copy
// brings into shared memory.
constexpr int kHalfRows = 128;
constexpr int kFp4CodeBytes = 64;        // 128 e2m1 codes
constexpr int kFp4ScaleBytes = 8;        // an e4m3 scale per 16 head dims
constexpr int kFp4ScaleOff = kHalfRows * kFp4CodeBytes;
constexpr int kFp4HalfBytes = kHalfRows * (kFp4CodeBytes + kFp4ScaleBytes);

// TMA descriptors of one K/V source: the page pool (source 0) or a slab.
struct KVMaps {
  CUtensorMap k;
  CUtensorMap v;
};

struct RunInfo {
  const int32_t* page_table;  // device; nullptr => slab source
  int32_t src;                // index into maps[]
  int32_t seq_len;
  int32_t row0;               // first row, relative to this launch
  int32_t nrows;
  int32_t pos0;               // position of the first row
  int32_t nsplit;             // decode and verify: splits of this stream
  int32_t pps;                // decode and verify: pages per split
  int32_t item0;              // first work item of this run
  int32_t slab_cap;           // slab capacity in positions (slab runs)
  int32_t pad_;
};

// The parts of a launch that change as streams grow (lengths, positions,
// split counts, item and CTA ranges).  A launch reads them from its own
// parameters, or, for a plan in device mode, from a device copy (`dyn`),
// which lets a captured launch be replayed step after step with new data.
struct DecodeDyn {
  RunInfo runs[kMaxRuns];
  int32_t nruns;
  int32_t n_items;
  int32_t pad_[2];
  // CTA b takes the work items [cta_item0[b], cta_item0[b + 1]), ranges the
  // host balances by the items' key stages.
  int32_t cta_item0[kMaxDecodeGrid + 1];
};

struct DecodeParams {
  KVMaps maps[kMaxSources];
  DecodeDyn d;
  const DecodeDyn* dyn;       // device copy of d to read instead, or nullptr
  const __nv_bfloat16* q;     // rows of this launch: [rows][hq][128]
  const uint64_t* anc;        // rows of this launch: ancestor masks, or nullptr (causal)
  float* part_o;              // [cap_rows][hq][max_splits][128]
  float* part_ml;             // [cap_rows][hq][max_splits][2]
  const float* k_scale;       // fp8: [hkv]
  const float* v_scale;
  int32_t* err_flag;
  // Append (k_rows != nullptr): the rows' new K and V ([rows][hkv][128]
  // bf16, rows of this launch) are stored by the CTAs whose keys include
  // them, before they read them; a source's K / V base is where its rows
  // go (pool: [num_pages][hkv][256][128], slab: [hkv][slab_cap][128]).
  const __nv_bfloat16* k_rows;
  const __nv_bfloat16* v_rows;
  // A 4-bit cache is read through these bases too (bulk copies, no maps).
  void* k_base[kMaxSources];
  void* v_base[kMaxSources];
  // Merge in the partial kernel (arrive != nullptr): per (row, head) of a
  // group's first query vector, the splits finished so far; the last CTA
  // to finish one merges the group into out / lse (rows of this launch).
  uint32_t* arrive;           // [cap_rows][hq], scratch rows of this launch
  __nv_bfloat16* out;         // [rows][hq][128]
  float* lse;                 // [rows][hq] or nullptr
  int32_t nsrc;
  int32_t hq, hkv, group;     // group = hq / hkv
  int32_t max_splits;
  int32_t num_pages;
  int32_t rows;
  float scale_log2;           // softmax_scale * log2(e)
};

struct MergeRun {
  int32_t row0;
  int32_t nrows;
  int32_t nsplit;
  int32_t pad_;
};

struct MergeDyn {
  MergeRun runs[kMaxRuns * 2];
  int32_t nruns;
  int32_t rows;
  int32_t pad_[2];
};

struct MergeParams {
  MergeDyn d;
  const MergeDyn* dyn;        // device copy of d to read instead, or nullptr
  const float* part_o;
  const float* part_ml;
  __nv_bfloat16* out;         // rows of this launch: [rows][hq][128]
  float* lse;                 // [rows][hq] or nullptr
  int32_t hq;
  int32_t max_splits;
};

struct WriteRun {
  const int32_t* page_table;  // nullptr => slab
  void* k_dst;                // pool base or slab base
  void* v_dst;
  int32_t row0;               // first row of the run, relative to this launch
  int32_t nrows;
  int32_t pos0;
  int32_t slab_cap;
  int32_t seq_len;
  int32_t pad_;
};

struct WriteDyn {
  WriteRun runs[kMaxRuns];
  int32_t nruns;
  int32_t rows;
  int32_t pad_[2];
};

struct WriteParams {
  WriteDyn d;
  const WriteDyn* dyn;        // device copy of d to read instead, or nullptr
  const __nv_bfloat16* k_rows;  // [rows][hkv][128], rows of this launch
  const __nv_bfloat16* v_rows;
  const float* k_scale;
  const float* v_scale;
  int32_t* err_flag;
  // Rotary store (nullptr rope_cos: plain store): K is rotated by rope_pos[row]
  // (nullptr: the storage position) with the caller's cos/sin [rope_n][64].
  const float* rope_cos;
  const float* rope_sin;
  const int32_t* rope_pos;    // rows of this launch
  int32_t rope_n;
  int32_t hkv;
  int32_t num_pages;
  int32_t kv;                 // KvType
};

// Keep: stored rows copied between positions of a stream (all kv heads).
constexpr int kMaxKeep = 256;
struct KeepPair {
  const int32_t* page_table;  // nullptr => slab
  void* k_slab;
  void* v_slab;
  int32_t slab_cap;
  int32_t src;
  int32_t dst;
  int32_t pad_;
};

struct KeepParams {
  KeepPair pairs[kMaxKeep];
  void* k_pool;
  void* v_pool;
  int32_t* err_flag;
  int32_t n;
  int32_t hkv;
  int32_t num_pages;
  int32_t row_bytes;          // 256 (bf16), 128 (e4m3) or 72 (4 bits: codes and scales)
};

// Prefill: one work tile = (run, kv head g, query-head pair, 128 rows).
// The same kernel in verify mode (decode runs of many query vectors, on
// tensor cores): one work tile = (run, kv head g, 128 / G rows, key split);
// its query vectors (rows x the group's G heads, at most 128) form one Q
// tile that both MMA slots read, slot A taking the split's even key tiles
// and slot B the odd ones, each leaving its own split partial.
constexpr int kVerifyVectors = 128;
struct PrefillParams {
  KVMaps maps[kMaxSources];
  CUtensorMap qmap;           // q as 3D [rows][hq][128], 128B swizzle; box 64 x 1 x 128
                              // (prefill) or 64 x G x (128 / G) (verify)
  RunInfo runs[kMaxRuns];     // item0 = first tile of the run
  const __nv_bfloat16* q;     // [rows][hq][128]
  __nv_bfloat16* out;         // prefill
  float* lse;                 // prefill, or nullptr
  const uint64_t* anc;        // verify: the rows' ancestor masks, or nullptr (causal)
  float* part_o;              // verify: [rows][hq][max_splits][128]
  float* part_ml;             // verify: [rows][hq][max_splits][2]
  const float* k_scale;
  const float* v_scale;
  int32_t* err_flag;
  int32_t nruns;
  int32_t nsrc;
  int32_t n_tiles;
  int32_t hq, hkv, group;
  int32_t num_pages;
  int32_t rows;
  int32_t max_splits;         // verify
  float scale_log2;
  const void* k_base[kMaxSources];   // 4-bit caches: read by bulk copies, no maps
  const void* v_base[kMaxSources];
};

// Page-table staging: ids written into a device page table on the stream.
constexpr int kMaxStage = 2048;
struct StageParams {
  int32_t* table;
  int32_t first;
  int32_t n;
  int32_t ids[kMaxStage];
};

// Save / restore of a stream's stored rows [p0, p1) to / from an image laid
// out [K, V][hkv][p1 - p0][row]; 4-bit rows: every row's codes, then every
// row's scales, each in that order.
struct CopyParams {
  const int32_t* page_table;  // nullptr => slab
  void* k_base;               // pool or slab
  void* v_base;
  uint8_t* image;
  int32_t* err_flag;
  int32_t slab_cap;
  int32_t p0, p1;
  int32_t page0;              // first page of the range
  int32_t hkv;
  int32_t num_pages;
  int32_t row_bytes;          // 256 (bf16), 128 (e4m3) or 72 (4 bits)
  int32_t restore;            // 0: cache -> image, 1: image -> cache
};

// Accumulated attention weight: the segments of a launch, each with its runs.
struct MassSeg {
  const int32_t* page_table;  // nullptr => slab
  const void* k_base;         // pool or slab
  int32_t index;              // the segment's index in the call (its planes of mass)
  int32_t seq_len;
  int32_t slab_cap;
  int32_t item0;              // first key tile of the segment
  int32_t run0, nruns;
  float decay;                // 1 when an earlier launch of the call has applied it
  int32_t src;                // index into maps[]
};
struct MassRun {
  int32_t row0;               // row of the call
  int32_t nrows;
  int32_t pos0;
};
struct MassParams {
  CUtensorMap maps[kMaxSources];   // K of each source (bf16, e4m3)
  MassSeg segs[kMaxRuns];
  MassRun runs[kMaxRuns];
  const __nv_bfloat16* q;     // [rows][hq][128]
  const float* lse;           // [rows][hq]
  float* mass;                // [nseg][hkv][mass_cap]
  const float* k_scale;
  int32_t* err_flag;
  int32_t nsegs;
  int32_t dbufs;              // 4 if no segment has more than 128 query vectors, else 2
  int32_t tiles;              // key tiles: hkv * ceil(seq_len / 128) of every segment
  int32_t hq, hkv, group;
  int32_t num_pages;
  int32_t mass_cap;
  float scale_log2;
};

// Eviction.
constexpr int kMaxEvictSegs = 64;
constexpr int32_t kSelectKeys = 49152;   // order keys that a select block's shared memory holds
// Slots of one of `blocks` select blocks (whole runs of 128).
__host__ __device__ inline int32_t select_chunk(int32_t seq_len, int32_t blocks) {
  return (int32_t)((((int64_t)seq_len + blocks - 1) / blocks + 127) & ~(int64_t)127);
}
constexpr int32_t kNextPosHeld = -1;     // next_pos: one past the largest key_pos held
struct EvictSeg {
  const int32_t* page_table;  // nullptr => slab
  void* k_base;               // pool or slab
  void* v_base;
  int32_t index;              // the segment's index in the call
  int32_t seq_len;
  int32_t keep;
  int32_t next_pos;
  int32_t slab_cap;
  int32_t pad_;
};
struct EvictParams {
  EvictSeg segs[kMaxEvictSegs];
  float* mass;                // [nseg][hkv][mass_cap]
  int32_t* key_pos;           // the same, or nullptr (a slot's position is its index)
  int32_t* moves;             // [nseg][hkv][mass_cap + 4]
  int32_t* err_flag;
  int32_t nsegs;
  int32_t hkv;
  int32_t num_pages;
  int32_t mass_cap;
  int32_t sink, recent;
  int32_t grid_x;             // move blocks of one (segment, kv head)
  int32_t cluster;            // select blocks of one (segment, kv head)
  int32_t key_slots;          // keys that one of them can keep in shared memory
};

// Launchers (defined next to their kernels).
cudaError_t launch_key_mass(const MassParams& p, int kv, int grid, cudaStream_t s);
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s);
cudaError_t launch_evict_move(const EvictParams& p, int kv, cudaStream_t s);
cudaError_t launch_write_kv(const WriteParams& p, cudaStream_t s);
// The rows' stored K and V as bf16, into p.k_rows / p.v_rows.
cudaError_t launch_read_kv(const WriteParams& p, cudaStream_t s);
cudaError_t launch_keep(const KeepParams& p, cudaStream_t s);
cudaError_t launch_stage(const StageParams& p, cudaStream_t s);
cudaError_t launch_copy(const CopyParams& p, int npages, cudaStream_t s);
cudaError_t launch_decode_partial(const DecodeParams& p, int kv, int grid, cudaStream_t s);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t s);
// Prefill launches a cluster of two CTAs per tile; verify one CTA per tile.
cudaError_t launch_prefill(const PrefillParams& p, int kv, int tiles, cudaStream_t s);
cudaError_t launch_verify(const PrefillParams& p, int kv, int tiles, cudaStream_t s);

}  // namespace tfpa
