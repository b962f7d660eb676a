/*
 * tfpa: GQA attention over a paged KV cache, for GB300 (sm_103a).
 *
 * Keys and values live in 256-position pages drawn from one shared pool; a
 * stream reaches its pages through its own page table (TensorFold PR #2011,
 * "What this changes": every stream takes 256-position pages from the core
 * pool).  A stream may instead hold a contiguous slab; both are read with one
 * arithmetic, so a stream's output is the same bytes paged or not, batched or
 * alone (PR #1373, "What changes"; Issue #1344, "Conclusion").
 *
 * Layouts (all row-major, element = bf16 or one e4m3 byte; a 4-bit cache holds
 * blocks of codes and scales in place of [256][128] elements, see
 * TFPA_FP4_BLOCK):
 *   pool  K, V : [num_pages][hkv][256][128]   key j of kv head g of a paged
 *                stream is pool[PT[j/256]][g][j%256]  (PR #2011, review
 *                "Is paged output the same as windowed output?": base
 *                PT[k0/256]*PS + (hk*256 + k0%256)*D)
 *   slab  K, V : [hkv][slab_cap][128]          key j of kv head g is slab[g][j]
 *   q, out     : bf16 [rows][hq][128]
 *   k_rows, v_rows (KV write input): bf16 [rows][hkv][128]
 *   lse        : float [rows][hq], natural log, nullable
 * Query head h reads kv head h / (hq/hkv).
 *
 * Rows and segments.  A call covers `rows` query rows; row r belongs to
 * segment row_seg[r] (an index into `segs`) and sits at cache position
 * row_pos[r]; it attends to keys 0..row_pos[r] of its segment (causal).
 * Rows of one segment should be contiguous with consecutive positions (a
 * decode/verify group or a prompt chunk); other orders are accepted and run
 * as more, smaller groups.
 *
 * Memory and ownership.  Every buffer is allocated by the caller.  Pointers
 * marked DEVICE are device memory of the current device; HOST arrays are read
 * during the call only and not retained.  The library allocates no device
 * memory, keeps no state between calls except host-side caches (TMA tensor
 * maps, per host thread; each device's SM count) and the plans a caller
 * creates (a plan may own a CUDA graph, see tfpa_plan_capture), and never
 * synchronises the stream: all work is enqueued on `stream`.
 *
 * Pinned host memory on the decode path.  Where DEVICE is marked below for
 * q, k_rows, v_rows, out or lse of tfpa_decode, tfpa_decode_tree,
 * tfpa_decode_append, tfpa_merge, tfpa_write_kv and tfpa_write_kv_rope (and
 * their plans), and for a device-mode plan's buffer, page-locked host memory
 * mapped at its own address (cudaHostAlloc / cudaMallocHost under unified
 * addressing, or cudaHostRegister with cudaHostRegisterMapped) may stand in:
 * the kernels read and write it with plain loads and stores over the host
 * link (NVLink-C2C on a Grace-Blackwell node), with no copy-engine copy.
 * Data the host writes there before it enqueues a call is what the call
 * reads; results are the host's once the stream has passed the call.  A
 * slice with rows for the tensor-core verify path and tfpa_prefill load q
 * by TMA from device memory only: host memory there returns TFPA_EINVAL.
 * The K/V rows that tfpa_read_kv writes and the q and lse that tfpa_key_mass
 * reads may be host memory too; mass, key_pos and moves are device memory.
 * Memory that is not page-locked is not supported (and not checked).
 *
 * Threads.  Calls may be made from several host threads at once, on any
 * streams and devices: each thread builds its launch parameters in its own
 * buffers and no call takes a lock on that path (the pool ledger and the
 * static-scratch address lookup lock their own state).  Work enqueued on
 * different streams runs concurrently on the GPU, so two calls must not
 * write the same output, scratch or cache rows at once.
 * tfpa_set_launch_hook must not run while another call is in progress.
 *
 * Errors.  Every call returns TFPA_OK (0) or a negative code below and
 * enqueues nothing on error.  Kernels never trap: a page id outside
 * [0, num_pages) found on the device is skipped (its keys take no part in
 * attention; the KV write skips its rows) and sets bit 1 of cache->err_flag
 * (if non-NULL); a wait inside a kernel that gives up sets bit 2.
 */
#ifndef TFPA_H
#define TFPA_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TFPA_PAGE 256          /* positions per page (compile-time constant) */
#define TFPA_HEAD_DIM 128      /* the only head size built                  */
#define TFPA_MAX_SPLITS 32     /* split-K partials per (row, head), at most */

enum {
  TFPA_OK = 0,
  TFPA_EINVAL = -1,      /* bad dims, dtype, NULL pointer, misalignment, or a
                            softmax_scale that is not finite and positive   */
  TFPA_ERANGE = -2,      /* a position, segment or (host-mirrored) page id out of range */
  TFPA_ECAPACITY = -3,   /* scratch too small for the requested rows/splits */
  TFPA_ECUDA = -4,       /* a CUDA runtime/driver call or a launch failed    */
  TFPA_EDEVICE = -5,     /* current device is not sm_100-family (tcgen05)    */
  TFPA_ELANEMEM = -6,    /* the page pool cannot hold the claim now: wait     */
  TFPA_ENOMEM = -7       /* host memory ran out inside the call               */
};

typedef enum { TFPA_BF16 = 0, TFPA_FP8_E4M3 = 1, TFPA_FP4_E2M1 = 2 } tfpa_kv_dtype;

/* A 4-bit cache (TFPA_FP4_E2M1): each value is an e2m1 code (0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives) times the e4m3 scale of its 16 head dims
 * times k_scale[g] / v_scale[g]: 72 bytes a row and kv head, K or V.  Where
 * the layouts above say [256][128] elements, a page of one kv head is one
 * block of TFPA_FP4_BLOCK bytes: two half-blocks of 128 positions, each
 * [128][64] bytes of codes (byte i of a row: dim 2i in the low nibble, 2i + 1
 * in the high one) and then [128][8] scale bytes.  So a pool is
 * [num_pages][hkv][TFPA_FP4_BLOCK] bytes and a slab
 * [hkv][slab_cap / 256][TFPA_FP4_BLOCK].
 *   Store (tfpa_write_kv, tfpa_write_kv_rope, tfpa_decode_append): with x the
 * value in float32 (a NaN counts as 0), each product and quotient rounded to
 * float32, block scale = e4m3(max |x| / (6 k_scale[g])) and code =
 * e2m1(x / (scale k_scale[g])), both rounded to nearest even and saturating;
 * a block whose scale rounds to 0 holds zeros.  k_scale[g] = max |x| / 2688
 * over a head's values uses the scales' whole range.  The stored form has no
 * NaN and no infinity.
 *   A save / restore image holds all rows' codes, [K, V][hkv][p1 - p0][64]
 * bytes, and then all rows' scales, [K, V][hkv][p1 - p0][8]. */
#define TFPA_FP4_BLOCK 18432

/* One stream (a segment of the call). */
typedef struct {
  int32_t seq_len;                /* valid keys, >= 1 (includes rows written by this round) */
  const int32_t* page_table;      /* DEVICE int32[ceil(seq_len/256)]; NULL => slab stream   */
  const int32_t* page_table_host; /* optional HOST mirror, checked against num_pages        */
  void* k_slab;                   /* DEVICE [hkv][slab_cap][128], slab streams only          */
  void* v_slab;
  int32_t slab_cap;               /* slab capacity in positions, multiple of 256            */
} tfpa_seg;

/* One layer's KV cache. */
typedef struct {
  tfpa_kv_dtype dtype;
  int32_t hq, hkv, head_dim;      /* hq % hkv == 0, head_dim == 128                        */
  void* k_pool;                   /* DEVICE [num_pages][hkv][256][128], 1024-byte aligned;  */
  void* v_pool;                   /*   may be NULL when no segment is paged                 */
  int32_t num_pages;
  const float* k_scale;           /* DEVICE float[hkv], fp8: value = e4m3 * scale; fp4: see above */
  const float* v_scale;
  int32_t* err_flag;              /* optional DEVICE int32: OR-ed with 1 on a bad page id,
                                     4 on a rotary position outside the table */
} tfpa_cache;

/* Split-K scratch for decode partials (float32).
 *   part_o  : DEVICE [cap_rows][hq][max_splits][128]  unnormalised outputs o
 *   part_ml : DEVICE [cap_rows][hq][max_splits][2]    (m, l): running max of the
 *             scores in log2 units (score * log2(e)) and the sum of 2^(s2 - m)
 *   arrive  : optional DEVICE uint32[cap_rows][hq], all zero before the first
 *             call.  With it, tfpa_decode merges a slice inside the partial
 *             kernel when each of its streams has at most 4 splits
 *             (seq_len <= 1,024): the last CTA to finish a split of a group
 *             of query vectors (counted here) merges that group's splits in
 *             split order, with the merge kernel's arithmetic, so the output
 *             bytes are those of the separate merge; a launch leaves every
 *             counter at zero again.  Longer streams, tfpa_decode_tree,
 *             plans in device mode and slices with rows for the tensor-core
 *             verify path keep the separate merge (a group's in-kernel merge
 *             runs on one SM at the kernel's tail: for 32 splits it was
 *             measured slower than the separate launch).  After a call that
 *             set the cache's err_flag the counters may be left non-zero:
 *             zero them before the next call.  NULL: always the separate
 *             merge. */
typedef struct {
  float* part_o;
  float* part_ml;
  int32_t cap_rows;               /* rows one partial launch can hold                      */
  int32_t max_splits;             /* >= tfpa_num_splits(seq_len) of every segment used     */
  uint32_t* arrive;
} tfpa_scratch;

/* KV write with rotary position embedding: tfpa_write_kv, with each row's K
 * rotated before it is stored.  The pages list "rope stores" among the paged
 * KV store's checks (PR #1373 review) without defining the rotation; this
 * reading is used: for i < 64, with c = rope_cos[t][i], s = rope_sin[t][i]
 * and t the row's rotary position,
 *   k'[i] = k[i] c - k[i+64] s,   k'[i+64] = k[i+64] c + k[i] s,
 * each product, difference and sum rounded to float32 (no fused multiply-
 * add), then stored as bf16 (round to nearest even) or as tfpa_write_kv
 * stores an fp8 value.  V is stored as tfpa_write_kv stores it.
 *   rope_pos : DEVICE int32[rows], 4-byte aligned, each in [0, rope_n); or
 *              NULL: the storage positions row_pos (then checked on the host,
 *              TFPA_ERANGE).  A device position outside the table leaves the
 *              row unwritten and ORs 4 into cache->err_flag.  The rotary
 *              position may differ from the storage position (a draft-tree
 *              node is rotated by its depth and stored at its index).
 *   rope_cos, rope_sin : DEVICE float32 [rope_n][64], 16-byte aligned.
 * Sliced like the rows.  TFPA_EINVAL for a NULL or misaligned table. */
int tfpa_write_kv_rope(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                       const void* k_rows, const void* v_rows, const int32_t* row_seg,
                       const int32_t* row_pos, const int32_t* rope_pos, const float* rope_cos,
                       const float* rope_sin, int32_t rope_n, int32_t rows,
                       cudaStream_t stream);

/* Keep: copy stored K/V rows (every kv head, the stored bytes unchanged)
 * from position keep_src[i] to keep_dst[i] of segment keep_seg[i] (HOST
 * int32[n] each), e.g. to move a draft tree's accepted path to the committed
 * positions.  The pages list "keep" among the paged store's checks (PR #1373
 * review); reading used: every source row is read before any destination is
 * written, so chains of moves within one call are exact.  Positions must lie
 * in [0, seq_len) (TFPA_ERANGE); a destination may appear only once per
 * segment (TFPA_EINVAL); at most 256 pairs a call (TFPA_ECAPACITY).  A page
 * id out of range skips that pair and ORs 1 into cache->err_flag. */
int tfpa_keep_kv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                 const int32_t* keep_seg, const int32_t* keep_src, const int32_t* keep_dst,
                 int32_t n, cudaStream_t stream);

/* ---- Page pool admission (host) ------------------------------------------
 * The pages' memory admission (PR #2011 review, "Memory admission"): a
 * request claims its pages (prompt, max_tokens and one more forward) up front
 * when it is seated, never grows them, waits with LaneMemory when the pool is
 * full, and is turned away by fits() when it could never fit.  Reading used:
 * a claim is all or nothing and takes the lowest free page ids (pages need not
 * be contiguous, so only the free count decides); a released page may be
 * claimed again.  Thread-safe.  No CUDA call. */
typedef struct tfpa_pool tfpa_pool;
tfpa_pool* tfpa_pool_create(int32_t num_pages);      /* NULL if num_pages < 1 or out of memory */
void tfpa_pool_destroy(tfpa_pool* pool);
int32_t tfpa_pool_free(const tfpa_pool* pool);        /* pages free now              */
int tfpa_pool_fits(const tfpa_pool* pool, int32_t npages);  /* 1 if npages <= pool size */
/* Claims npages pages into pages_out (HOST int32[npages], ascending).
 * TFPA_ELANEMEM when fewer are free now (nothing claimed), TFPA_ECAPACITY
 * when the pool could never hold them, TFPA_EINVAL for npages < 0 or NULL. */
int tfpa_pool_claim(tfpa_pool* pool, int32_t npages, int32_t* pages_out);
/* Returns pages (HOST int32[n]).  TFPA_EINVAL (and nothing released) if one
 * is out of range, not claimed, or listed twice. */
int tfpa_pool_release(tfpa_pool* pool, const int32_t* pages, int32_t n);

/* Device-side page-table staging (the pages stage a prompt chunk's page ids
 * between chunks, PR #2011 review, and measure host gaps from it): writes
 * pages[0..n) (HOST int32) into page_table (DEVICE int32) at [first, first+n)
 * on the stream.  The ids travel in kernel parameters (up to 2,048 a launch),
 * so there is no copy call and no host synchronisation; later work on the
 * stream sees the entries.  TFPA_EINVAL for NULL, first < 0 or n < 0. */
int tfpa_stage_pages(int32_t* page_table, int32_t first, const int32_t* pages, int32_t n,
                     cudaStream_t stream);

/* ---- Save and restore a stream's stored rows ------------------------------
 * Page-granular save/restore of a stream's K and V (PR #2011 review: save
 * and restore copies, one copy per page, and a kernel writing mapped host
 * memory measured faster than copies at 32k).  Positions [p0, p1) of segment
 * seg, every kv head, the stored bytes unchanged, to or from an image laid out
 * [K, V][hkv][p1 - p0][128] elements of the cache's dtype (2 or 1 bytes):
 *   image : a pointer the GPU can access, 16-byte aligned: pinned (page-
 *           locked) host memory, registered host memory, or device memory.
 * One kernel launch; the copy runs on the stream (no host synchronisation).
 * A page id out of range skips its rows and ORs 1 into cache->err_flag.
 * TFPA_ERANGE unless 0 <= p0 <= p1 <= seq_len; TFPA_EINVAL for a NULL or
 * misaligned image. */
int tfpa_save_kv(const tfpa_cache* cache, const tfpa_seg* seg, int32_t p0, int32_t p1,
                 void* image, cudaStream_t stream);
int tfpa_restore_kv(const tfpa_cache* cache, const tfpa_seg* seg, int32_t p0, int32_t p1,
                    const void* image, cudaStream_t stream);

/* Split policy, a function of a stream's own length only (so a stream's
 * partials never depend on its batch): pages_per_split = 1 for npages <= 16,
 * else max(2, ceil(npages / 32)); nsplit = ceil(npages / pages_per_split).
 * A 4-bit cache has longer splits, never more of them (tfpa_row_splits gives
 * each row's): tfpa_num_splits is what a scratch is sized by for every type. */
int32_t tfpa_pages_per_split(int32_t seq_len);
int32_t tfpa_num_splits(int32_t seq_len);

/* The split count of each row as tfpa_decode_partial leaves its partials
 * (the nsplit to pass to tfpa_merge for the same rows).  Rows are grouped
 * into runs (consecutive rows of one segment at consecutive positions); a
 * run of at least 49 query vectors per kv head (ceil(nrows * G / 16) >= 4,
 * G = hq / hkv <= 128) takes the tensor-core verify path, whose splits are
 * at least 24 pages and at most 7 a stream; every other row has
 * tfpa_num_splits(seq_len).  Over a 4-bit cache the verify path takes runs
 * of 17 or more query vectors per kv head, in splits of at least 16 pages;
 * the other rows' splits are 1 page for npages <= 8, 2 pages for npages <=
 * 16, else max(4, ceil(npages / 16)) pages, or max(2, ceil(npages / 32)) for
 * fewer than eight kv heads.  Host only (no GPU work): nsplit is HOST
 * int32[rows].  TFPA_EINVAL / TFPA_ERANGE as tfpa_decode. */
int tfpa_row_splits(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                    const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                    int32_t* nsplit);

/* KV write (the KV store kernels that write a stream's page run, PR #1373,
 * "What changes"): row r's K and V for every kv head go to position
 * row_pos[r] of segment row_seg[r], through its page table or slab.  bf16
 * caches copy the bits; fp8 caches store e4m3(RNE, saturating) of
 * float32(x) / scale[g]; fp4 caches: see TFPA_FP4_BLOCK.  row_seg/row_pos are
 * HOST int32[rows].  A position of a segment may be named once in a call (two
 * rows that name one leave a mixture of both, which over a 4-bit cache can be
 * neither's values). */
int tfpa_write_kv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                  const void* k_rows, const void* v_rows,
                  const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                  cudaStream_t stream);

/* KV read: the stored K and V of row_pos[r] of segment row_seg[r], every kv
 * head, as bf16 into k_rows / v_rows (DEVICE bf16 [rows][hkv][128], 16-byte
 * aligned): the inverse of tfpa_write_kv.  bf16 caches copy the bits; fp8
 * values are e4m3 * scale[g] and fp4 values (code * block scale) * scale[g],
 * the product rounded to float32 and then to bf16.  A row on a page whose id
 * is out of range is left unwritten and ORs 1 into cache->err_flag.  Errors
 * as tfpa_write_kv. */
int tfpa_read_kv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg, void* k_rows,
                 void* v_rows, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                 cudaStream_t stream);

/* Decode/verify split-K partials (Issue #1344, "Mechanism": the partial
 * kernels write pm/pl/po, then attn_merge).  For each row r < rows, head h
 * and split s < nsplit[r]: (m, l, o) at scratch row r, where nsplit[r] is
 * what tfpa_row_splits gives for the same rows (tfpa_num_splits(seq_len),
 * or fewer for rows of a run on the tensor-core verify path and for a 4-bit
 * cache).
 * Requires rows <= scratch->cap_rows (TFPA_ECAPACITY otherwise). */
int tfpa_decode_partial(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                        const void* q, const int32_t* row_seg, const int32_t* row_pos,
                        int32_t rows, float softmax_scale, const tfpa_scratch* scratch,
                        cudaStream_t stream);

/* Log-sum-exp merge of scratch rows 0..rows-1 (PR #1355: one merge per slice
 * of at most most_verify rows): out = sum_s o_s 2^(m_s-M) / sum_s l_s 2^(m_s-M),
 * lse = ln2 * (M + log2 sum_s l_s 2^(m_s-M)).  nsplit is HOST int32[rows]. */
int tfpa_merge(const tfpa_scratch* scratch, int32_t hq, int32_t rows,
               const int32_t* nsplit, void* out, float* lse, cudaStream_t stream);

/* Decode/verify attention: partial + merge, in slices of at most
 * scratch->cap_rows rows on shifted q/row-table/out pointers (PR #1355,
 * "Follow-up checks": slices never overrun the partial scratch). */
int tfpa_decode(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                const void* q, const int32_t* row_seg, const int32_t* row_pos,
                int32_t rows, float softmax_scale, const tfpa_scratch* scratch,
                void* out, float* lse, cudaStream_t stream);

/* A decode step in one call: the rows' K and V are stored (as tfpa_write_kv
 * stores them; k_rows, v_rows: DEVICE bf16 [rows][hkv][128], 16-byte
 * aligned) and the rows are decoded (as tfpa_decode decodes them), so the
 * cache and the output hold the bytes of tfpa_write_kv followed by
 * tfpa_decode.  When every run goes to the decode partial kernel and no
 * segment has two runs in the call, that kernel stores the rows itself:
 * the CTAs whose keys include a new row store it before they read it, and
 * no write launch runs.  Otherwise one KV write launch precedes the decode
 * launches.  TFPA_EINVAL for NULL or misaligned rows. */
int tfpa_decode_append(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                       const void* k_rows, const void* v_rows, const void* q,
                       const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                       float softmax_scale, const tfpa_scratch* scratch, void* out, float* lse,
                       cudaStream_t stream);

/* Draft-tree verify: tfpa_decode whose rows see the keys their ancestor
 * masks allow instead of every earlier key.  The pages' partial and merge
 * kernels index the queries, the row tables, the ancestor table (rowanc),
 * the partials and the output by row, and a sliced launch shifts the
 * ancestor table with the other row tables (PR #1355, "Follow-up checks");
 * the pages do not spell out the table's format, and this reading is used:
 *   row_anc : DEVICE uint64[rows], 8-byte aligned, read from the launch's
 *             stream.  Bit d of row_anc[r] set: the key at position
 *             row_pos[r] - d is visible to row r.  Keys more than 63
 *             positions back are always visible, keys after row_pos[r] never.
 *             Bit 0 (the row's own key) must be set.  All bits set is the
 *             causal row, and then the result equals tfpa_decode's bytes.
 * A draft tree of at most 64 nodes laid out at consecutive positions sets,
 * for node i, the bits of its ancestors and itself and every bit that
 * reaches before the root (the committed prefix).  Errors as tfpa_decode;
 * TFPA_EINVAL also for a NULL or misaligned row_anc. */
int tfpa_decode_tree(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                     const void* q, const int32_t* row_seg, const int32_t* row_pos,
                     const uint64_t* row_anc, int32_t rows, float softmax_scale,
                     const tfpa_scratch* scratch, void* out, float* lse, cudaStream_t stream);

/* Decode/verify attention for callers that cannot allocate device memory.
 *
 * Some callers cannot call cudaMalloc: code that runs inside another
 * framework's memory manager, a plug-in that may not grow its host process's
 * device footprint, or a runtime whose allocations are all made before it
 * starts serving.  This entry point needs no caller scratch: the split-K
 * partials live in one array compiled into the library (a file-scope
 * __device__ array of TFPA_STATIC_SCRATCH_SLOTS slots of 130 floats, about
 * 4.3 MB), which every device that loads the library holds until the process
 * exits.  None of the TensorFold sources has a counterpart to this entry
 * point.
 *
 * Same arguments and result as tfpa_decode without `scratch`; rows are
 * processed in slices of TFPA_STATIC_SCRATCH_SLOTS / (hq * TFPA_MAX_SPLITS)
 * rows (8 at hq = 32), which gives the same bytes as tfpa_decode.  Head
 * counts with hq * TFPA_MAX_SPLITS > TFPA_STATIC_SCRATCH_SLOTS (hq > 256) are
 * refused with TFPA_ECAPACITY.  It allocates no device memory and calls no
 * allocating CUDA or library routine.
 *
 * The first call on a device looks up the array's device address on that
 * device (cudaGetSymbolAddress, with that device current); make that first
 * call before any stream capture.  The address is kept per device context:
 * if the context is replaced (cudaDeviceReset, then new work), the next call
 * looks it up again, so it is also a set-up call.  Every call shares the one array and it
 * keeps the last call's contents; nothing in it needs to start at zero, as
 * every slot the merge reads is written by the partial kernel of the same
 * call.  Calls that overlap on the GPU (other streams, other host threads)
 * race on the array: serialise them. */
#define TFPA_STATIC_SCRATCH_SLOTS 8192
int tfpa_decode_static(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                       const void* q, const int32_t* row_seg, const int32_t* row_pos,
                       int32_t rows, float softmax_scale, void* out, float* lse,
                       cudaStream_t stream);

/* ---- Plans: planning a call apart from enqueueing it -----------------------
 * A decode loop's host work (checks, grouping rows into runs, split counts,
 * per-CTA item ranges, tensor maps) does not need the GPU.  A plan does that
 * work for a tfpa_write_kv, tfpa_decode or tfpa_decode_append call (same
 * arguments, without the stream) and keeps the resulting launches by value; tfpa_plan_launch then
 * only enqueues them.  A loop can plan step i + 1 while the GPU runs step i,
 * so that between the host's wait for step i's output and step i + 1's
 * kernels there are only the launches.  None of the TensorFold sources has a
 * counterpart to this.
 *
 * A plan keeps the pointers it was given (device buffers, the cache's pools,
 * scales and page tables, the scratch) and reads them when its launches
 * run: they must stay valid and hold that step's data then.  Host arrays
 * (segs, row tables, host page-table mirrors) are read during the planning
 * call only.  Planning calls append to the plan in order; tfpa_plan_launch
 * enqueues every launch on `stream` in that order and may be called any
 * number of times.  A planning call that fails returns its error code (as
 * the direct call would) and leaves the plan as it was.  A plan is used by
 * one host thread at a time.  tfpa_plan_create returns NULL if host memory
 * runs out; tfpa_plan_launch returns TFPA_ECUDA if a launch fails (launches
 * before it stay enqueued). */
typedef struct tfpa_plan tfpa_plan;
tfpa_plan* tfpa_plan_create(void);
void tfpa_plan_destroy(tfpa_plan* plan);
void tfpa_plan_clear(tfpa_plan* plan);                 /* drops every planned launch */
int32_t tfpa_plan_launches(const tfpa_plan* plan);     /* launches planned so far    */
int tfpa_plan_write_kv(tfpa_plan* plan, const tfpa_cache* cache, const tfpa_seg* segs,
                       int32_t nseg, const void* k_rows, const void* v_rows,
                       const int32_t* row_seg, const int32_t* row_pos, int32_t rows);
int tfpa_plan_decode(tfpa_plan* plan, const tfpa_cache* cache, const tfpa_seg* segs,
                     int32_t nseg, const void* q, const int32_t* row_seg,
                     const int32_t* row_pos, int32_t rows, float softmax_scale,
                     const tfpa_scratch* scratch, void* out, float* lse);
int tfpa_plan_decode_append(tfpa_plan* plan, const tfpa_cache* cache, const tfpa_seg* segs,
                            int32_t nseg, const void* k_rows, const void* v_rows, const void* q,
                            const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                            float softmax_scale, const tfpa_scratch* scratch, void* out,
                            float* lse);
int tfpa_plan_launch(const tfpa_plan* plan, cudaStream_t stream);

/* Device mode: replaying a captured plan as the streams grow.
 * A plan's launches normally carry everything by value, so a CUDA graph
 * captured from tfpa_plan_launch repeats the lengths it was captured with.
 * In device mode each write, decode and merge launch instead reads the data
 * that changes as streams grow (run lengths and positions, split counts,
 * work-item and per-CTA ranges) from its own slot of a DEVICE buffer that
 * the caller owns, and the launch shapes stop depending on the lengths: a
 * decode partial launch takes one CTA per SM (at most 256) whatever its
 * work.  A decode loop then captures once [copy of the packed data into the
 * buffer, tfpa_plan_launch] and, each step, re-plans with the new lengths,
 * packs and replays.
 *
 * tfpa_plan_set_device(plan, dyn, bytes): dyn = DEVICE buffer, 16-byte
 *   aligned, `bytes` long, or NULL to go back to parameter mode.  dyn may
 *   be mapped pinned host memory (see "Pinned host memory" above): then
 *   tfpa_plan_dyn_pack may write the packed data into dyn itself, with no
 *   copy, while no launch that reads it is pending.  Only on an
 *   empty plan (after create or clear), else TFPA_EINVAL.  The plan keeps the
 *   pointer; tfpa_plan_clear keeps the mode.  A planning call whose slots do
 *   not fit returns TFPA_ECAPACITY; rows that would take the tensor-core
 *   verify path (a run of 49 or more query vectors per kv head, 17 or more
 *   over a 4-bit cache, whose grid follows the lengths) return TFPA_EINVAL.
 * tfpa_plan_dyn_bytes: bytes of the buffer the planned launches use (about
 *   4 KB per decode launch, 2.6 KB per write, 2 KB per merge).
 * tfpa_plan_dyn_pack(plan, host, bytes): writes those bytes, the data of
 *   the launches as planned now, to HOST memory `host` (the caller copies
 *   them to `dyn` before the launches run, e.g. with a copy captured in the
 *   same graph from pinned memory; the host buffer must not change while
 *   such a copy is pending).  TFPA_EINVAL outside device mode,
 *   TFPA_ECAPACITY if bytes < tfpa_plan_dyn_bytes.
 * tfpa_plan_shape: a 64-bit hash of everything the launches take by value
 *   except that data (kinds, grids, pointers, tensor maps, head counts).
 *   Two plans with the same shape may replay one captured graph; a
 *   different shape (new rows, a stream moved between pool and slab, a
 *   slice boundary moved) needs a new capture. */
int tfpa_plan_set_device(tfpa_plan* plan, void* dyn, size_t bytes);
size_t tfpa_plan_dyn_bytes(const tfpa_plan* plan);
int tfpa_plan_dyn_pack(const tfpa_plan* plan, void* host, size_t bytes);
uint64_t tfpa_plan_shape(const tfpa_plan* plan);

/* A plan as one CUDA graph, owned by the plan.
 * tfpa_plan_capture(plan, before, nbefore, after, nafter, stream) captures,
 *   on `stream` (a created stream: not NULL, not cudaStreamLegacy; nothing
 *   else may be enqueued on it meanwhile), the copies `before` (each a
 *   cudaMemcpyAsync of `bytes` from src to dst, kind inferred: e.g. a step's
 *   inputs and, in device mode, its packed data from pinned host memory),
 *   the plan's launches and the copies `after` (e.g. the output to pinned
 *   host memory), instantiates the graph and keeps it with the plan's shape
 *   (tfpa_plan_shape), replacing an earlier one.  The copies read and write
 *   their buffers when the graph runs.  TFPA_EINVAL for an empty plan, bad
 *   copies or stream; TFPA_ECUDA if capture or instantiation fails (the
 *   plan keeps its earlier graph).  Launch the plan once before its first
 *   capture on a device, so that kernel attributes are set outside capture.
 * tfpa_plan_replay(plan, stream): launches the graph on `stream`.
 *   TFPA_EINVAL if nothing was captured or the plan's shape has changed
 *   since (re-planned with other rows, streams or pointers: capture again).
 *   In device mode a loop re-plans each step (tfpa_plan_clear + planning
 *   calls), packs into the host buffer the graph's first copy reads, and
 *   replays.  The graph is destroyed with the plan; tfpa_plan_clear keeps it. */
typedef struct {
  void* dst;
  const void* src;
  size_t bytes;
} tfpa_copy;
int tfpa_plan_capture(tfpa_plan* plan, const tfpa_copy* before, int32_t nbefore,
                      const tfpa_copy* after, int32_t nafter, cudaStream_t stream);
int tfpa_plan_replay(const tfpa_plan* plan, cudaStream_t stream);

/* Causal prompt-chunk attention over the paged prefix, one pass with online
 * softmax on tcgen05/TMEM tiles (PR #2011, "hpattn_p256_kernel": page size a
 * constant 256, one page lookup per key tile).  max_rows_per_launch > 0 runs
 * the rows in slices of that many (a slice's result is the same bytes as one
 * launch); 0 = one launch.  Every cache type. */
int tfpa_prefill(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                 const void* q, const int32_t* row_seg, const int32_t* row_pos,
                 int32_t rows, float softmax_scale, int32_t max_rows_per_launch,
                 void* out, float* lse, cudaStream_t stream);

/* ---- Eviction by accumulated attention weight ------------------------------
 * A long stream keeps the keys its rows attend to: their weights are summed
 * up as the stream is served, and from time to time all but the keys of
 * largest sum leave the cache, each kv head choosing its own.  None of the
 * TensorFold sources has a counterpart to this.
 *
 * tfpa_key_mass adds the attention weights of the call's rows to the keys'
 * sums.  For every segment s that has a row in the call, kv head g and key j
 * < seq_len:
 *   mass[s][g][j] = decay mass[s][g][j]
 *                 + sum over the segment's rows r with row_pos[r] >= j and the
 *                   query heads h of g of exp(softmax_scale q_rh.k_j - lse[r][h])
 * so with lse as tfpa_decode or tfpa_prefill left it for the same rows and
 * cache, a row adds 1 per query head in all.  The sum's order is fixed, so the
 * bytes are too.
 *   q    : DEVICE bf16 [rows][hq][128], 16-byte aligned (any memory the GPU
 *          can read); lse: DEVICE float [rows][hq] (a row with lse = -inf adds
 *          nothing, whatever its q holds).  Over an e4m3 or 4-bit cache up to
 *          256 query vectors of a kv head are taken in f16 under one power of
 *          two: exact within 2^30 of their largest finite element.
 *   mass : DEVICE float [nseg][hkv][mass_cap], planes by the segment's index
 *          in the call; zero before a stream's first call.  Entries from
 *          seq_len on, and segments without rows, are left as they are.
 *          mass_cap >= seq_len of every segment used (TFPA_ECAPACITY).
 *   decay: finite and >= 0; 0 does not read the old sums.
 * K is read once (V not at all).  Keys of a page whose id is out of range keep
 * their entries and OR 1 into cache->err_flag.  Rows may come in any order; a
 * segment's rows count together however they are grouped. */
int tfpa_key_mass(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg, const void* q,
                  const float* lse, const int32_t* row_seg, const int32_t* row_pos, int32_t rows,
                  float softmax_scale, float decay, float* mass, int32_t mass_cap,
                  cudaStream_t stream);

/* tfpa_evict_kv cuts every segment s of the call to keep[s] keys (HOST
 * int32[nseg], 1 <= keep[s] <= seq_len, TFPA_ERANGE), for each kv head those
 * that come first in this order: positions below `sink` and positions from
 * next_pos[s] - recent on; then larger mass (a NaN counts as largest); then
 * the lower slot.  The kept keys are packed into slots [0, keep[s]) in place:
 * a kept key below keep[s] stays in its slot, and the evicted slots below
 * keep[s], ascending, take the kept keys behind it, ascending (K and V rows,
 * mass and key_pos; the stored bytes unchanged).  mass becomes 0 and key_pos
 * -1 in [keep[s], seq_len).  The stream goes on with seq_len = keep[s]: its
 * next row is stored at that slot, with its own rotary position.
 *   key_pos : DEVICE int32 [nseg][hkv][mass_cap], the position that each
 *             slot's key has in its stream, all different; NULL: its slot.  Only
 *             read and moved here: the caller writes a new row's entry.  A
 *             negative entry is no position: neither among the first nor among
 *             the last ones.
 *   next_pos: HOST int32[nseg], the position the stream's next row will have,
 *             at least seq_len (TFPA_ERANGE); NULL: seq_len without key_pos,
 *             else one past the largest position among the kv head's slots.
 *   sink, recent >= 0, with sink + recent <= keep[s] where keep[s] < seq_len
 *             (TFPA_EINVAL).
 *   mass    : as tfpa_key_mass, 16-byte aligned like key_pos; mass_cap a
 *             multiple of 4.
 *   moves   : DEVICE int32 [nseg][hkv][mass_cap + 4], 16-byte aligned, written:
 *             [0] the number m of rows moved, and from [4] on m pairs (from
 *             slot, to slot), for whoever keeps more per key than this cache.
 * A pair on a page whose id is out of range leaves both slots' K and V rows,
 * mass and key_pos as they are and ORs 1 into cache->err_flag (moves lists it).
 * Two segments of a call must not share pages, and a
 * stream that goes on reading a page must not share it with one that is cut. */
int tfpa_evict_kv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                  const int32_t* keep, const int32_t* next_pos, int32_t sink, int32_t recent,
                  float* mass, int32_t* key_pos, int32_t mass_cap, int32_t* moves,
                  cudaStream_t stream);

/* ---- From the projection to attention over a part of a long stream ----------
 * A decode step of a long stream: tfpa_write_qkv turns the projection's rows
 * into q and stored K / V, tfpa_key_bounds brings the bounds of the blocks they
 * fell into up to date, tfpa_select_blocks chooses for each row and kv head the
 * blocks worth reading, and tfpa_decode_blocks attends to them.  None of the
 * TensorFold sources has a counterpart to this.  Every call can be captured
 * in a graph (lengths and positions are kept as they were then). */

/* Rotary tables: cos and sin of position t and frequency f_i, i < rot_dim / 2,
 * times attn_scale, with f_i = base^(-2 i / rot_dim) radians a position, and
 * for a context stretched `factor` times beyond orig_len positions
 *   TFPA_ROPE_LINEAR  f_i / factor
 *   TFPA_ROPE_BASE    base * factor^(rot_dim / (rot_dim - 2)) in base's place
 *   TFPA_ROPE_BANDS   f_i u + f_i / factor (1 - u), where
 *                     u = (turns_i - low) / (high - low), cut to [0, 1], and
 *                     turns_i = orig_len f_i / 2 pi
 *   TFPA_ROPE_RAMP    the same with u = 1 - (i - a) / max(b - a, 0.001), cut to
 *                     [0, 1]; dim(n) = rot_dim ln(orig_len / (2 pi n)) /
 *                     (2 ln base), a = max(floor(dim(high)), 0),
 *                     b = min(ceil(dim(low)), rot_dim - 1)
 * The frequencies are formed in 64 bits, and position times frequency modulo one
 * turn is exact for the frequency as it is held.  So an angle is off by the
 * position times the frequency's own error, which is 2^-65 of a turn and (but
 * for a frequency of 1) a few 2^-53 of the frequency: below 10^-10 radians at
 * position 131,072 and 10^-6 at 2^31, beside the tables' own rounding to float32. */
enum {
  TFPA_ROPE_NONE = 0,
  TFPA_ROPE_LINEAR = 1,
  TFPA_ROPE_BASE = 2,
  TFPA_ROPE_BANDS = 3,
  TFPA_ROPE_RAMP = 4
};
typedef struct {
  double base;                    /* > 1                                                   */
  double factor;                  /* >= 1 (not read for TFPA_ROPE_NONE)                    */
  double low, high;               /* TFPA_ROPE_BANDS, _RAMP: 0 < low < high                */
  double attn_scale;              /* > 0, also as a float; 1: none                         */
  int32_t rot_dim;                /* a multiple of 16, at most 128                         */
  int32_t scaling;
  int32_t orig_len;               /* TFPA_ROPE_BANDS, _RAMP: >= 1                          */
} tfpa_rope_spec;
/* Writes the rows of positions first .. first + n - 1 to cos and sin (DEVICE
 * float [n][rot_dim / 2], 16-byte aligned).  TFPA_ERANGE unless 0 <= first and
 * first + n <= 2^31.  With rot_dim = 128 they are the tables of
 * tfpa_write_kv_rope too. */
int tfpa_rope_table(const tfpa_rope_spec* spec, int64_t first, int32_t n, float* cos, float* sin,
                    cudaStream_t stream);

/* A projection's rows.  Row r's q, k and v lie at their pointers plus r times
 * their strides (so all three may point into one fused projection's output);
 * heads are [128] one after the other.  For every q head (k head)
 *   with q_weight (k_weight): y = x (1 / sqrt(mean x^2 + eps)) w; the squares
 *     are added in pairs of neighbours, then pairs of those sums, and so on;
 *   with rope_cos: the first rot_dim dims rotated by row t of the table, t the
 *     row's rotary position (rope_pos, or NULL: row_pos): each pair (a, b)
 *     becomes (a c - b s, b c + a s), where a pair is dims i and
 *     i + rot_dim / 2, or with `interleaved` dims 2 i and 2 i + 1;
 * each product, sum, quotient and root rounded to float32 (no fused multiply-
 * add).  q is rounded to bf16 into q_out (DEVICE bf16 [rows][hq][128]); K and V
 * are stored as tfpa_write_kv stores them (K unrounded before a quantised
 * store).  q and q_out may both be NULL (K and V only), and q_out may be q
 * itself when q_stride is hq * 128; else q_out shares no memory with an input
 * (TFPA_EINVAL).  A position that two rows of one call name holds either's K and
 * V afterwards, or some of both.
 * A rotary position outside the table leaves the row's q_out, K and V unwritten
 * and ORs 4 into cache->err_flag (without rope_pos it is TFPA_ERANGE); a page
 * id out of range leaves its K and V unwritten and ORs 1. */
typedef struct {
  const void* q;                  /* DEVICE bf16, 16-byte aligned like k and v             */
  const void* k;
  const void* v;
  int64_t q_stride;               /* elements between rows: a multiple of 8, >= heads * 128 */
  int64_t k_stride;
  int64_t v_stride;
  const float* q_weight;          /* DEVICE float[128], 16-byte aligned; NULL: not normed  */
  const float* k_weight;
  const float* rope_cos;          /* DEVICE float[rope_n][rot_dim / 2], 16-byte aligned;   */
  const float* rope_sin;          /*   NULL: not rotated                                   */
  const int32_t* rope_pos;        /* DEVICE int32[rows], or NULL                           */
  int32_t rope_n;
  int32_t rot_dim;                /* a multiple of 16, at most 128                         */
  int32_t interleaved;
  float eps;                      /* > 0 with a weight                                     */
} tfpa_qkv;
int tfpa_write_qkv(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                   const tfpa_qkv* in, const int32_t* row_seg, const int32_t* row_pos,
                   int32_t rows, void* q_out, cudaStream_t stream);

/* Bounds of the keys.  A stream's positions are cut into blocks of `block`
 * positions (64, 128 or 256, counted from position 0).  For each block and kv
 * head the smallest and then the largest stored K of every head dim is kept,
 * as the stored value without k_scale (exact in bf16 for every cache type; a
 * NaN counts as 0).  Bounds go with the pages: streams that share a page share
 * its bounds (a block that one of them ends in is then taken up to the end of
 * the one whose rows were called last: of two in one call either, or some of
 * both).  A call that
 * stores, moves or restores keys leaves them as they are: tfpa_key_bounds brings
 * them up to date. */
typedef struct {
  int32_t block;
  void* pool;                     /* DEVICE bf16 [num_pages][hkv][256 / block][2][128],    */
                                  /*   16-byte aligned; may be NULL without paged segments */
  void* const* slabs;             /* HOST [nseg]: a slab segment's DEVICE bf16             */
                                  /*   [hkv][slab_cap / block][2][128]; NULL without slabs */
} tfpa_bounds;

/* Takes the bounds of every block that holds one of the call's rows anew, from
 * the keys stored at its positions below seq_len (so a block whose rows were
 * overwritten, or that a cut left in part, is right again after a call with
 * one of its rows).  A block on a page whose id is out of range is left as it
 * is and ORs 1 into cache->err_flag.  After tfpa_evict_kv a stream's keys have
 * moved: call with all of its rows. */
int tfpa_key_bounds(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                    const tfpa_bounds* bounds, const int32_t* row_seg, const int32_t* row_pos,
                    int32_t rows, cudaStream_t stream);

/* For each row and kv head the nsel blocks to attend to, of the blocks up to
 * the row's own: the first `sink`, the last `recent` (the row's own the last of
 * them), then those of largest
 *   score = sum over the kv head's query heads h and dims d of
 *           max(q_hd, 0) largest_d + min(q_hd, 0) smallest_d,
 * which (k_scale above 0) no sum of the heads' scores with a key of the block
 * exceeds, k_scale and softmax_scale left out; ties go to
 * the lower block, and a score that is not a number (an infinite bound under a
 * zero of q) counts as larger than an infinite one.  Scores too near the border
 * for float32 are taken in float64, every block's sum in the same order: off by
 * (14 + query heads a kv head) * 2^-53 of the sum of its terms' magnitudes at
 * most, so the choice is that of exact arithmetic but between blocks whose scores
 * are nearer than that (equal bounds give equal scores).
 *   q      : DEVICE bf16 [rows][hq][128], 16-byte aligned (as tfpa_decode's)
 *   blocks : DEVICE int32 [rows][hkv][nsel], written: block numbers ascending,
 *            -1 behind the last where there are fewer than nsel.
 * A block on a page whose id is out of range is not chosen and ORs 1 into
 * cache->err_flag.  sink, recent >= 0, sink + recent <= nsel (TFPA_EINVAL).  At
 * most 18,432 blocks up to a row (TFPA_ECAPACITY). */
int tfpa_select_blocks(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                       const tfpa_bounds* bounds, const void* q, const int32_t* row_seg,
                       const int32_t* row_pos, int32_t rows, int32_t nsel, int32_t sink,
                       int32_t recent, int32_t* blocks, cudaStream_t stream);

/* Attention of each row over its own blocks: tfpa_decode whose row r and kv
 * head g see the keys of the blocks blocks[r][g][0..nsel) (DEVICE int32, as
 * tfpa_select_blocks leaves them) up to row_pos[r].  Entries may come in any
 * order; a negative one, and one past the row's own block, is passed over; a
 * block that is named twice counts twice.  A row that sees no key gets out = 0
 * and lse = -inf.  No scratch.  1 <= nsel <= 2^24.  A page id out of range: as
 * tfpa_decode. */
int tfpa_decode_blocks(const tfpa_cache* cache, const tfpa_seg* segs, int32_t nseg,
                       const void* q, const int32_t* row_seg, const int32_t* row_pos,
                       int32_t rows, int32_t block, int32_t nsel, const int32_t* blocks,
                       float softmax_scale, void* out, float* lse, cudaStream_t stream);

/* The five calls above with their arguments in memory: tfpa_call(&c) is the call
 * that c.op names, with c's fields as its arguments (those that it does not
 * have are not read), and returns what it returns.  For callers that pay for
 * each argument of a call, as a foreign-function interface does: from Python
 * tfpa_decode_blocks takes 7.9 us of host time this way, 10.2 us otherwise. */
enum {
  TFPA_OP_ROPE_TABLE = 0,
  TFPA_OP_WRITE_QKV = 1,
  TFPA_OP_KEY_BOUNDS = 2,
  TFPA_OP_SELECT_BLOCKS = 3,
  TFPA_OP_DECODE_BLOCKS = 4
};
typedef struct {
  int32_t op;
  int32_t nseg;
  const tfpa_cache* cache;
  const tfpa_seg* segs;
  const int32_t* row_seg;
  const int32_t* row_pos;
  cudaStream_t stream;
  const tfpa_bounds* bounds;
  const void* q;
  int32_t* blocks;
  void* out;                      /* TFPA_OP_WRITE_QKV: q_out                              */
  float* lse;
  int32_t rows;                   /* TFPA_OP_ROPE_TABLE: n                                 */
  int32_t block;
  int32_t nsel;
  int32_t sink;
  int32_t recent;
  int32_t reserved;               /* not read                                              */
  double softmax_scale;           /* rounded to float                                      */
  union {                         /* read by the two calls that have them                  */
    tfpa_qkv qkv;
    struct {
      const tfpa_rope_spec* spec;
      int64_t first;
      float* cos;
      float* sin;
    } rope;
  } u;
} tfpa_call_args;
int tfpa_call(const tfpa_call_args* c);

/* Launch recording for host tests (PR #1355: "a launch-recording host test
 * where a 257-row chunk issues 3 slices").  With a hook installed every
 * launch is reported; with dry_run != 0 nothing is enqueued and no CUDA call
 * is made, so the slicing logic runs on a machine without a GPU. */
typedef struct {
  int32_t kind;          /* 0 write_kv, 1 decode partial, 2 merge, 3 prefill, 4 keep,
                            5 stage pages, 6 save, 7 restore, 8 verify (decode or tree
                            rows of runs with 49 or more query vectors per kv head, 17
                            over a 4-bit cache, on tensor cores; items = tiles),
                            9 read_kv, 10 key_mass, 11 evict (choice), 12 evict (moves),
                            13 rope_table, 14 write_qkv, 15 key_bounds, 16 select_blocks,
                            17 decode_blocks */
  int32_t row0;          /* first row of the call this launch covers */
  int32_t rows;          /* rows it covers */
  int32_t runs;          /* row groups (segment, consecutive positions) */
  int32_t items;         /* work items (decode: tiles of (kv head, m-tile, split)) */
  int32_t grid;          /* CTAs (prefill: two per tile, in clusters of two) */
  int64_t q_offset;      /* element offset of the q pointer it got, from the call's q */
  int64_t out_offset;    /* element offset of the out pointer, from the call's out */
} tfpa_launch_record;
typedef void (*tfpa_launch_hook)(const tfpa_launch_record* rec, void* user);
void tfpa_set_launch_hook(tfpa_launch_hook hook, void* user, int dry_run);

const char* tfpa_strerror(int code);
const char* tfpa_version(void);

#ifdef __cplusplus
}
#endif
#endif /* TFPA_H */
