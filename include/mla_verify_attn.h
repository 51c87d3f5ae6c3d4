/*
 * mla_verify_attn.h -- C ABI of the GB300 (sm_103a) absorbed-MLA verify-attention library.
 *
 * The operation (pages by title):
 *   "The Flash Attention Kernel That Had to Be Built: Designing sm_120 MLA
 *   Verify for Blackwell Consumer GPUs", section "What Input Knowledge Is
 *   Required to Understand This Message": each cache row is a 512-wide latent
 *   kv_c followed by a 64-wide decoupled RoPE key k_pe; a query row is an
 *   absorbed q_nope (512) and q_pe (64); score = q_nope . kv_c + q_pe . k_pe;
 *   the latent kv_c is also the value; a draft query sees the keys its
 *   candidate tree allows (paragraph "Speculative Decoding with DFlash"), the
 *   others are set to -inf before a softmax ("Flash Attention Algorithm").
 *   "The Decisive Microbench: When Theory Meets Silicon", section "The
 *   KV-Split Solution": the key range is split across thread blocks whose
 *   unnormalised partial states are merged by a second kernel with the
 *   online-softmax combine.
 *
 * For stream b, draft i < q_len, head h < H, with prefix_b = seq_lens[b] - q_len:
 *   visible(t) = t < prefix_b  or  (t < seq_lens[b] and bit (t - prefix_b) of mask row i)
 *   s_t        = scale * (sum_d q_nope[b,i,h,d] kv[b,t,d] + sum_e q_rope[b,i,h,e] kv[b,t,512+e])
 *   out[b,i,h] = sum_{visible t} softmax(s)_t * kv[b,t,0:512]
 *   lse[b,i,h] = ln sum_{visible t} exp(s_t)          (-inf and out = 0 if nothing is visible)
 *
 * Conventions for every entry point:
 *   - Device pointers unless stated otherwise; the caller owns all memory.
 *     The library allocates no device memory.
 *   - Calls are asynchronous on `stream`.  Argument errors are detected on the
 *     host and returned before anything is launched.  Problems only the GPU can
 *     see (a seq_lens value out of range, an internal wait that timed out) are
 *     recorded in a per-device status word read by mla_verify_attn_last_device_error.
 *   - bf16 tensors are passed as `const void*` holding IEEE bfloat16 values.
 *   - Results are deterministic for fixed inputs, Smax and device.
 *   - Precision: scores, softmax statistics and the output accumulate in fp32;
 *     the softmax weights enter the weights-times-values product in bf16 (the
 *     cache is bf16).  Their rounding is compensated where it would show:
 *     streams of up to 4096 keys (mla_verify_attn_set_two_term_max_keys moves
 *     the limit) send the weights as two bf16 terms; longer ones send one and
 *     add back the rounding error of each row's largest-score key.  Measured
 *     against an fp64 evaluation of the formula above: max |out error| <= 5e-4
 *     on N(0,1) inputs of every length and <= 6.4e-4 with a planted dominant
 *     key; a row whose weight several strong keys share keeps the rounding of
 *     all but the largest (3.0e-3 with 20 planted keys in one 126-tile slice,
 *     removed by two terms).  The tests hold it to 2e-3 (lse: 1e-3).
 *   - Stream capture: no entry point reads device memory on the host or
 *     synchronises inside mla_verify_attn.  Grid, split plan and tensor maps
 *     depend only on (B, q_len, H, Smax), the pointers and the device, so after
 *     the first call on a device (one-time setup: kernel attributes, occupancy
 *     query) a call may be captured into a CUDA graph; each replay reads the
 *     inputs' contents at replay time (seq_lens may change, within Smax).
 */
#ifndef MLA_VERIFY_ATTN_H
#define MLA_VERIFY_ATTN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes (returned by the entry points and by the device status). */
enum mla_status {
  MLA_OK = 0,
  MLA_ERR_NULLPTR = -1,            /* a required pointer is NULL */
  MLA_ERR_SHAPE = -2,              /* B, q_len, H or Smax outside the supported range */
  MLA_ERR_ALIGN = -3,              /* a pointer misses its required alignment */
  MLA_ERR_WORKSPACE = -4,          /* workspace smaller than mla_verify_attn_workspace_size() */
  MLA_ERR_UNSUPPORTED_DEVICE = -5, /* current device is not sm_103 (GB300) or has no CUDA context */
  MLA_ERR_LAUNCH = -6,             /* a kernel launch or tensor-map creation failed */
  MLA_ERR_DEVICE_TIMEOUT = -7,     /* (device status) an internal pipeline wait gave up */
  MLA_ERR_SEQLEN = -8,             /* (device status) some seq_lens[b] outside [q_len, Smax] */
  MLA_ERR_ARG = -9,                /* any other invalid argument (e.g. non-finite scale) */
  MLA_ERR_PAGE = -10,              /* (device status) a block-table entry outside the page pool */
  MLA_ERR_POOL = -11,              /* (device status) the free-page list is too short (extend) or its array too small (trim) */
  MLA_ERR_SLOT = -12               /* (device status) a cache slot or draft index outside its range */
};

/*
 * Bytes of scratch memory mla_verify_attn needs for these sizes on the
 * current device (0 when the key range is not split).  The value depends only
 * on (B, q_len, H, Smax) and the device's SM count.  Host-only; launches
 * nothing.  Returns 0 as well for invalid sizes (mla_verify_attn then reports
 * MLA_ERR_SHAPE).
 * Scratch holds the per-split partial states of the key-range split (page
 * "The Decisive Microbench: When Theory Meets Silicon", section "The KV-Split
 * Solution"): [nsplit][B*q_len*H][512] fp32 accumulators followed by
 * [nsplit][B*q_len*H][2] fp32 (running max, running sum), then, at a
 * 256-byte boundary, 256 bytes where calls with 2 to 32 streams keep the
 * slice plan the device chose from seq_lens (a smaller slice count than the
 * host's nsplit when the streams are ragged).
 */
size_t mla_verify_attn_workspace_size(int B, int q_len, int H, int Smax);

/*
 * Verify attention for B streams of q_len draft queries over a latent cache.
 *
 *   q_nope_abs  [B, q_len, H, 512] bf16, contiguous; 16-byte aligned.
 *   q_rope      [B, q_len, H, 64]  bf16, contiguous; 16-byte aligned.
 *   kv          [B, Smax, 576]     bf16, contiguous; row = latent (512) | rope (64);
 *               16-byte aligned.  Rows t < seq_lens[b] must be finite; rows at or
 *               beyond seq_lens[b] may hold anything (NaN included) and are never used.
 *   seq_lens    [B] int32: prefix_b + q_len, with q_len <= seq_lens[b] <= Smax.  The
 *               drafts' own cache rows are rows prefix_b .. seq_lens[b]-1.
 *   tree_mask   [B, q_len, ceil(q_len/32)] uint32; bit j (LSB first, word j/32) of row
 *               i set <=> draft i sees draft j.  Bits >= q_len are ignored.
 *   B >= 0, 1 <= q_len <= 64, 1 <= H, q_len*H*B < 2^31, 1 <= Smax < 2^24.
 *   scale       finite float multiplying every score (e.g. 1/sqrt(192)).
 *   out         [B, q_len, H, 512] fp32, normalised output; 16-byte aligned.
 *   lse         [B, q_len, H] fp32, natural log-sum-exp of the scaled scores; 4-byte aligned.
 *   workspace   device scratch of at least mla_verify_attn_workspace_size(B, q_len, H,
 *               Smax) bytes, 256-byte aligned (may be NULL when that size is 0).  Its
 *               contents on entry do not matter; it is not read after the call.
 *   stream      CUDA stream (0 = legacy default stream).
 *
 * Returns MLA_OK after enqueuing the work, or a negative mla_status with nothing
 * enqueued.  Calls that share a workspace must not overlap on the GPU.
 */
int mla_verify_attn(const void* q_nope_abs, const void* q_rope, const void* kv,
                    const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len, int H,
                    int Smax, float scale, float* out, float* lse, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/*
 * mla_verify_attn over a paged cache.  The pages have no paged interface; they
 * name a paged cache (page_size 1, scattered rows) as the production layout
 * (page "The Moment of Truth: Benchmarking a Custom sm_120 Flash Attention
 * Kernel", section "Output Knowledge Created").  Pages of a multiple of 64 keys
 * are read in place with whole-tile TMA loads; for any other page size (1
 * included) a first kernel copies each stream's rows, in key order, into a
 * contiguous cache in the workspace, which the split kernel then reads (the
 * results equal the contiguous call's bit for bit).  The computation is that
 * of mla_verify_attn with
 *   kv[b, t, :] = kv_pool[block_table[b, t / page_size] * page_size + t % page_size, :]
 * i.e. key t of stream b lives in page block_table[b][t / page_size] of the pool.
 *
 *   kv_pool      [pool_rows, 576] bf16, rows = pages x page_size, 16-byte aligned.
 *                Rows of pages no stream refers to, and rows past a stream's
 *                seq_len, may hold anything (NaN included).
 *   pool_rows    rows in the pool: a multiple of page_size, < 2^31.
 *   block_table  [B, max_blocks] int32, 4-byte aligned: the page of each
 *                page_size-key block; entries past ceil(seq_lens[b] / page_size)
 *                are not read.  An entry outside [0, pool_rows / page_size) is
 *                reported as MLA_ERR_PAGE through the device status (that
 *                stream's results are then undefined).
 *   max_blocks   blocks per stream in block_table; Smax = max_blocks * page_size
 *                (< 2^24) bounds seq_lens[b].
 *   workspace    at least mla_verify_attn_paged_workspace_size(B, q_len, H,
 *                max_blocks, page_size) bytes (MLA_ERR_WORKSPACE otherwise).
 *   page_size    keys per page, >= 1 (MLA_ERR_SHAPE otherwise).  Multiples of 64
 *                are the fast path: a 64-key tile then never crosses a page.
 * All other arguments, results and errors as for mla_verify_attn.
 */
/*
 * Workspace bytes mla_verify_attn_paged needs on the current device: that of
 * mla_verify_attn for Smax = max_blocks * page_size, plus, when page_size is
 * not a multiple of 64, a contiguous copy of the cache (B * Smax * 1152 bytes,
 * after the partials at a 256-byte boundary).  0 for arguments the call would
 * reject (and, like mla_verify_attn_workspace_size, without a usable device).
 * Host-only.
 */
size_t mla_verify_attn_paged_workspace_size(int B, int q_len, int H, int max_blocks, int page_size);

int mla_verify_attn_paged(const void* q_nope_abs, const void* q_rope, const void* kv_pool,
                          long long pool_rows, const int32_t* block_table, int max_blocks,
                          int page_size, const int32_t* seq_lens, const uint32_t* tree_mask, int B,
                          int q_len, int H, float scale, float* out, float* lse, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/*
 * Synchronises `stream`, then returns and clears the current device's status
 * word: MLA_OK, or of the errors recorded the first in the order MLA_ERR_SEQLEN,
 * MLA_ERR_DEVICE_TIMEOUT, MLA_ERR_PAGE, MLA_ERR_POOL, MLA_ERR_SLOT,
 * or MLA_ERR_LAUNCH if the synchronisation itself failed.  The word is shared
 * by all calls on the device since it was last read.
 * Every internal pipeline wait gives up after 2 s; the call's kernels then
 * unwind (waiting, again bounded, for their own copies in flight) and leave
 * the context usable.  mla_verify_attn_set_test_controls can make one work
 * unit withhold a cache load, to exercise that path.
 */
int mla_verify_attn_last_device_error(cudaStream_t stream);

/* Human-readable name of a status code (static string; never NULL). */
const char* mla_verify_attn_strerror(int status);

/*
 * The split plan mla_verify_attn uses, for inspection and tests (host-only):
 *   n_row_tiles  = ceil(q_len*H / 128) query-row tiles per stream,
 *   nsplit       = number of key-range slices (1 = no split, no scratch),
 *   chunk_tiles  = 64-key tiles per slice.
 * `max_clusters` is the number of 2-CTA clusters that fit on the device at
 * once (pass <= 0 to query the current device).  Honours a slice count forced
 * with mla_verify_attn_set_test_controls.  For 2 to 32 streams (count not
 * forced) this is the largest plan: a one-block planning kernel of the call
 * may choose fewer slices from the device's seq_lens, and the slices then
 * start longest first.
 * Returns MLA_OK or a status.
 */
int mla_verify_attn_plan(int B, int q_len, int H, int Smax, int max_clusters, int* n_row_tiles,
                         int* nsplit, int* chunk_tiles);

/*
 * Measurement aid; the pages have no counterpart.  While both events are
 * non-NULL, every mla_verify_attn call records `before_split` on its stream
 * just before the split kernel is launched and `after_split` just after it, so
 * cudaEventElapsedTime(before_split, after_split) is the split kernel's own
 * duration.  While they are set, the slice merge is launched without overlapping
 * the split kernel's tail.  NULL, NULL switches recording off.  The events are
 * the caller's (cudaEventCreate); the library only records them.  Set this only
 * while no other thread is calling into the library.  Returns MLA_OK, or
 * MLA_ERR_NULLPTR when exactly one event is NULL.
 */
int mla_verify_attn_set_timing_events(cudaEvent_t before_split, cudaEvent_t after_split);

/*
 * Precision control; the pages have no counterpart (their kernels keep P in
 * fp32).  V is bf16 in the cache and the tensor-core product takes P and V in
 * one type, so P is rounded to bf16.  Streams of at most `max_keys` keys
 * (seq_lens[b] <= max_keys) send P as two bf16 terms, hi + lo, and run the
 * P.V product once per term: outputs then match fp32 P to ~1e-5.  Longer
 * streams send one term and remove the rounding of each row's largest-score
 * key; a row whose weight several strong keys share keeps the others'
 * rounding (up to ~2^-9 of a value entry), which two terms remove at the cost
 * of the second product (the 64k-key, 9-draft call takes ~36 % longer).
 * Default 4096; 0 sends one term for every stream; INT_MAX two terms for every
 * stream.  Process-wide, for calls enqueued after it returns.  Returns MLA_OK,
 * or MLA_ERR_ARG for a negative `max_keys`.  Host-only.
 */
int mla_verify_attn_set_two_term_max_keys(int max_keys);

/*
 * Test controls; the pages have no counterpart.  Process-wide settings that
 * every later call reads (a relaxed atomic load per call, no environment
 * lookup), meant for the library's own tests:
 *   force_nsplit > 0  forces the number of key-range slices (at most one per
 *                     64-key tile of Smax), so that small inputs exercise the
 *                     split and merge path; it also changes what
 *                     mla_verify_attn_plan and the workspace sizes report,
 *                     and switches the device-side slice plan off.  0 restores
 *                     the library's own plan.
 *   stall != 0        makes work unit 0 of every later call withhold one of its
 *                     cache loads: its bounded waits run out after 2 s, the
 *                     call's kernels unwind and the device status reports
 *                     MLA_ERR_DEVICE_TIMEOUT.  0 switches this off.
 * Set these only while no call is being made from another thread.  Returns
 * MLA_OK, or MLA_ERR_ARG for a negative force_nsplit (nothing changes then).
 */
int mla_verify_attn_set_test_controls(int force_nsplit, int stall);

/*
 * mla_verify_attn without a caller-provided workspace.  This entry point has no
 * counterpart on the pages; it exists for callers that cannot allocate device
 * memory for scratch: code whose device memory is entirely pre-planned by its
 * own arena allocator (no way to hand out an extra buffer), latency-critical
 * loops where cudaMalloc/cudaFree would synchronise the device, and plain C
 * callers that link only this library and have no allocator of their own.
 *
 * Arguments and results are those of mla_verify_attn minus workspace and
 * workspace_bytes.  The key-split partials live instead in one fixed scratch
 * array of MLA_VERIFY_NOALLOC_SCRATCH_BYTES (32 MiB) compiled into this library
 * (a file-scope __device__ array: every GPU that loads the library holds it
 * until the process exits).  Calls whose partials need more than that return
 * MLA_ERR_WORKSPACE and enqueue nothing; use mla_verify_attn with a workspace
 * for them.  Nothing here calls cudaMalloc, cudaFree or any allocating routine.
 *
 * The first call on a device looks up the scratch array's device address
 * (cudaGetSymbolAddress) and caches it; make that first call before any stream
 * capture.  All calls on a device share that device's array, and it keeps the
 * last call's contents; nothing in it needs to start at zero (each call writes
 * every partial it later reads).  Calls on the same device that overlap on the
 * GPU (e.g. issued to two streams without ordering between them) race on the
 * array and may corrupt each other's results: order them, e.g. on one stream.
 */
#define MLA_VERIFY_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int mla_verify_attn_noalloc(const void* q_nope_abs, const void* q_rope, const void* kv,
                            const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len,
                            int H, int Smax, float scale, float* out, float* lse,
                            cudaStream_t stream);

/* ------------------------------------------------------------------------
 * The cache around a verify step.  The pages have no counterpart for these
 * entry points: they name a paged cache and its defragmentation as parts of the
 * serving system around the kernel.  One step over a paged cache is
 *   mla_blocks_extend   rows for the drafts: block table, lengths, slot map
 *   mla_cache_append    the drafts' rows into the pool, by slot
 *   mla_verify_attn_paged or mla_gqa_verify_attn_paged
 *   mla_cache_keep      the accepted path's rows move together
 *   mla_blocks_trim     lengths back to what was accepted, pages given back
 * All of them work in place on the caller's device arrays, in stream order,
 * read nothing on the host and may be captured into a CUDA graph.  Problems
 * only the GPU can see are recorded in the device status word.
 */

/*
 * Room for new tokens: grows every stream b by new_lens[b] tokens.  With
 *   have_b = ceil(seq_lens[b] / page_size), need_b = ceil((seq_lens[b] + new_lens[b]) / page_size) - have_b
 * the k-th new block of the batch (streams in order, then blocks in order) is
 * page free_pages[free_count - 1 - k]; it is written to its entry of
 * block_table.  Then seq_lens[b] += new_lens[b] and free_count -= sum need_b.
 * slots[t] is the pool row of the t-th new token (streams in order, positions
 * in order); slots past the last new token become -1.
 *
 *   seq_lens     [B] int32, in and out.
 *   new_lens     [B] int32, >= 0 (0 for streams that do not grow, unused ones too).
 *   block_table  [B, max_blocks] int32, in and out; only entries of new blocks are written.
 *   free_pages   [free_capacity] int32, a stack of distinct free pages; not written.
 *   free_count   [1] int32, pages on the stack; in and out.
 *   pool_pages   pages in the pool; an entry used outside [0, pool_pages) gives the
 *                token slot -1 and MLA_ERR_PAGE.
 *   slots        [max_tokens] int32 (may be NULL when max_tokens is 0).
 *   0 <= B <= 16384, page_size >= 1, max_blocks >= 1, max_blocks * page_size < 2^31,
 *   pool_pages * page_size < 2^31, free_capacity and max_tokens <= 2^31 - 2; all pointers
 *   4-byte aligned (slots: 16).
 *
 * Either the whole batch grows or nothing does: with too few free pages
 * (MLA_ERR_POOL), or a negative length, a stream that would outgrow its table
 * row or more than max_tokens new tokens (MLA_ERR_SEQLEN), tables, lengths and
 * the free list stay as they were and every slot is -1.
 */
int mla_blocks_extend(int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table, int B,
                      int max_blocks, int page_size, const int32_t* free_pages, int free_capacity,
                      int32_t* free_count, int pool_pages, int32_t* slots, int max_tokens,
                      cudaStream_t stream);

/*
 * The inverse: shortens every stream b to keep_lens[b] <= seq_lens[b] tokens
 * (0 gives all its pages back).  The R = sum_b ceil(seq_lens[b] / page_size) -
 * ceil(keep_lens[b] / page_size) released blocks go back onto the stack, the
 * k-th of the batch to free_pages[free_count + R - 1 - k], so that a trim back
 * to the old lengths undoes an extend exactly.  Then seq_lens[b] = keep_lens[b]
 * and free_count += R.  Released entries of block_table keep their values.
 * A stream's length that would grow or be negative (MLA_ERR_SEQLEN), a stack
 * that would outgrow free_capacity (MLA_ERR_POOL): nothing changes.  Pages
 * shared between streams must not be trimmed twice; nothing checks that.
 */
int mla_blocks_trim(int32_t* seq_lens, const int32_t* keep_lens, const int32_t* block_table, int B,
                    int max_blocks, int page_size, int32_t* free_pages, int free_capacity,
                    int32_t* free_count, cudaStream_t stream);

/*
 * Writes T rows into cache pools by slot: for every t with slots[t] >= 0
 *   pool_a[slots[t]] = a[t] (a_bytes bytes), pool_b[slots[t]] = b[t] (b_bytes bytes).
 * For the latent cache a = kv_c (1024 bytes), b = k_pe (128 bytes), pool_a the pool
 * and pool_b the pool's address + 1024, both with a row stride of 1152 bytes;
 * for separate keys and values a = k, b = v.  A contiguous cache is a pool of
 * B * Smax rows.
 *   a, b          T rows at a_stride / b_stride bytes, apart from the pools.
 *   pool_rows     rows in the pool(s), < 2^31; row strides in bytes.
 *   slots         [T] int32; a negative slot skips its token; one at or beyond
 *                 pool_rows skips it too and records MLA_ERR_SLOT.
 * Addresses, strides and widths are multiples of 16 bytes; b_bytes may be 0.
 * Slots of one call must be distinct: of two tokens with one slot, each 16-byte
 * piece of the row may come from either.
 */
int mla_cache_append(const void* a, long long a_stride, int a_bytes, void* pool_a, long long pool_a_stride,
                     const void* b, long long b_stride, int b_bytes, void* pool_b, long long pool_b_stride,
                     long long pool_rows, const int32_t* slots, int T, cudaStream_t stream);

/*
 * After a tree was verified: moves the rows of each stream's accepted drafts
 * together.  With prefix_b = seq_lens[b] - q_len, row prefix_b + j of stream b
 * takes the value row prefix_b + path[b][j] had before the call, for every
 * j < keep[b]; the other rows stay (seq_lens too: mla_blocks_trim with
 * prefix_b + keep[b] follows).  Any path is allowed, repeated drafts included.
 *   pool_a, pool_b as for mla_cache_append (b_bytes may be 0).
 *   block_table  [B, max_blocks] int32; row t of stream b is
 *                block_table[b][t / page_size] * page_size + t % page_size.
 *                A contiguous cache is one page of Smax rows per stream.
 *   seq_lens     [B] int32, q_len <= seq_lens[b] <= max_blocks * page_size where
 *                keep[b] > 0 (MLA_ERR_SEQLEN otherwise, and the stream is left as it was).
 *   path         [B, q_len] int32 draft indices in [0, q_len); entries past keep[b] are not used.
 *   keep         [B] int32 in [0, q_len].
 * A draft index or count out of range (MLA_ERR_SLOT) or a page outside the pool
 * (MLA_ERR_PAGE) leaves that stream as it was.  1 <= q_len <= 64.  No row may
 * be a draft row of two streams.
 */
int mla_cache_keep(void* pool_a, long long pool_a_stride, int a_bytes, void* pool_b,
                   long long pool_b_stride, int b_bytes, long long pool_rows,
                   const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                   const int32_t* path, const int32_t* keep, int B, int q_len, cudaStream_t stream);

/* Types of the grouped-head caches and queries. */
enum mla_dtype { MLA_BF16 = 0, MLA_FP16 = 1 };

/*
 * Verify attention with grouped query heads: the counterpart of
 * mla_verify_attn for models whose keys and values are separate and shared by
 * G = H / Hkv query heads (drafters, and targets without a latent cache).  For
 * stream b, draft i < q_len, head h < H and its key head g = h / G:
 *   s_t        = scale * sum_d q[b,i,h,d] k[b,t,g,d]        for the t visible to (b, i) as in mla_verify_attn
 *   out[b,i,h] = sum_{visible t} softmax(s)_t v[b,t,g,:]    (0 if nothing is visible)
 *   lse[b,i,h] = ln sum_{visible t} exp(s_t)                (-inf if nothing is visible)
 * q_len = 1 with mask bit 0 set is ordinary decoding.
 *
 *   q, out     [B, q_len, H, D], k and v [B, Smax, Hkv, D], all of type `dtype`, D = 64 or 128,
 *              H a multiple of Hkv; 16-byte aligned; out and lse [B, q_len, H] fp32 contiguous
 *              and apart from all inputs (q is still read while rows are written).
 *   strides    NULL for contiguous tensors, or a host array of nine element strides
 *              {q: batch, draft, head; k: batch, row, head; v: batch, row, head}, multiples
 *              of 8 in [8, 2^38); the innermost dimension is contiguous.  Strides of
 *              dimensions of size 1 are not used.
 *   seq_lens   as for mla_verify_attn, and 0 for an unused stream (out 0, lse -inf).  A
 *              stream with any other value outside [q_len, Smax] records MLA_ERR_SEQLEN and
 *              gets the same result.  Rows of k and v past seq_lens[b], and those of drafts
 *              that no draft of the stream sees (a batch padded to one q_len), may hold anything
 *              (NaN included).  A row of v that some draft sees must be finite, or the
 *              stream's other drafts get its NaN, too; NaN in a row of q, or in a key that a
 *              draft sees, gives that draft's rows NaN.
 *   tree_mask, scale, q_len, Smax and the errors as for mla_verify_attn; B < 2^20, and
 *              B * ceil(Smax / 64) * Hkv * ceil(q_len * H / Hkv / 128) < 2^31.
 *   workspace  at least mla_gqa_workspace_size(B, q_len, H, Hkv, D) bytes, 256-byte aligned;
 *              contents do not matter, not read after the call; calls that share it must not overlap.
 * Scores, softmax statistics and sums are fp32; the weights enter the product
 * with v in v's type and out is rounded once to `dtype`.  Deterministic for
 * fixed inputs and device.
 */
size_t mla_gqa_workspace_size(int B, int q_len, int H, int Hkv, int D);

int mla_gqa_verify_attn(const void* q, const void* k, const void* v, const int64_t* strides,
                        const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len, int H,
                        int Hkv, int D, int Smax, int dtype, float scale, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The same over a paged cache: k and v are pools [pool_rows, Hkv, D] (their
 * batch strides are not used), key t of stream b is pool row
 * block_table[b][t / page_size] * page_size + t % page_size, Smax = max_blocks *
 * page_size.  Any page_size >= 1 is read in place.  Entries past
 * ceil(seq_lens[b] / page_size) are not read; an entry outside the pool is
 * recorded as MLA_ERR_PAGE (that stream's results are then undefined).
 */
int mla_gqa_verify_attn_paged(const void* q, const void* k_pool, const void* v_pool,
                              const int64_t* strides, long long pool_rows, const int32_t* block_table,
                              int max_blocks, int page_size, const int32_t* seq_lens,
                              const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D,
                              int dtype, float scale, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Long caches kept small, for grouped heads: a window over the cache, a cache
 * held in 4 bits, and eviction by the weight that keys got.
 */

/*
 * mla_gqa_verify_attn and mla_gqa_verify_attn_paged with a sliding window: of
 * the keys that draft i sees by its mask, in the cache's order, it attends to
 * the last `window` and to those in the cache's first `sinks` rows.  For a mask of
 * ancestors (itself among them) that is what a window over positions gives: a
 * draft at depth n sees `window` - n - 1 keys of the prefix, and the sinks.
 *   window   >= 1; sinks >= 0 (MLA_ERR_SHAPE).
 * Rows of the cache from `sinks` up to max(0, seq_lens[b] - q_len - window) are not
 * used: they may hold anything (NaN included), and block_table entries of
 * pages that lie wholly there are not read, so such pages may have been given
 * away.  Tiles of 64 keys that lie there are not read either.  All other
 * arguments, results, errors and the workspace as for the calls without a window.
 */
int mla_gqa_verify_attn_window(const void* q, const void* k, const void* v, const int64_t* strides,
                               const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len, int H,
                               int Hkv, int D, int Smax, int dtype, float scale, int window, int sinks,
                               void* out, float* lse, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

int mla_gqa_verify_attn_window_paged(const void* q, const void* k_pool, const void* v_pool,
                                     const int64_t* strides, long long pool_rows, const int32_t* block_table,
                                     int max_blocks, int page_size, const int32_t* seq_lens,
                                     const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D,
                                     int dtype, float scale, int window, int sinks, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * A cache of Hkv heads x D values in 4 bits.  A pool row is
 *   Hkv * D / 2 bytes of codes (E2M1; heads in order, dimension 2 i in the low
 *     half of a head's byte i),
 *   Hkv * D / 16 bytes of steps (E4M3), one for every 16 values of a head,
 *   padding up to a multiple of 16 bytes, without a meaning and never written,
 * mla_gqa_fp4_row_bytes in all (0 for sizes that are not supported: D is 64 or
 * 128, Hkv <= MLA_FP4_MAX_HEADS), and stands for the values
 *   E2M1(code) * E4M3(step) * factor
 * with one factor for all rows of a pool, a positive number between 2^-64 and
 * 2^64 (MLA_ERR_ARG).  Rows move like any other: mla_cache_keep and
 * mla_cache_compact take them as bytes.
 */
#define MLA_FP4_MAX_HEADS 4096
size_t mla_gqa_fp4_row_bytes(int Hkv, int D);

/*
 * mla_cache_append into such pools: for every t with slots[t] >= 0 row slots[t] of
 * k_pool and v_pool takes k[t] and v[t], of type `dtype`.  For each 16 values x
 *   step = the E4M3 nearest to min(448, max|x| / (6 factor)),
 *   code = the E2M1 nearest to x / (step factor)   (both ties to even; 0 where the step is 0);
 * a group with a NaN gets a NaN step.  Exact for factors that are powers of two; with
 * others 6 factor, step factor and the quotients are rounded to fp32, so that a quotient
 * within 2^-22 (relative) of halfway between two numbers may become either.
 *   k, v            T rows [Hkv, D] at k_stride / v_stride bytes; 16-byte aligned, as all
 *                   rows and strides here; apart from the pools.
 *   k_held, v_held  NULL, or T rows [Hkv, D] of type `dtype` that take the values that
 *                   the pools now hold for each token (rounded to `dtype`; rows of skipped
 *                   tokens stay as they are): a prompt that attends to itself then
 *                   sees what later tokens will.
 * Slots as for mla_cache_append.  0 <= T < 2^30.
 */
int mla_gqa_cache_append_fp4(const void* k, long long k_stride, const void* v, long long v_stride, int Hkv, int D,
                             int dtype, float k_factor, float v_factor, void* k_pool, long long k_pool_stride,
                             void* v_pool, long long v_pool_stride, long long pool_rows, const int32_t* slots, int T,
                             void* k_held, long long k_held_stride, void* v_held, long long v_held_stride,
                             cudaStream_t stream);

/*
 * mla_gqa_verify_attn_paged over such pools: the formula with the values that the
 * rows stand for as k and v.
 *   q, out, q_strides  of type `dtype`; q_strides NULL or q's three element strides.
 *   k_pool, v_pool     [pool_rows] rows at k_pool_stride / v_pool_stride bytes (multiples of
 *                      16 of at least mla_gqa_fp4_row_bytes(Hkv, D)); 16-byte aligned.
 *   k_factor, v_factor the pools' factors; scale * k_factor finite (MLA_ERR_ARG).
 *   workspace          mla_gqa_fp4_workspace_size(B, q_len, H, Hkv, D) bytes.
 * A contiguous cache [B, Smax] is a pool of one page of Smax rows a stream.  All
 * other arguments, results and errors as for mla_gqa_verify_attn_paged (a step of
 * NaN is a row that is not finite).  A row of q enters the products in fp16,
 * brought to its range by a power of two: values below 2^-28 of the row's largest
 * lose digits.  The weights are fp16, too.
 */
size_t mla_gqa_fp4_workspace_size(int B, int q_len, int H, int Hkv, int D);

int mla_gqa_verify_attn_fp4_paged(const void* q, const int64_t* q_strides, const void* k_pool, long long k_pool_stride,
                                  const void* v_pool, long long v_pool_stride, long long pool_rows,
                                  const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                                  const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D, int dtype,
                                  float scale, float k_factor, float v_factor, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * The attention weight that each key got from a verify (or decoding) step, added
 * to what is there: for key head g of stream b and every key t < seq_lens[b]
 *   weights[b][g][t] += sum exp(s - lse[b,i,h])
 * over the drafts i that see t by their mask and the query heads h of g, s the
 * score as in mla_gqa_verify_attn.  With the lse of that call over the same keys a
 * row's weights add up to 1.
 *   q, k, strides (q's three and k's three), seq_lens, tree_mask, the sizes, the
 *              types, the paged form and the errors as for mla_gqa_verify_attn
 *              (streams of another length than q_len .. Smax get nothing).
 *   lse        [B, q_len, H] fp32.  A row with lse +inf or -inf adds nothing, whatever
 *              its q holds: +inf leaves out drafts that were not accepted, or padding.
 *   weights    [B, Hkv, Smax] fp32 (Smax = max_blocks * page_size), in and out; entries
 *              from seq_lens[b] on are neither read nor written.
 * Scores, exponentials and sums are fp32; deterministic.  No workspace.
 * Sums belong to places of the cache, and no other call than mla_cache_compact touches
 * them: mla_cache_keep moves the accepted drafts' rows without their sums, and a place
 * that mla_blocks_trim gives up keeps its sum, from which its next key would go on.  So
 * after a step that does not keep all its drafts either move those sums as the rows are
 * moved and clear the places behind them, or use mla_cache_compact in place of
 * mla_cache_keep (kept: the whole prefix, then the accepted drafts' places).
 */
int mla_gqa_attn_weights(const void* q, const void* k, const int64_t* strides, const int32_t* seq_lens,
                         const uint32_t* tree_mask, const float* lse, int B, int q_len, int H, int Hkv, int D, int Smax,
                         int dtype, float scale, float* weights, cudaStream_t stream);

int mla_gqa_attn_weights_paged(const void* q, const void* k_pool, const int64_t* strides, long long pool_rows,
                               const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                               const uint32_t* tree_mask, const float* lse, int B, int q_len, int H, int Hkv, int D,
                               int dtype, float scale, float* weights, cudaStream_t stream);

/*
 * Which keys of each stream stay, by the weight that they got.  A stream of S =
 * seq_lens[b] > budget keys keeps its first `sinks`, its last `recent`, and of the
 * keys between those with the largest totals, to `budget` in all; of equal totals
 * the first.  The total of key t is the fp32 sum of weights[b][h][t] over the heads
 * h, in order (NaN counts as the largest).  A stream of at most `budget` keys
 * keeps them all.
 *   weights    [B, Hkv, Smax] fp32; only t < seq_lens[b] is read.
 *   kept       [B, budget] int32, out: the kept positions in order, -1 behind them.
 *   keep_lens  [B] int32, out: min(seq_lens[b], budget), as mla_blocks_trim takes it.
 *   workspace  mla_evict_workspace_size(B, Smax) bytes, 4-byte aligned (NULL where that
 *              is 0, as up to 393,216 keys); contents do not matter.
 *   0 <= B < 2^20, 1 <= Smax < 2^24, 1 <= Hkv <= 65536, sinks, recent >= 0 and
 *   sinks + recent <= budget <= 2^30 (MLA_ERR_SHAPE).
 * A seq_lens[b] outside [0, Smax] records MLA_ERR_SEQLEN and keeps nothing.
 */
size_t mla_evict_workspace_size(int B, int Smax);

int mla_evict_select(const float* weights, const int32_t* seq_lens, int B, int Hkv, int Smax, int sinks, int recent,
                     int32_t* kept, int budget, int32_t* keep_lens, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream);

/*
 * The rows that stay move together, in place: row j of stream b takes the value
 * that row kept[b][j] had before the call, for every j < keep_lens[b]; what is left
 * behind them keeps no particular value.  seq_lens stays as it is: mla_blocks_trim to keep_lens follows.
 *   pool_a, pool_b, block_table, max_blocks, page_size  as for mla_cache_keep;
 *              max_blocks * page_size <= 2^30 and budget <= 2^30 (MLA_ERR_SHAPE).
 *   weights    NULL, or [B, Hkv, max_blocks * page_size] fp32 that move along; entries
 *              from keep_lens[b] up to seq_lens[b] become 0.
 *   kept       [B, budget] int32, increasing in each stream, as mla_evict_select leaves it.
 *   keep_lens  [B] int32 in [0, min(seq_lens[b], budget)]
 * An entry of kept below its own place or not below seq_lens[b] records
 * MLA_ERR_SLOT and its row stays; entries in another order leave rows with
 * undefined contents.  A count or length out of range (MLA_ERR_SLOT,
 * MLA_ERR_SEQLEN) leaves the stream as it was; a row whose page lies outside the pool
 * (MLA_ERR_PAGE) is not moved.  No page may belong to two streams.
 */
int mla_cache_compact(void* pool_a, long long pool_a_stride, int a_bytes, void* pool_b, long long pool_b_stride,
                      int b_bytes, long long pool_rows, float* weights, int Hkv, const int32_t* block_table,
                      int max_blocks, int page_size, const int32_t* seq_lens, const int32_t* kept, int budget,
                      const int32_t* keep_lens, int B, cudaStream_t stream);

/*
 * The calls of the two sections above with their arguments in one array of 64-bit values,
 * in the order of their declarations: integers and addresses as such, a float
 * as the bits of a double.  For bindings to which each argument costs more than
 * its share of the launch.  Returns what the call returns, or MLA_ERR_ARG for an
 * unknown `call`; an integer argument that does not fit its type is MLA_ERR_SHAPE.
 */
enum mla_packed {
  MLA_CALL_BLOCKS_EXTEND = 0,
  MLA_CALL_BLOCKS_TRIM = 1,
  MLA_CALL_CACHE_APPEND = 2,
  MLA_CALL_CACHE_KEEP = 3,
  MLA_CALL_GQA_VERIFY_ATTN = 4,
  MLA_CALL_GQA_VERIFY_ATTN_PAGED = 5,
  /* 6 and 7 are not calls */
  MLA_CALL_GQA_VERIFY_ATTN_WINDOW = 8,
  MLA_CALL_GQA_VERIFY_ATTN_WINDOW_PAGED = 9,
  MLA_CALL_GQA_CACHE_APPEND_FP4 = 10,
  MLA_CALL_EVICT_SELECT = 11,
  MLA_CALL_CACHE_COMPACT = 12,
  MLA_CALL_GQA_ATTN_WEIGHTS = 13,
  MLA_CALL_GQA_ATTN_WEIGHTS_PAGED = 14,
  MLA_CALL_GQA_VERIFY_ATTN_FP4_PAGED = 15
};
int mla_call_packed(int call, const int64_t* args);

#ifdef __cplusplus
}
#endif
#endif /* MLA_VERIFY_ATTN_H */
