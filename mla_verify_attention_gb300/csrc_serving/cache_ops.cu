// The cache operators around a verify step: block tables and slot maps from
// request lengths (mla_blocks_extend / _trim), rows into a pool by slot
// (mla_cache_append) and the accepted path's rows together (mla_cache_keep).
// Declared, with their exact meaning, in include/mla_verify_attn.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "launch.h"
#include "mla_verify_attn.h"
#include "ptx.cuh"

namespace mla {

// ------------------------------------------------------------ block tables
//
// need_b and the new tokens of each stream are summed up by a scan over the
// batch; every new token and every new block then finds its stream by a binary
// search in those sums, so that the work is even however ragged the batch is
// (one long prompt among single tokens).
//
// A call for a verify step is a chain of a few dependent reads, so it is one
// block of as many threads as there are streams or token quads, launched as a
// dependent of the grid before it: 3 us for 8 streams x 9 tokens (5.3 us with
// 1,024 threads and a plain launch).  More work is shared by a cluster of eight
// blocks, each with a scan of its own; the first writes the lengths and the free
// count once all have read them (the cluster's barrier).  Extends beyond that (of
// prompts) are shared by as many blocks as they fill, and a second grid takes the
// place of the barrier.  Extend and trim, us, with one block / a cluster / two
// grids for the extend and a cluster for the trim:
//   64 streams x 9 tokens, page 16     7.0    7.2    8.1
//   64 x 64                            7.0    6.5    7.2
//   8 x 4,096, page 64                13.7    6.9    6.9
//   64 x 1,024, page 16               26.4    9.4    7.7
//   512 x 64                          18.6    9.2    9.5
//   512 x 424                         91.7   22.2    9.3
// How many blocks a trim releases is not known on the host: one block of threads
// does it where the table itself is small (an empty trim 1.7 us, 2.0 with a
// cluster).
constexpr int kMaxThreads = 1024;
constexpr int kMaxStreams = 16384;     // three int32 a stream in shared memory
constexpr int kOneBlockTokens = 2048;
constexpr int kClusterTokens = 32768;
constexpr int kOneBlockStreams = 16, kOneBlockEntries = 16384;
constexpr unsigned kClusterBlocks = 8;
constexpr int kMostBlocks = 152;
// Sums stay there: more than any limit they are held to, and twice as much is
// still less than 2^32.  (A test before the addition cost an extend and a trim
// of 512 prompts 0.3 us.)
constexpr unsigned kFull = (1u << 31) - 1;
constexpr int kMostCounted = (1u << 31) - 2;

struct BlocksParams {
  int32_t* seq_lens;
  const int32_t* target;      // extend: new tokens; trim: lengths to keep
  int32_t* table;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* slots;
  unsigned int* status;
  int B, max_blocks, free_capacity, pool_pages, max_tokens;
  Divisor page;
};

__device__ __forceinline__ unsigned add_full(unsigned a, unsigned b) { return min(a + b, kFull); }

// Largest i in [0, n) with pre[i] <= x, for pre[0] = 0 <= x < pre[n].
__device__ __forceinline__ int find_stream(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }

// What a grid does: everything, in one block or in one cluster; or one of the two parts.
enum { kAll = 0, kCluster = 1, kItems = 2, kCommit = 3 };

template <bool kExtend, int kPart>
__global__ void __launch_bounds__(kMaxThreads, 1) blocks_kernel(const BlocksParams p) {
  extern __shared__ int shared[];
  int* const base_len = shared;                   // [B] extend: old lengths; trim: kept lengths
  int* const blk_pre = base_len + p.B;            // [B + 1] blocks before stream b
  int* const tok_pre = blk_pre + p.B + 1;         // [B + 1] new tokens before stream b (extend)
  __shared__ unsigned warp_sum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, first = blockIdx.x * threads + tid, all_threads = gridDim.x * threads;
  grid_dependency_wait();
  if (tid == 0) grid_launch_dependents();
  const int fc = *p.free_count;

  // Each thread sums a run of consecutive streams; then a scan over threads.
  const int per = (p.B + threads - 1) / threads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const long long room = static_cast<long long>(p.max_blocks) * p.page.d;
  unsigned blocks = 0, tokens = 0;
  bool bad = false;
  int len = 0, x = 0;                             // of the last stream: the only one of most calls' threads
  for (int b = b0; b < b1; ++b) {
    len = p.seq_lens[b];
    x = p.target[b];
    const bool wrong = len < 0 || x < 0 || (kExtend ? len + static_cast<long long>(x) > room : x > len || len > room);
    bad |= wrong;
    if (wrong) continue;
    blocks = add_full(blocks, kExtend ? p.page.up(len + x) - p.page.up(len) : p.page.up(len) - p.page.up(x));
    if (kExtend) tokens = add_full(tokens, x);
  }
  unsigned ib = blocks, it = tokens;              // inclusive sums over the warp's threads
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned ob = __shfl_up_sync(0xFFFFFFFFu, ib, d), ot = __shfl_up_sync(0xFFFFFFFFu, it, d);
    if (lane >= d) {
      ib = add_full(ib, ob);
      it = add_full(it, ot);
    }
  }
  if (lane == 31) {
    warp_sum[0][warp] = ib;
    warp_sum[1][warp] = it;
  }
  bad = __syncthreads_or(bad) != 0;
  // Every warp scans the warps' sums.
  unsigned wb = lane < threads / 32 ? warp_sum[0][lane] : 0, wt = lane < threads / 32 ? warp_sum[1][lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned ob = __shfl_up_sync(0xFFFFFFFFu, wb, d), ot = __shfl_up_sync(0xFFFFFFFFu, wt, d);
    if (lane >= d) {
      wb = add_full(wb, ob);
      wt = add_full(wt, ot);
    }
  }
  const unsigned all_b = __shfl_sync(0xFFFFFFFFu, wb, 31), all_t = __shfl_sync(0xFFFFFFFFu, wt, 31);
  const unsigned before_b = warp ? __shfl_sync(0xFFFFFFFFu, wb, warp - 1) : 0;
  const unsigned before_t = warp ? __shfl_sync(0xFFFFFFFFu, wt, warp - 1) : 0;

  // Anything wrong: the batch stays as it was (the same verdict in every block).
  const bool no_pages = fc < 0 || fc > p.free_capacity ||
                        all_b > static_cast<unsigned>(kExtend ? fc : p.free_capacity - fc);
  bad |= kExtend && all_t > static_cast<unsigned>(p.max_tokens);
  if (bad || no_pages) {
    if (kExtend && kPart != kCommit)
      for (long long t = first; t < p.max_tokens; t += all_threads) p.slots[t] = -1;
    if (kPart != kItems && first == 0) atomicOr(p.status, bad ? kBitSeqLen : kBitPool);
    return;
  }
  const int n_blocks = static_cast<int>(all_b), n_tokens = static_cast<int>(all_t);

  if (kPart != kCommit) {
    int eb = static_cast<int>(before_b + ib - blocks), et = static_cast<int>(before_t + it - tokens);
    for (int b = b0; b < b1; ++b) {
      if (per > 1) {
        len = p.seq_lens[b];
        x = p.target[b];
      }
      base_len[b] = kExtend ? len : x;
      blk_pre[b] = eb;
      eb += kExtend ? p.page.up(len + x) - p.page.up(len) : p.page.up(len) - p.page.up(x);
      if (kExtend) {
        tok_pre[b] = et;
        et += x;
      }
    }
    if (tid == 0) {
      blk_pre[p.B] = n_blocks;
      if (kExtend) tok_pre[p.B] = n_tokens;
    }
    __syncthreads();
    if (kPart == kCluster) cluster_arrive();         // this block has read the lengths and the free count

    // Four consecutive blocks a thread: one search (the searches' shared-memory
    // reads are what a release of thousands of pages costs), and four reads
    // under way together.
    for (long long k4 = 4ll * first; k4 < n_blocks; k4 += 4ll * all_threads) {
      const int k0 = static_cast<int>(k4), n = min(4, n_blocks - k0);
      int b = find_stream(blk_pre, p.B, k0);
      int end = blk_pre[b + 1];
      int32_t* entry = p.table + static_cast<size_t>(b) * p.max_blocks + p.page.up(base_len[b]) + (k0 - blk_pre[b]);
      int32_t* at[4];
      int page[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= n) break;
        if (k0 + e >= end) {
          do end = blk_pre[++b + 1]; while (k0 + e >= end);
          entry = p.table + static_cast<size_t>(b) * p.max_blocks + p.page.up(base_len[b]);
        }
        at[e] = entry++;
        page[e] = kExtend ? p.free_pages[fc - 1 - (k0 + e)] : *at[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= n) break;
        if (kExtend) *at[e] = page[e];
        else p.free_pages[fc + n_blocks - 1 - (k0 + e)] = page[e];
      }
    }
    if (kExtend) {
      // Four consecutive tokens a thread: one search, one 16-byte store.  The
      // page of a token's new block is read from the free list, not the table.
      bool off = false;
      for (long long t4 = 4ll * first; t4 < p.max_tokens; t4 += 4ll * all_threads) {
        const int t0 = static_cast<int>(t4);
        int s[4] = {-1, -1, -1, -1};
        if (t0 < n_tokens) {
          int b = find_stream(tok_pre, p.B, t0);
          int held = -1, row0 = 0;                 // the block that `row0` belongs to, of stream b
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + e;
            if (t >= n_tokens) break;
            while (t >= tok_pre[b + 1]) {
              ++b;
              held = -1;
            }
            const int old = base_len[b], pos = old + (t - tok_pre[b]), blk = p.page.of(pos);
            if (blk != held) {
              const int have = p.page.up(old);
              const int page = blk < have ? p.table[static_cast<size_t>(b) * p.max_blocks + blk]
                                          : p.free_pages[fc - 1 - (blk_pre[b] + blk - have)];
              const bool ok = page >= 0 && page < p.pool_pages;
              off |= !ok;
              row0 = ok ? page * static_cast<int>(p.page.d) : -1;
              held = blk;
            }
            s[e] = row0 < 0 ? -1 : row0 + (pos - blk * static_cast<int>(p.page.d));
          }
        }
        if (p.max_tokens - t0 >= 4) {
          *reinterpret_cast<int4*>(p.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
        } else {
          for (int e = 0; t0 + e < p.max_tokens; ++e) p.slots[t0 + e] = s[e];
        }
      }
      if (off) atomicOr(p.status, kBitPage);
    }
  }

  if (kPart == kCluster) {
    __syncwarp();
    cluster_wait();
    if (blockIdx.x != 0) return;
  }
  if (kPart != kItems) {
    // Every thread reads and writes its own streams; the lengths that the
    // searches above used are in shared memory.
    for (int b = b0; b < b1; ++b) {
      if (per > 1) {
        len = p.seq_lens[b];
        x = p.target[b];
      }
      p.seq_lens[b] = kExtend ? len + x : x;
    }
    __syncthreads();                               // every thread has used the free count it read
    if (tid == 0) *p.free_count = kExtend ? fc - n_blocks : fc + n_blocks;
  }
}

using BlocksFn = void (*)(BlocksParams);

int launch_blocks(BlocksFn fn, const BlocksParams& p, unsigned blocks, unsigned threads, cudaStream_t stream,
                  unsigned cluster = 1) {
  // Beyond 48 KB, the kernel's own arrays (256 bytes, room for 1 KB) counted, a
  // block's shared memory has to be asked for.
  const size_t smem = (3 * static_cast<size_t>(p.B) + 2) * sizeof(int);
  if (smem > 47 * 1024 && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((3 * kMaxStreams + 2) * sizeof(int))) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return launch_dependent(fn, p, dim3(blocks), threads, smem, stream, cluster);
}

// Threads of a block that has this many streams and items to see to.
unsigned threads_for(long long n) {
  return n <= 128 ? 128 : (n >= kMaxThreads ? kMaxThreads : static_cast<unsigned>((n + 31) / 32 * 32));
}

// The same of blocks that share the work: 1,024 threads only to scan many streams.
int shared_threads(int B) { return B > kMaxThreads / 2 ? kMaxThreads : kMaxThreads / 2; }

bool blocks_shape_ok(int B, int max_blocks, int page, int free_capacity) {
  return B >= 0 && B <= kMaxStreams && max_blocks >= 1 && page >= 1 && free_capacity >= 0 &&
         free_capacity <= kMostCounted && static_cast<long long>(max_blocks) * page < (1ll << 31);
}

// ------------------------------------------------------------ rows by slot
//
// Pure copies.  One warp a row, its 16-byte units over the lanes, four loads
// in flight a lane: the rows of one token are 1152 bytes (latent) to a few KB.
// 32,251 tokens of 4 KB, cut out of rows of 8 KB: 40.9 us, 6.5 TB/s (95 % of the
// measured copy rate); 72 latent rows: 1.7 us.
struct RowsParams {
  uint8_t* pool[2];
  long long pool_stride[2];
  int units[2];                 // 16-byte units of a row in each pool
  long long pool_rows;
  unsigned int* status;
};

struct AppendParams {
  RowsParams r;
  const uint8_t* src[2];
  long long src_stride[2];
  const int32_t* slots;
  int T;
};

constexpr int kAppendWarps = 8;

__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if (t >= p.T) return;
  const int slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.r.pool_rows) {
    if (lane == 0) atomicOr(p.r.status, kBitSlot);
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4* src = reinterpret_cast<const uint4*>(p.src[k] + t * p.src_stride[k]);
    uint4* dst = reinterpret_cast<uint4*>(p.r.pool[k] + slot * p.r.pool_stride[k]);
    const int n = p.r.units[k];
    for (int c = lane; c < n; c += 128) {
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + 32 * e < n) v[e] = src[c + 32 * e];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + 32 * e < n) dst[c + 32 * e] = v[e];
    }
  }
}

struct KeepParams {
  RowsParams r;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* path;
  const int32_t* keep;
  int max_blocks, pool_pages, B, q;
  int columns;                  // a block
  Divisor page;
};

// One block a stream and one or two 512-byte columns of the pool rows: eight
// warps read the path's rows (kRows a warp at most) into registers, and after a
// barrier write them to their new places, so that any path is safe in place.
// Rows that stay where they are are neither read nor written.
// Before that the block works out the rows (a thread a row; count, length and
// path are read together, then the pages): two dependent reads that the columns
// share.  One column while those blocks all fit the device (8 streams x 9
// latent rows 2.1 us, 2.5 with two); two beyond that (256 streams, 17 of 33 rows
// of 4 KB on average, of which 13 move: 6.4 us; one 6.7, four 7.3 us.  Reading and
// writing the kept rows at the copy rate would take 5.1 us, those that move 4.2).
// Fewer rows a warp leave registers for more blocks: six an SM with five rows
// (6.8 us with eight rows and four blocks, 8.1 with three).
constexpr int kKeepWarps = 8;
constexpr int kKeepBlocks = 6;                     // an SM, about

template <int kRows>
__global__ void __launch_bounds__(32 * kKeepWarps, kRows <= 5 ? kKeepBlocks : 4) keep_kernel(const KeepParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int rows[2][64];                      // pool rows the j-th kept draft moves from / to
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int units = p.r.units[0] + p.r.units[1];
  const int to = threadIdx.x & 1, j_mine = threadIdx.x >> 1;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int n = p.keep[b], len = p.seq_lens[b];
    int i = j_mine;
    if (to == 0 && j_mine < p.q) i = p.path[static_cast<size_t>(b) * p.q + j_mine];   // (used below keep[b] only)
    if (n == 0) continue;
    uint32_t wrong = 0;
    if (n < 0 || n > p.q) wrong = kBitSlot;
    else if (len < p.q || len > static_cast<long long>(p.max_blocks) * p.page.d) wrong = kBitSeqLen;
    else if (j_mine < n) {
      if (i < 0 || i >= p.q) {
        wrong = kBitSlot;
        i = 0;
      }
      const int pos = len - p.q + i, blk = p.page.of(pos);
      const int page = p.table[static_cast<size_t>(b) * p.max_blocks + blk];
      if (page < 0 || page >= p.pool_pages) wrong |= kBitPage;
      else rows[to][j_mine] = page * static_cast<int>(p.page.d) + (pos - blk * static_cast<int>(p.page.d));
    }
    if (wrong) atomicOr(p.r.status, wrong);
    if (__syncthreads_or(static_cast<int>(wrong))) continue;   // this stream stays as it was
#pragma unroll 1
    for (int col = 0; col < p.columns; ++col) {
      const int c = (static_cast<int>(blockIdx.x) * p.columns + col) * 32 + lane;
      // (Selected, not indexed: an index would put the parameters on the stack.)
      const bool second = c >= p.r.units[0];
      uint8_t* const pool = second ? p.r.pool[1] + 16ll * (c - p.r.units[0]) : p.r.pool[0] + 16ll * c;
      const long long stride = second ? p.r.pool_stride[1] : p.r.pool_stride[0];
      uint4 v[kRows];
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int j = warp + kKeepWarps * e;
        if (j < n && c < units && rows[0][j] != rows[1][j])
          v[e] = *reinterpret_cast<const uint4*>(pool + rows[0][j] * stride);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int j = warp + kKeepWarps * e;
        if (j < n && c < units && rows[0][j] != rows[1][j])
          *reinterpret_cast<uint4*>(pool + rows[1][j] * stride) = v[e];
      }
    }
    __syncthreads();                                            // `rows` is rewritten for the next stream
  }
}

// Checks of a pool pair that append and keep share.
int rows_params(void* pool_a, long long stride_a, int bytes_a, void* pool_b, long long stride_b, int bytes_b,
                long long pool_rows, RowsParams* r) {
  if (bytes_a < 1 || bytes_b < 0 || pool_rows < 1 || pool_rows >= (1ll << 31)) return MLA_ERR_SHAPE;
  const long long limit = 1ll << 32;
  if (stride_a < bytes_a || stride_a > limit || (bytes_b > 0 && (stride_b < bytes_b || stride_b > limit)))
    return MLA_ERR_SHAPE;
  if (!pool_a || (bytes_b > 0 && !pool_b)) return MLA_ERR_NULLPTR;
  if (!aligned_to(pool_a, 16) || stride_a % 16 || bytes_a % 16 || bytes_b % 16 ||
      (bytes_b > 0 && (!aligned_to(pool_b, 16) || stride_b % 16)))
    return MLA_ERR_ALIGN;
  r->pool[0] = static_cast<uint8_t*>(pool_a);
  r->pool[1] = static_cast<uint8_t*>(bytes_b > 0 ? pool_b : pool_a);
  r->pool_stride[0] = stride_a;
  r->pool_stride[1] = bytes_b > 0 ? stride_b : 0;
  r->units[0] = bytes_a / 16;
  r->units[1] = bytes_b / 16;
  r->pool_rows = pool_rows;
  return MLA_OK;
}

}  // namespace mla

extern "C" {

int mla_blocks_extend(int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table, int B,
                      int max_blocks, int page_size, const int32_t* free_pages, int free_capacity,
                      int32_t* free_count, int pool_pages, int32_t* slots, int max_tokens,
                      cudaStream_t stream) {
  using namespace mla;
  if (!blocks_shape_ok(B, max_blocks, page_size, free_capacity) || max_tokens < 0 || max_tokens > kMostCounted ||
      pool_pages < 1 ||
      static_cast<long long>(pool_pages) * page_size >= (1ll << 31))
    return MLA_ERR_SHAPE;
  if (B == 0 && max_tokens == 0) return MLA_OK;
  if ((B > 0 && (!seq_lens || !new_lens || !block_table)) || !free_count || (free_capacity > 0 && !free_pages) ||
      (max_tokens > 0 && !slots))
    return MLA_ERR_NULLPTR;
  if (!aligned_to(seq_lens, 4) || !aligned_to(new_lens, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(free_pages, 4) || !aligned_to(free_count, 4) || !aligned_to(slots, 16))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  const int st = device_common(&d);
  if (st != MLA_OK) return st;
  BlocksParams p = {seq_lens, new_lens, block_table, const_cast<int32_t*>(free_pages), free_count, slots,
                    d.status_word, B, max_blocks, free_capacity, pool_pages, max_tokens, Divisor(page_size)};
  const long long quads = (static_cast<long long>(max_tokens) + 3) / 4;
  if (max_tokens <= kOneBlockTokens && B <= kMaxThreads)
    return launch_blocks(blocks_kernel<true, kAll>, p, 1, threads_for(quads > B ? quads : B), stream);
  const int threads = shared_threads(B);
  if (max_tokens <= kClusterTokens)
    return launch_blocks(blocks_kernel<true, kCluster>, p, kClusterBlocks, threads, stream, kClusterBlocks);
  const long long wanted = (quads + threads - 1) / threads;
  const unsigned blocks = static_cast<unsigned>(wanted < kMostBlocks ? wanted : kMostBlocks);
  const int first = launch_blocks(blocks_kernel<true, kItems>, p, blocks, threads, stream);
  return first != MLA_OK ? first : launch_blocks(blocks_kernel<true, kCommit>, p, 1, threads_for(B), stream);
}

int mla_blocks_trim(int32_t* seq_lens, const int32_t* keep_lens, const int32_t* block_table, int B,
                    int max_blocks, int page_size, int32_t* free_pages, int free_capacity,
                    int32_t* free_count, cudaStream_t stream) {
  using namespace mla;
  if (!blocks_shape_ok(B, max_blocks, page_size, free_capacity)) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!seq_lens || !keep_lens || !block_table || !free_count || (free_capacity > 0 && !free_pages))
    return MLA_ERR_NULLPTR;
  if (!aligned_to(seq_lens, 4) || !aligned_to(keep_lens, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(free_pages, 4) || !aligned_to(free_count, 4))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  const int st = device_common(&d);
  if (st != MLA_OK) return st;
  BlocksParams p = {seq_lens, keep_lens, const_cast<int32_t*>(block_table), free_pages, free_count, nullptr,
                    d.status_word, B, max_blocks, free_capacity, 0, 0, Divisor(page_size)};
  if (B <= kOneBlockStreams && static_cast<long long>(B) * max_blocks <= kOneBlockEntries)
    return launch_blocks(blocks_kernel<false, kAll>, p, 1, threads_for(B), stream);
  return launch_blocks(blocks_kernel<false, kCluster>, p, kClusterBlocks, shared_threads(B), stream, kClusterBlocks);
}

int mla_cache_append(const void* a, long long a_stride, int a_bytes, void* pool_a, long long pool_a_stride,
                     const void* b, long long b_stride, int b_bytes, void* pool_b, long long pool_b_stride,
                     long long pool_rows, const int32_t* slots, int T, cudaStream_t stream) {
  using namespace mla;
  if (T < 0) return MLA_ERR_SHAPE;
  AppendParams p;
  int st = rows_params(pool_a, pool_a_stride, a_bytes, pool_b, pool_b_stride, b_bytes, pool_rows, &p.r);
  if (st != MLA_OK) return st;
  if (a_stride < 0 || b_stride < 0) return MLA_ERR_SHAPE;
  if (T == 0) return MLA_OK;
  if (!a || (b_bytes > 0 && !b) || !slots) return MLA_ERR_NULLPTR;
  if (!aligned_to(a, 16) || a_stride % 16 || (b_bytes > 0 && (!aligned_to(b, 16) || b_stride % 16)) ||
      !aligned_to(slots, 4))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  st = device_common(&d);
  if (st != MLA_OK) return st;
  p.r.status = d.status_word;
  p.src[0] = static_cast<const uint8_t*>(a);
  p.src[1] = static_cast<const uint8_t*>(b_bytes > 0 ? b : a);
  p.src_stride[0] = a_stride;
  p.src_stride[1] = b_bytes > 0 ? b_stride : 0;
  p.slots = slots;
  p.T = T;
  return launch_dependent(append_kernel, p,
                          dim3(static_cast<unsigned>((static_cast<long long>(T) + kAppendWarps - 1) / kAppendWarps)),
                          32 * kAppendWarps, 0, stream);
}

int mla_cache_keep(void* pool_a, long long pool_a_stride, int a_bytes, void* pool_b,
                   long long pool_b_stride, int b_bytes, long long pool_rows,
                   const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                   const int32_t* path, const int32_t* keep, int B, int q_len, cudaStream_t stream) {
  using namespace mla;
  KeepParams p;
  if (B < 0 || q_len < 1 || q_len > 64 || max_blocks < 1 || page_size < 1 ||
      static_cast<long long>(max_blocks) * page_size >= (1ll << 31))
    return MLA_ERR_SHAPE;
  int st = rows_params(pool_a, pool_a_stride, a_bytes, pool_b, pool_b_stride, b_bytes, pool_rows, &p.r);
  if (st != MLA_OK) return st;
  if (pool_rows < page_size) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!block_table || !seq_lens || !path || !keep) return MLA_ERR_NULLPTR;
  if (!aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(path, 4) || !aligned_to(keep, 4))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  st = device_common(&d);
  if (st != MLA_OK) return st;
  p.r.status = d.status_word;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.path = path;
  p.keep = keep;
  p.max_blocks = max_blocks;
  p.page = Divisor(page_size);
  p.pool_pages = static_cast<int>(pool_rows / page_size);
  p.B = B;
  p.q = q_len;
  const unsigned cols = (static_cast<unsigned>(p.r.units[0]) + p.r.units[1] + 31) / 32;
  p.columns = static_cast<long long>(cols) * B <= kKeepBlocks * d.sms ? 1 : 2;
  const dim3 grid((cols + p.columns - 1) / p.columns, B < 65535 ? B : 65535);
  void (*const fn)(KeepParams) = q_len <= 2 * kKeepWarps   ? keep_kernel<2>
                                 : q_len <= 5 * kKeepWarps ? keep_kernel<5>
                                                           : keep_kernel<8>;
  return launch_dependent(fn, p, grid, 32 * kKeepWarps, 0, stream);
}

}  // extern "C"
