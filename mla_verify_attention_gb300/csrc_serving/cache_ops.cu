// The cache operators around a verify step: block tables and slot maps from
// request lengths (mla_blocks_extend / _trim), rows into a pool by slot
// (mla_cache_append) and the accepted path's rows together (mla_cache_keep).
// Declared, with their exact meaning, in include/mla_verify_attn.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "mla_verify_attn.h"
#include "ptx.cuh"

namespace mla {

// ------------------------------------------------------------ block tables
//
// need_b and the new tokens of each stream are summed up by a scan over the
// batch; every new token and every new block then finds its stream by a binary
// search in those sums, so that the work is even however ragged the batch is
// (one long prompt among single tokens).  The call is latency bound (a few
// dependent global reads and the scan), so it is one launch: one block, or for
// many tokens one cluster of eight blocks that each repeat the scan and share
// the tokens.  The in-place results (lengths, free count) are written by one
// block after a cluster barrier, when every block has read the old ones.
constexpr int kBlockThreads = 1024;
constexpr int kMaxStreams = 16384;     // three int32 a stream in shared memory
constexpr int kClusterBlocks = 8;

struct BlocksParams {
  int32_t* seq_lens;
  const int32_t* target;      // extend: new tokens; trim: lengths to keep
  int32_t* table;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* slots;
  unsigned int* status;
  int B, max_blocks, page, free_capacity, pool_pages, max_tokens;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Largest i in [0, n) with pre[i] <= x, for pre[0] = 0 <= x < pre[n].
__device__ __forceinline__ int find_stream(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool kExtend>
__global__ void __launch_bounds__(kBlockThreads, 1) blocks_kernel(const BlocksParams p) {
  extern __shared__ int shared[];
  int* const base_len = shared;                   // [B] extend: old lengths; trim: kept lengths
  int* const blk_pre = base_len + p.B;            // [B + 1] blocks before stream b
  int* const tok_pre = blk_pre + p.B + 1;         // [B + 1] new tokens before stream b (extend)
  __shared__ long long warp_sum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int nthreads = static_cast<int>(gridDim.x) * kBlockThreads;
  const int fc = *p.free_count;

  // Each thread sums a run of consecutive streams; then a scan over threads.
  const int per = (p.B + kBlockThreads - 1) / kBlockThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const long long room = static_cast<long long>(p.max_blocks) * p.page;
  long long blocks = 0, tokens = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int len = p.seq_lens[b], x = p.target[b];
    const bool wrong = len < 0 || x < 0 || (kExtend ? len + static_cast<long long>(x) > room : x > len || len > room);
    bad |= wrong;
    if (wrong) continue;
    blocks += kExtend ? ceil_div(len + x, p.page) - ceil_div(len, p.page)
                      : ceil_div(len, p.page) - ceil_div(x, p.page);
    if (kExtend) tokens += x;
  }
  long long ib = blocks, it = tokens;             // inclusive sums over the warp's threads
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ob = __shfl_up_sync(0xFFFFFFFFu, ib, d), ot = __shfl_up_sync(0xFFFFFFFFu, it, d);
    if (lane >= d) { ib += ob; it += ot; }
  }
  if (lane == 31) { warp_sum[0][warp] = ib; warp_sum[1][warp] = it; }
  bad = __syncthreads_or(bad) != 0;
  long long before_b = 0, before_t = 0, all_b = 0, all_t = 0;
  for (int w = 0; w < 32; ++w) {
    if (w == warp) { before_b = all_b; before_t = all_t; }
    all_b += warp_sum[0][w];
    all_t += warp_sum[1][w];
  }

  // Anything wrong: the batch stays as it was (the same verdict in every block).
  const bool no_pages = fc < 0 || fc > p.free_capacity || (kExtend ? all_b > fc : all_b > p.free_capacity - fc);
  bad |= kExtend && all_t > p.max_tokens;
  if (bad || no_pages) {
    if (kExtend)
      for (int t = rank * kBlockThreads + tid; t < p.max_tokens; t += nthreads) p.slots[t] = -1;
    if (rank == 0 && tid == 0) atomicOr(p.status, bad ? kBitSeqLen : kBitPool);
    return;
  }
  const int n_blocks = static_cast<int>(all_b), n_tokens = static_cast<int>(all_t);

  int eb = static_cast<int>(before_b + ib - blocks), et = static_cast<int>(before_t + it - tokens);
  for (int b = b0; b < b1; ++b) {
    const int len = p.seq_lens[b], x = p.target[b];
    base_len[b] = kExtend ? len : x;
    blk_pre[b] = eb;
    eb += kExtend ? ceil_div(len + x, p.page) - ceil_div(len, p.page) : ceil_div(len, p.page) - ceil_div(x, p.page);
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

  for (int k = rank * kBlockThreads + tid; k < n_blocks; k += nthreads) {
    const int b = find_stream(blk_pre, p.B, k);
    int32_t* const entry = p.table + static_cast<size_t>(b) * p.max_blocks + ceil_div(base_len[b], p.page) + (k - blk_pre[b]);
    if (kExtend) *entry = p.free_pages[fc - 1 - k];
    else p.free_pages[fc + n_blocks - 1 - k] = *entry;
  }
  if (kExtend) {
    // Four consecutive tokens a thread: one search, one 16-byte store.  The
    // page of a token's new block is read from the free list, not the table.
    bool off = false;
    for (long long t4 = 4ll * (rank * kBlockThreads + tid); t4 < p.max_tokens; t4 += 4ll * nthreads) {
      const int t0 = static_cast<int>(t4);
      int s[4] = {-1, -1, -1, -1};
      if (t0 < n_tokens) {
        int b = find_stream(tok_pre, p.B, t0);
        int held = -1, row0 = 0;                 // the block that `row0` belongs to, of stream b
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + e;
          if (t >= n_tokens) break;
          while (t >= tok_pre[b + 1]) { ++b; held = -1; }
          const int len = base_len[b], pos = len + (t - tok_pre[b]), blk = pos / p.page;
          if (blk != held) {
            const int have = ceil_div(len, p.page);
            const int page = blk < have ? p.table[static_cast<size_t>(b) * p.max_blocks + blk]
                                        : p.free_pages[fc - 1 - (blk_pre[b] + blk - have)];
            const bool ok = page >= 0 && page < p.pool_pages;
            off |= !ok;
            row0 = ok ? page * p.page : -1;
            held = blk;
          }
          s[e] = row0 < 0 ? -1 : row0 + (pos - blk * p.page);
        }
      }
      if (t0 + 4 <= p.max_tokens) {
        *reinterpret_cast<int4*>(p.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
      } else {
        for (int e = 0; t0 + e < p.max_tokens; ++e) p.slots[t0 + e] = s[e];
      }
    }
    if (off) atomicOr(p.status, kBitPage);
  }

  cluster_sync_all();   // every block has read the lengths and the free count
  if (rank == 0) {
    for (int b = tid; b < p.B; b += kBlockThreads)
      p.seq_lens[b] = kExtend ? base_len[b] + (tok_pre[b + 1] - tok_pre[b]) : base_len[b];
    if (tid == 0) *p.free_count = kExtend ? fc - n_blocks : fc + n_blocks;
  }
}

template <bool kExtend>
int launch_blocks(const BlocksParams& p, long long items, cudaStream_t stream) {
  const size_t smem = (3 * static_cast<size_t>(p.B) + 2) * sizeof(int);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(blocks_kernel<kExtend>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>((3 * kMaxStreams + 2) * sizeof(int))) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  const unsigned blocks = items > 4 * kBlockThreads ? kClusterBlocks : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kBlockThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, blocks_kernel<kExtend>, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

bool blocks_shape_ok(int B, int max_blocks, int page, int free_capacity) {
  return B >= 0 && B <= kMaxStreams && max_blocks >= 1 && page >= 1 && free_capacity >= 0 &&
         static_cast<long long>(max_blocks) * page < (1ll << 31);
}

// ------------------------------------------------------------ rows by slot
//
// Pure copies.  One warp a row, its 16-byte units over the lanes, four loads
// in flight a lane: the rows of one token are 1152 bytes (latent) to a few KB.
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
        if (c + 32 * e < n) v[e] = __ldg(src + c + 32 * e);
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
  int max_blocks, page, pool_pages, B, q;
};

// One block a stream and 512-byte column of the pool rows: eight warps read
// the path's rows (eight rows a warp at most) into registers, and after a
// barrier write them to their new places, so that any path is safe in place.
constexpr int kKeepWarps = 8;
constexpr int kKeepRows = 64 / kKeepWarps;

__global__ void __launch_bounds__(32 * kKeepWarps) keep_kernel(const KeepParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int rows[2][64];                      // pool rows the j-th kept draft moves from / to
  const int units = p.r.units[0] + p.r.units[1];
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  const int which = c < p.r.units[0] ? 0 : 1;
  uint8_t* const pool = p.r.pool[which] + 16ll * (which ? c - p.r.units[0] : c);
  const long long stride = p.r.pool_stride[which];
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int n = p.keep[b];
    if (n == 0) continue;
    const int len = p.seq_lens[b];
    uint32_t wrong = 0;
    if (n < 0 || n > p.q) wrong = kBitSlot;
    else if (len < p.q || len > static_cast<long long>(p.max_blocks) * p.page) wrong = kBitSeqLen;
    else if (threadIdx.x < 2 * n) {
      const int to = threadIdx.x & 1, j = threadIdx.x >> 1;
      int i = j;
      if (!to) {
        i = p.path[static_cast<size_t>(b) * p.q + j];
        if (i < 0 || i >= p.q) { wrong = kBitSlot; i = 0; }
      }
      const int pos = len - p.q + i, blk = pos / p.page;
      const int page = p.table[static_cast<size_t>(b) * p.max_blocks + blk];
      if (page < 0 || page >= p.pool_pages) wrong |= kBitPage;
      rows[to][j] = page * p.page + (pos - blk * p.page);
    }
    if (wrong) atomicOr(p.r.status, wrong);
    if (__syncthreads_or(static_cast<int>(wrong))) continue;   // this stream stays as it was
    uint4 v[kKeepRows];
#pragma unroll
    for (int e = 0; e < kKeepRows; ++e) {
      const int j = warp + kKeepWarps * e;
      if (j < n && c < units && rows[0][j] != rows[1][j])
        v[e] = *reinterpret_cast<const uint4*>(pool + rows[0][j] * stride);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kKeepRows; ++e) {
      const int j = warp + kKeepWarps * e;
      if (j < n && c < units && rows[0][j] != rows[1][j])
        *reinterpret_cast<uint4*>(pool + rows[1][j] * stride) = v[e];
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

int launched() {
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_LAUNCH;
  return MLA_OK;
}

}  // namespace mla

extern "C" {

int mla_blocks_extend(int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table, int B,
                      int max_blocks, int page_size, const int32_t* free_pages, int free_capacity,
                      int32_t* free_count, int pool_pages, int32_t* slots, int max_tokens,
                      cudaStream_t stream) {
  using namespace mla;
  if (!blocks_shape_ok(B, max_blocks, page_size, free_capacity) || max_tokens < 0 || pool_pages < 1 ||
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
                    d.status_word, B, max_blocks, page_size, free_capacity, pool_pages, max_tokens};
  return launch_blocks<true>(p, max_tokens, stream);
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
                    d.status_word, B, max_blocks, page_size, free_capacity, 0, 0};
  // At most this many pages come back.
  const long long table = static_cast<long long>(B) * max_blocks;
  return launch_blocks<false>(p, table < free_capacity ? table : free_capacity, stream);
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
  append_kernel<<<static_cast<unsigned>((static_cast<long long>(T) + kAppendWarps - 1) / kAppendWarps),
                  32 * kAppendWarps, 0, stream>>>(p);
  return launched();
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
  p.page = page_size;
  p.pool_pages = static_cast<int>(pool_rows / page_size);
  p.B = B;
  p.q = q_len;
  const unsigned cols = (static_cast<unsigned>(p.r.units[0]) + p.r.units[1] + 31) / 32;
  keep_kernel<<<dim3(cols, B < 65535 ? B : 65535), 32 * kKeepWarps, 0, stream>>>(p);
  return launched();
}

}  // extern "C"
