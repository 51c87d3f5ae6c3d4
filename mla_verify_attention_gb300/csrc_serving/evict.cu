// Eviction from a cache: which keys stay (mla_evict_select) and their rows
// together (mla_cache_compact).  Declared, with their exact meaning, in
// include/mla_verify_attn.h.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "internal.h"
#include "launch.h"
#include "mla_verify_attn.h"
#include "ptx.cuh"

namespace mla {
namespace evict {

// ------------------------------------------------------------ select
//
// Of a stream's keys between the first `sinks` and the last `recent`, those with the
// n largest totals (of the key heads' weights) stay, of equal ones the first.  A
// cluster of blocks takes a stream, each a run of its keys: they sum the heads, in order,
// into an unsigned number that orders as the total does, and keep it in shared
// memory.  Four passes of a histogram of eight bits, each over what shares the leading
// bits found so far, give the n-th largest total and how many equal to it stay; a scan
// over the keys then gives each kept one its place.  Weights are read once.
//
// What bounds it beside that read: chains of barriers and reads.  Blocks send their
// histograms and counts to all others' shared memory and meet once a pass: read from
// there after the barrier instead, 2,048 bins took 8,000 cycles a pass, more than
// two passes of 256 take in all (one stream of 64k keys, 8 heads 30.6 -> 15.8 us).
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kPasses = 4;
constexpr int kMostBlocks = 8;
constexpr int kMaxDevices = 64;
constexpr int kMostKeys = 49152;           // a block holds in shared memory
// Rows and budgets at most: positions are counted on past them in 32 bits.
constexpr long long kMostBudget = 1ll << 30;

struct SelectParams {
  const float* weights;                    // [B][Hkv][Smax]
  const int32_t* seq_lens;
  int32_t* kept;                           // [B][budget]
  int32_t* keep;
  uint32_t* spill;                         // [B][Smax], where a block's run does not fit
  unsigned int* status;
  int Hkv, Smax, budget, sinks, recent;
};

struct SelectShared {
  uint32_t mine[kPasses][kBins];                           // this block's histograms
  uint32_t all[2][kMostBlocks][kBins];     // and everyone's, of every second pass (there is a barrier between)
  uint64_t counts[kMostBlocks];            // keys above the threshold (upper half), equal to it
  uint64_t warp_counts[kWarps];
  uint32_t warp_sum[kBins / 32];
  uint32_t digit, left;
};

__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);             // (-0 counts as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <class T>
__device__ __forceinline__ void send(T* mine, uint32_t rank, T x) {
  const uint32_t at = mapa_shared(smem_u32(mine), rank);
  if constexpr (sizeof(T) == 8) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
  else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// All threads of a cluster; what they have sent has arrived.
template <int kBlocks>
__device__ __forceinline__ void sync_blocks() {
  if (kBlocks > 1) cluster_sync_all();
  else __syncthreads();
}

// All blocks of the cluster have started (the other half of the kernel's first arrival).
template <int kBlocks>
__device__ __forceinline__ void await_blocks() {
  __syncwarp();
  if (kBlocks > 1) cluster_wait();
}

// kBlocks: of a stream's cluster.
template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t shared_keys[];
  __shared__ SelectShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = kBlocks > 1 ? cluster_ctarank() : 0u;
  const int b = static_cast<int>(blockIdx.x / kBlocks);
  // Another block's shared memory may be written once that block has started: all arrive
  // here, and wait (await_blocks) before the first of them sends or returns.
  if (kBlocks > 1) cluster_arrive_relaxed();
  for (int i = tid; i < kPasses * kBins; i += kThreads) sm.mine[0][i] = 0;
  grid_dependency_wait();
  if (tid == 0) grid_launch_dependents();
  int S = p.seq_lens[b];
  if (S < 0 || S > p.Smax) {
    if (tid == 0 && rank == 0) atomicOr(p.status, kBitSeqLen);
    S = 0;
  }
  const int n = min(S, p.budget);
  int32_t* const kept = p.kept + static_cast<size_t>(b) * p.budget;
  if (tid == 0 && rank == 0) p.keep[b] = n;
  const int threads = kBlocks * kThreads, me = static_cast<int>(rank) * kThreads + tid;
  for (int j = n + me; j < p.budget; j += threads) kept[j] = -1;
  if (S <= p.budget) {                                     // (the whole cluster)
    await_blocks<kBlocks>();
    for (int j = me; j < n; j += threads) kept[j] = j;
    return;
  }
  const int run = (S + kBlocks - 1) / kBlocks, t0 = min(S, static_cast<int>(rank) * run), t1 = min(S, t0 + run);
  uint32_t* const keys = p.spill ? p.spill + static_cast<size_t>(b) * p.Smax + t0 : shared_keys;
  const int from = max(t0, p.sinks), to = min(t1, S - p.recent);   // of this block's keys, those that are chosen from
  __syncthreads();
  constexpr int kAtOnce = 8;                               // keys a thread
  for (int t = from + tid; t < to; t += kAtOnce * kThreads) {
    const float* w = p.weights + static_cast<size_t>(b) * p.Hkv * p.Smax + t;
    float sum[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) sum[e] = t + e * kThreads < to ? w[e * kThreads] : 0.f;
#pragma unroll 4
    for (int h = 1; h < p.Hkv; ++h) {
      w += p.Smax;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        if (t + e * kThreads < to) sum[e] += w[e * kThreads];
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      if (t + e * kThreads >= to) continue;
      const uint32_t key = ordered(sum[e]);
      keys[t + e * kThreads - t0] = key;
      atomicAdd(&sm.mine[0][key >> 24], 1u);
    }
  }
  await_blocks<kBlocks>();
  const int choose = n - p.sinks - p.recent;               // how many of them
  uint32_t prefix = 0, left = static_cast<uint32_t>(choose);
  if (choose > 0) {
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = 24 - 8 * pass;
      if (pass > 0) {
        for (int t = from + tid; t < to; t += kThreads) {
          const uint32_t key = keys[t - t0];
          if (key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&sm.mine[pass][key >> shift & 0xFFu], 1u);
        }
      }
      const uint32_t* sums = sm.mine[pass];
      __syncthreads();
      if (kBlocks > 1) {
#pragma unroll
        for (int i = tid; i < kBlocks * kBins; i += kThreads)
          send(&sm.all[pass & 1][rank][i % kBins], static_cast<uint32_t>(i / kBins), sums[i % kBins]);
        sync_blocks<kBlocks>();
      }
      // A thread a bin, the highest first.
      uint32_t c = 0, inc = 0;
      if (tid < kBins) {
        const int bin = kBins - 1 - tid;
        if (kBlocks > 1) {
#pragma unroll
          for (int r = 0; r < kBlocks; ++r) c += sm.all[pass & 1][r][bin];
        } else {
          c = sums[bin];
        }
        inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
          if (lane >= d) inc += o;
        }
        if (lane == 31) sm.warp_sum[warp] = inc;
      }
      __syncthreads();
      if (tid < kBins) {
        for (int w = 0; w < warp; ++w) inc += sm.warp_sum[w];
        if (inc - c < left && left <= inc) {
          sm.digit = static_cast<uint32_t>(kBins - 1 - tid);
          sm.left = left - (inc - c);
        }
      }
      __syncthreads();
      prefix |= sm.digit << shift;
      left = sm.left;
    }
  }
  // Keys above the threshold stay, and the first `left` that equal it (choose = 0:
  // none).  Each warp counts a run of them, then they are put in their places.
  const uint64_t threshold = choose > 0 ? prefix : 1ull << 32;
  const int each = ((to - from + kThreads - 1) / kThreads) * 32;     // keys a warp (none: from > to)
  const int w0 = from + warp * each, w1 = min(to, w0 + each);
  uint32_t above = 0, equal = 0;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint64_t key = t < w1 ? keys[t - t0] : 0;
    above += __popc(__ballot_sync(0xFFFFFFFFu, t < w1 && key > threshold));
    equal += __popc(__ballot_sync(0xFFFFFFFFu, t < w1 && key == threshold));
  }
  if (lane == 0) sm.warp_counts[warp] = static_cast<uint64_t>(above) << 32 | equal;
  __syncthreads();
  uint64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total += sm.warp_counts[w];
  }
  if (kBlocks > 1) {
    if (tid < kBlocks) send(&sm.counts[rank], static_cast<uint32_t>(tid), total);
    sync_blocks<kBlocks>();
    for (uint32_t r = 0; r < rank; ++r) before += sm.counts[r];
  }
  above = static_cast<uint32_t>(before >> 32);
  equal = static_cast<uint32_t>(before);
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint64_t key = t < w1 ? keys[t - t0] : 0;
    const unsigned more = __ballot_sync(0xFFFFFFFFu, t < w1 && key > threshold);
    const unsigned same = __ballot_sync(0xFFFFFFFFu, t < w1 && key == threshold);
    const unsigned lower = (1u << lane) - 1u;
    const uint32_t e = equal + __popc(same & lower);
    if ((more >> lane & 1u) || ((same >> lane & 1u) && e < left))
      kept[p.sinks + static_cast<int>(above + __popc(more & lower) + min(e, left))] = t;
    above += __popc(more);
    equal += __popc(same);
  }
  // The first and the last keys, shared out among all.
  for (int t = me; t < p.sinks; t += threads) kept[t] = t;
  for (int t = me; t < p.recent; t += threads) kept[n - p.recent + t] = S - p.recent + t;
}

// ------------------------------------------------------------ compact
//
// Row j takes row kept[j] >= j, in place.  A block takes a slice of the rows
// (`slice` units of 16 bytes) of a stream from its first row to its last: it loads
// the sources of some hundred rows, and after a barrier writes them.  Later rows
// have later sources (behind every row written so far), so that nothing is
// overwritten that is still to be read, whatever is ahead of whom within the block,
// and slices have nothing to do with each other.  The weights of a key head are
// one more slice, of 4 bytes a key.  Bound by HBM: 8 streams of 16k to 32k keys to 8k,
// 4 KB a row 100 us, 5.4 TB/s (80 % of the measured copy rate) in slices of 128 bytes
// (of 32, 64, 256: 147, 124, 163 us with 256 threads).
struct CompactParams {
  uint8_t* pool[2];
  long long pool_stride[2];
  int units[2];
  float* weights;                          // [B][Hkv][Smax] or null
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* kept;
  const int32_t* keep;
  unsigned int* status;
  int max_blocks, pool_pages, Smax, budget, Hkv, B;
  int slice_shift, slices;                 // units a slice: 1 << slice_shift
  Divisor page;
};

constexpr int kMoveThreads = 512;
constexpr int kMoveLoads = 4;

// Pool row of a stream's row; -1 (and the page reported) where there is none.
__device__ __forceinline__ int pool_row(const CompactParams& p, int b, int t) {
  const int blk = p.page.of(t), page = p.table[static_cast<size_t>(b) * p.max_blocks + blk];
  if (page < 0 || page >= p.pool_pages) {
    atomicOr(p.status, kBitPage);
    return -1;
  }
  return page * static_cast<int>(p.page.d) + (t - blk * static_cast<int>(p.page.d));
}

__device__ __forceinline__ void move_rows(const CompactParams& p, int b, int S, int n, const int32_t* kept,
                                          int2 (*rows)[kMoveThreads * kMoveLoads]) {
  const int tid = threadIdx.x, lanes = 1 << p.slice_shift;
  const int step = kMoveThreads >> p.slice_shift;          // rows a load of the block
  const int chunk = step * kMoveLoads;
  const int unit = (static_cast<int>(blockIdx.x) << p.slice_shift) + (tid & (lanes - 1)), r0 = tid >> p.slice_shift;
  const bool second = unit >= p.units[0], mine = unit < p.units[0] + p.units[1];
  uint8_t* const pool = second ? p.pool[1] + 16ll * (unit - p.units[0]) : p.pool[0] + 16ll * unit;
  const long long stride = second ? p.pool_stride[1] : p.pool_stride[0];
  // A chunk's rows are looked up while the one before it is moved, what is kept another
  // chunk earlier: one read that waits for nothing but itself a chunk.
  int next[kMoveLoads];
  auto look_ahead = [&](int j0) {
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int r = tid + e * kMoveThreads, j = j0 + r;
      next[e] = r < chunk && j < n ? kept[j] : 0;
    }
  };
  auto look_up = [&](int j0, int buf) {
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int r = tid + e * kMoveThreads, j = j0 + r;
      if (r >= chunk) break;
      int2 at = make_int2(-1, -1);
      if (j < n) {
        const int t = next[e];
        if (t < j || t >= S) atomicOr(p.status, kBitSlot);
        else if (t > j) {
          at = make_int2(pool_row(p, b, t), pool_row(p, b, j));
          if (at.y < 0) at.x = -1;
        }
      }
      rows[buf][r] = at;
    }
  };
  look_ahead(0);
  look_up(0, 0);
  look_ahead(chunk);
  __syncthreads();
  int buf = 0;
  for (int j0 = 0; j0 < n; j0 += chunk, buf ^= 1) {
    uint4 v[kMoveLoads];
    int to[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int2 at = rows[buf][e * step + r0];
      to[e] = mine && at.x >= 0 ? at.y : -1;
      if (to[e] >= 0) v[e] = *reinterpret_cast<const uint4*>(pool + at.x * stride);
    }
    if (j0 + chunk < n) {
      look_up(j0 + chunk, buf ^ 1);
      look_ahead(j0 + 2 * chunk);
    }
    __syncthreads();                                       // all of this chunk's sources are read
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (to[e] >= 0) *reinterpret_cast<uint4*>(pool + to[e] * stride) = v[e];
  }
}

__device__ __forceinline__ void move_weights(const CompactParams& p, int b, int S, int n, const int32_t* kept, int head) {
  constexpr int chunk = kMoveThreads * kMoveLoads;
  float* const w = p.weights + (static_cast<size_t>(b) * p.Hkv + head) * p.Smax;
  for (int j0 = 0; j0 < n; j0 += chunk) {
    float v[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int j = j0 + e * kMoveThreads + static_cast<int>(threadIdx.x);
      if (j >= n) continue;
      const int t = kept[j];
      v[e] = w[t < j || t >= S ? j : t];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int j = j0 + e * kMoveThreads + static_cast<int>(threadIdx.x);
      if (j < n) w[j] = v[e];
    }
  }
  __syncthreads();                                         // (the last sources may lie behind row n)
  for (int t = n + static_cast<int>(threadIdx.x); t < S; t += kMoveThreads) w[t] = 0.f;
}

__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  __shared__ int2 rows[2][kMoveThreads * kMoveLoads];
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int S = p.seq_lens[b], n = p.keep[b];
    uint32_t wrong = 0;
    if (S < 0 || S > p.Smax) wrong = kBitSeqLen;
    else if (n < 0 || n > min(S, p.budget)) wrong = kBitSlot;
    if (wrong) {
      if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.status, wrong);
      continue;
    }
    const int32_t* const kept = p.kept + static_cast<size_t>(b) * p.budget;
    const int head = static_cast<int>(blockIdx.x) - p.slices;
    if (head >= 0) move_weights(p, b, S, n, kept, head);
    else move_rows(p, b, S, n, kept, rows);
    __syncthreads();
  }
}

// ------------------------------------------------------------ host

// Blocks of a stream's cluster: as many as the device takes at once, none of which a
// short stream needs: up to 4,096 keys one block is through sooner.  (Two an SM: that is
// so while a block has room for no more than some 22k keys; longer runs fill an SM each,
// and the last clusters wait for the first.)
int select_blocks(int B, int Smax, int sms) {
  if (Smax <= 4096) return 1;
  int blocks = kMostBlocks;
  while (blocks > 1 && static_cast<long long>(B) * blocks > 2 * sms && (Smax + blocks / 2 - 1) / (blocks / 2) <= kMostKeys)
    blocks /= 2;
  return blocks;
}
bool select_spills(int Smax) { return (Smax + kMostBlocks - 1) / kMostBlocks > kMostKeys; }

bool select_shape_ok(long long B, long long Smax) {
  return B >= 0 && B < (1 << 20) && Smax >= 1 && Smax < (1 << 24);
}

using SelectFn = void (*)(SelectParams);
constexpr int kForms = 4;                  // 1, 2, 4 and 8 blocks
std::mutex g_mutex;
bool g_ready[kMaxDevices];

int pick_select(int blocks, SelectFn* fn) {
  static const SelectFn all[kForms] = {select_kernel<1>, select_kernel<2>, select_kernel<4>, select_kernel<8>};
  *fn = all[blocks == 8 ? 3 : blocks == 4 ? 2 : blocks == 2 ? 1 : 0];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_ready[dev]) {
    for (SelectFn f : all)
      if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostKeys) != cudaSuccess) {
        cudaGetLastError();
        return MLA_ERR_LAUNCH;
      }
    g_ready[dev] = true;
  }
  return MLA_OK;
}

}  // namespace evict
}  // namespace mla

extern "C" {

size_t mla_evict_workspace_size(int B, int Smax) {
  using namespace mla::evict;
  if (!select_shape_ok(B, Smax) || !select_spills(Smax)) return 0;
  return 4 * static_cast<size_t>(B) * Smax;
}

int mla_evict_select(const float* weights, const int32_t* seq_lens, int B, int Hkv, int Smax, int sinks, int recent,
                     int32_t* kept, int budget, int32_t* keep_lens, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  using namespace mla;
  using namespace mla::evict;
  if (!select_shape_ok(B, Smax) || Hkv < 1 || Hkv > (1 << 16) || budget < 1 || budget > kMostBudget || sinks < 0 || recent < 0 ||
      static_cast<long long>(sinks) + recent > budget)
    return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!weights || !seq_lens || !kept || !keep_lens) return MLA_ERR_NULLPTR;
  if (!aligned_to(weights, 4) || !aligned_to(seq_lens, 4) || !aligned_to(kept, 4) || !aligned_to(keep_lens, 4) ||
      !aligned_to(workspace, 4))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  int st = device_common(&d);
  if (st != MLA_OK) return st;
  const size_t need = mla_evict_workspace_size(B, Smax);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MLA_ERR_WORKSPACE;
  const int blocks = select_blocks(B, Smax, d.sms);
  SelectFn fn;
  st = pick_select(blocks, &fn);
  if (st != MLA_OK) return st;
  const SelectParams p = {weights, seq_lens, kept, keep_lens, need > 0 ? static_cast<uint32_t*>(workspace) : nullptr,
                          d.status_word, Hkv, Smax, budget, sinks, recent};
  return launch_dependent(fn, p, dim3(static_cast<unsigned>(B) * blocks), kThreads,
                          need > 0 ? 0 : 4 * static_cast<size_t>((Smax + blocks - 1) / blocks), stream, blocks);
}

int mla_cache_compact(void* pool_a, long long pool_a_stride, int a_bytes, void* pool_b, long long pool_b_stride,
                      int b_bytes, long long pool_rows, float* weights, int Hkv, const int32_t* block_table,
                      int max_blocks, int page_size, const int32_t* seq_lens, const int32_t* kept, int budget,
                      const int32_t* keep_lens, int B, cudaStream_t stream) {
  using namespace mla;
  using namespace mla::evict;
  if (B < 0 || B >= (1 << 20) || budget < 1 || budget > kMostBudget || max_blocks < 1 || page_size < 1 ||
      static_cast<long long>(max_blocks) * page_size > kMostBudget || a_bytes < 16 || b_bytes < 0 || pool_rows < page_size ||
      pool_rows >= (1ll << 31) || (weights && (Hkv < 1 || Hkv > (1 << 16))))
    return MLA_ERR_SHAPE;
  const long long limit = 1ll << 32;
  if (pool_a_stride < a_bytes || pool_a_stride > limit || (b_bytes > 0 && (pool_b_stride < b_bytes || pool_b_stride > limit)))
    return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!pool_a || (b_bytes > 0 && !pool_b) || !block_table || !seq_lens || !kept || !keep_lens) return MLA_ERR_NULLPTR;
  if (!aligned_to(pool_a, 16) || pool_a_stride % 16 || a_bytes % 16 || b_bytes % 16 ||
      (b_bytes > 0 && (!aligned_to(pool_b, 16) || pool_b_stride % 16)) || !aligned_to(weights, 4) ||
      !aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(kept, 4) || !aligned_to(keep_lens, 4))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  const int st = device_common(&d);
  if (st != MLA_OK) return st;
  CompactParams p = {};
  p.pool[0] = static_cast<uint8_t*>(pool_a);
  p.pool[1] = static_cast<uint8_t*>(b_bytes > 0 ? pool_b : pool_a);
  p.pool_stride[0] = pool_a_stride;
  p.pool_stride[1] = b_bytes > 0 ? pool_b_stride : 0;
  p.units[0] = a_bytes / 16;
  p.units[1] = b_bytes / 16;
  p.weights = weights;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.kept = kept;
  p.keep = keep_lens;
  p.status = d.status_word;
  p.max_blocks = max_blocks;
  p.pool_pages = static_cast<int>(pool_rows / page_size);
  p.Smax = max_blocks * page_size;
  p.budget = budget;
  p.Hkv = weights ? Hkv : 0;
  p.B = B;
  p.page = Divisor(page_size);
  // Slices of 128 bytes, or of less, to 32, where those would leave SMs empty.
  const long long units = static_cast<long long>(p.units[0]) + p.units[1];
  p.slice_shift = 3;
  while (p.slice_shift > 1 && ((units + (1 << p.slice_shift) - 1) >> p.slice_shift) * B < d.sms) --p.slice_shift;
  p.slices = static_cast<int>((units + (1 << p.slice_shift) - 1) >> p.slice_shift);
  return launch_dependent(compact_kernel, p, dim3(p.slices + p.Hkv, B < 65535 ? B : 65535), kMoveThreads, 0, stream);
}

}  // extern "C"
