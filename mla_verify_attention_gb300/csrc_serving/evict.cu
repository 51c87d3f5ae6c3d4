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
// memory.  Three passes of a histogram (11, 11 and 10 bits, each over what shares
// the leading bits found so far), added up over the cluster by every block for
// itself, give the n-th largest total and how many equal to it stay; a scan over the
// keys then gives each kept one its place.  Weights are read once, and nothing but the
// histograms and counts passes between blocks.
constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxDevices = 64;
constexpr int kMostKeys = 49152;           // a block holds in shared memory

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
  uint32_t hist[3][kBins];
  unsigned long long warp_sum[32];
  unsigned long long counts;               // this block's: above the threshold (upper half), equal to it
  uint32_t digit, left;
};

__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);             // (-0 counts as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <class T>
__device__ __forceinline__ T remote(const T* mine, uint32_t rank) {
  const uint32_t at = mapa_shared(smem_u32(mine), rank);
  if constexpr (sizeof(T) == 8) {
    unsigned long long r;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(r) : "r"(at) : "memory");
    return static_cast<T>(r);
  } else {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return static_cast<T>(r);
  }
}

// Sum of x over the threads before this one (and, in `total`, over all).
__device__ __forceinline__ unsigned long long scan_before(unsigned long long x, unsigned long long* warp_sum,
                                                          unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();                                         // (the sums of the last scan have been read)
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long w = warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const unsigned long long before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0ull) + inc - x;
}

// kBlocks: of a stream's cluster.
template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t shared_keys[];
  __shared__ SelectShared sm;
  const int tid = threadIdx.x;
  const uint32_t rank = kBlocks > 1 ? cluster_ctarank() : 0u;
  const int b = static_cast<int>(blockIdx.x / kBlocks);
  for (int i = tid; i < 3 * kBins; i += kThreads) sm.hist[0][i] = 0;
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
  const int all = kBlocks * kThreads, me = static_cast<int>(rank) * kThreads + tid;
  for (int j = n + me; j < p.budget; j += all) kept[j] = -1;
  if (S <= p.budget) {                                     // (the whole cluster)
    for (int j = me; j < n; j += all) kept[j] = j;
    return;
  }
  const int run = (S + kBlocks - 1) / kBlocks, t0 = min(S, static_cast<int>(rank) * run), t1 = min(S, t0 + run);
  uint32_t* const keys = p.spill ? p.spill + static_cast<size_t>(b) * p.Smax + t0 : shared_keys;
  const int from = p.sinks, to = S - p.recent;             // the keys that are chosen from
  const float* const w = p.weights + static_cast<size_t>(b) * p.Hkv * p.Smax;
  __syncthreads();
  for (int t = t0 + tid; t < t1; t += kThreads) {
    if (t < from || t >= to) continue;
    float sum = w[t];
#pragma unroll 8
    for (int h = 1; h < p.Hkv; ++h) sum += w[static_cast<size_t>(h) * p.Smax + t];
    const uint32_t key = ordered(sum);
    keys[t - t0] = key;
    atomicAdd(&sm.hist[0][key >> 21], 1u);
  }
  const int choose = n - p.sinks - p.recent;               // how many of them
  uint32_t prefix = 0, left = static_cast<uint32_t>(choose);
  if (choose > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      if (pass > 0) {
        const int above = pass == 1 ? 21 : 10;
        for (int t = max(t0, from) + tid; t < min(t1, to); t += kThreads) {
          const uint32_t key = keys[t - t0];
          if (key >> above == prefix >> above) atomicAdd(&sm.hist[pass][(key >> shift) & (bins - 1)], 1u);
        }
      }
      if (kBlocks > 1) cluster_sync_all(); else __syncthreads();
      // Each thread two bins, the highest first.
      const int high = bins - 1 - 2 * tid;
      uint32_t c0 = 0, c1 = 0;
      if (high > 0) {
#pragma unroll
        for (int r = 0; r < kBlocks; ++r) {
          c0 += kBlocks > 1 ? remote(&sm.hist[pass][high], r) : sm.hist[pass][high];
          c1 += kBlocks > 1 ? remote(&sm.hist[pass][high - 1], r) : sm.hist[pass][high - 1];
        }
      }
      unsigned long long total;
      const uint32_t before = static_cast<uint32_t>(scan_before(c0 + c1, sm.warp_sum, total));
      if (high > 0 && before < left && left <= before + c0 + c1) {
        const bool second = left > before + c0;
        sm.digit = static_cast<uint32_t>(second ? high - 1 : high);
        sm.left = left - before - (second ? c0 : 0);
      }
      __syncthreads();
      prefix |= sm.digit << shift;
      left = sm.left;
    }
  }
  // Keys above the threshold stay, and the first `left` that equal it (choose = 0: none).
  const uint64_t threshold = choose > 0 ? prefix : 1ull << 32;
  const int per = (t1 - t0 + kThreads - 1) / kThreads;
  const int i0 = min(t1, t0 + tid * per), i1 = min(t1, i0 + per);
  unsigned long long mine = 0;
  for (int t = max(i0, from); t < min(i1, to); ++t) {
    const uint64_t key = keys[t - t0];
    mine += key > threshold ? 1ull << 32 : key == threshold ? 1ull : 0ull;
  }
  unsigned long long total;
  unsigned long long before = scan_before(mine, sm.warp_sum, total);
  if (kBlocks > 1) {
    if (tid == 0) sm.counts = total;
    cluster_sync_all();
    for (uint32_t r = 0; r < rank; ++r) before += remote(&sm.counts, r);
  }
  uint32_t above = static_cast<uint32_t>(before >> 32), equal = static_cast<uint32_t>(before);
  for (int t = i0; t < i1; ++t) {
    if (t < from) {
      kept[t] = t;
    } else if (t >= to) {
      kept[n - (S - t)] = t;
    } else {
      const uint64_t key = keys[t - t0];
      const int at = from + static_cast<int>(above + min(equal, left));
      const bool stays = key > threshold || (key == threshold && equal < left);
      if (stays) kept[at] = t;
      above += key > threshold;
      equal += key == threshold;
    }
  }
  if (kBlocks > 1) cluster_sync_all();                    // (others have read this block's counts)
}

// ------------------------------------------------------------ compact
//
// Row j takes row kept[j] >= j, in place.  A block takes a slice of the rows
// (`slice` units of 16 bytes) of a stream from its first row to its last: it loads
// the sources of some hundred rows, and after a barrier writes them.  Later rows
// have later sources (behind every row written so far), so that nothing is
// overwritten that is still to be read, whatever is ahead of whom within the block,
// and slices have nothing to do with each other.  The weights of a key head are
// one more slice, of 4 bytes a key.
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

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;

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
  auto look_up = [&](int j0, int buf) {
    for (int r = tid; r < chunk; r += kMoveThreads) {
      const int j = j0 + r;
      int2 at = make_int2(-1, -1);
      if (j < n) {
        const int t = kept[j];
        if (t < j || t >= S) atomicOr(p.status, kBitSlot);
        else if (t > j) {
          at = make_int2(pool_row(p, b, t), pool_row(p, b, j));
          if (at.y < 0) at.x = -1;
        }
      }
      rows[buf][r] = at;
    }
  };
  look_up(0, 0);
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
    if (j0 + chunk < n) look_up(j0 + chunk, buf ^ 1);
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

// Blocks a stream's cluster has: one where a block gets through its keys soon enough.
constexpr int kBlocks = 8;
int select_blocks(int Smax) { return Smax <= 4096 ? 1 : kBlocks; }
int select_run(int Smax) { return (Smax + select_blocks(Smax) - 1) / select_blocks(Smax); }

bool select_shape_ok(long long B, long long Smax) {
  return B >= 0 && B < (1 << 20) && Smax >= 1 && Smax < (1 << 24);
}

std::mutex g_mutex;
bool g_ready[kMaxDevices];

int select_ready() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_ready[dev]) {
    if (cudaFuncSetAttribute(select_kernel<kBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostKeys) !=
        cudaSuccess) {
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
  if (!select_shape_ok(B, Smax) || select_run(Smax) <= kMostKeys) return 0;
  return 4 * static_cast<size_t>(B) * Smax;
}

int mla_evict_select(const float* weights, const int32_t* seq_lens, int B, int Hkv, int Smax, int sinks, int recent,
                     int32_t* kept, int budget, int32_t* keep_lens, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  using namespace mla;
  using namespace mla::evict;
  if (!select_shape_ok(B, Smax) || Hkv < 1 || Hkv > (1 << 16) || budget < 1 || sinks < 0 || recent < 0 ||
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
  st = select_ready();
  if (st != MLA_OK) return st;
  const int blocks = select_blocks(Smax);
  const SelectParams p = {weights, seq_lens, kept, keep_lens, need > 0 ? static_cast<uint32_t*>(workspace) : nullptr,
                          d.status_word, Hkv, Smax, budget, sinks, recent};
  return launch_dependent(blocks > 1 ? select_kernel<kBlocks> : select_kernel<1>, p, dim3(static_cast<unsigned>(B) * blocks), kThreads,
                          need > 0 ? 0 : 4 * static_cast<size_t>(select_run(Smax)), stream, blocks);
}

int mla_cache_compact(void* pool_a, long long pool_a_stride, int a_bytes, void* pool_b, long long pool_b_stride,
                      int b_bytes, long long pool_rows, float* weights, int Hkv, const int32_t* block_table,
                      int max_blocks, int page_size, const int32_t* seq_lens, const int32_t* kept, int budget,
                      const int32_t* keep_lens, int B, cudaStream_t stream) {
  using namespace mla;
  using namespace mla::evict;
  if (B < 0 || B >= (1 << 20) || budget < 1 || max_blocks < 1 || page_size < 1 ||
      static_cast<long long>(max_blocks) * page_size >= (1ll << 31) || a_bytes < 16 || b_bytes < 0 || pool_rows < page_size ||
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
  // Slices of 64 bytes, or of less where those would leave the device half empty.
  const long long units = static_cast<long long>(p.units[0]) + p.units[1];
  p.slice_shift = 2;
  while (p.slice_shift > 0 && ((units + (1 << p.slice_shift) - 1) >> p.slice_shift) * B < 2 * d.sms) --p.slice_shift;
  p.slices = static_cast<int>((units + (1 << p.slice_shift) - 1) >> p.slice_shift);
  return launch_dependent(compact_kernel, p, dim3(p.slices + p.Hkv, B < 65535 ? B : 65535), kMoveThreads, 0, stream);
}

}  // extern "C"
