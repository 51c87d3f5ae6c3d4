// The attention weight that each cached key got (mla_gqa_attn_weights and its
// paged form, declared in include/mla_verify_attn.h).
//
// Mathematics.  With the log-sum-exps that the attention call returned, a weight is
// exp(score - lse): weights[b][g][t] += the sum of that over the drafts and the
// query heads of key head g that see key t.  One product a tile, S = K Q^T with the
// keys as its 128 rows: a thread then has a key, adds up its columns in
// registers, and no sum crosses threads, tiles or blocks.
//
// What bounds it: K is read once (2 D bytes a key and head; the weights add 8), up to
// ~100 rows; beyond, a thread's exponentials: 16 a cycle and SM.  Measured (GPU time, D =
// 128, loads first): 64 streams of 1k to 32k keys, one token, 16-row pages, 8 heads a key
// head 207 us, 6.0 TB/s (88 % of the measured copy rate); one stream of 64k keys, 9 drafts
// 30 us, of 262k 93 us (87 %); 64 drafts (512 rows a key head) over 8k keys 24 us.
//
// Split.  As in the attention kernel: equal runs of 64-key tiles, teams of CTAs
// with the key heads of a cache row side by side.  A run's tiles are taken two at a
// time.  Query rows come in chunks of 128; one chunk stays in shared memory for the
// whole run of a stream and head, several are loaded again for every two tiles (a
// chunk's exponentials take longer than its 32 KB from L2).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "gqa_attn.cuh"
#include "gqa_host.h"
#include "mla_verify_attn.h"

namespace mla {
namespace gqa {
namespace weights {

constexpr int kTileKeys = 2 * kKeys;
constexpr int kChunkRows = 128;            // query rows a product (MMA N)

struct WeightParams : Params {
  const float* given_lse;                  // [B][q][H]
  float* weights;                          // [B][Hkv][Smax]
  int chunks, chunk_rows;                  // chunk_rows: of the only chunk, a multiple of 16, or 128
};

template <int D>
struct WShape {
  static constexpr int kChunks = D / 64;                   // 64-wide column chunks
  static constexpr int kTile = kTileKeys * D * 2;
  static constexpr int kQTile = kChunkRows * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;        // 160 KB of K
};

template <int D>
struct __align__(1024) WSmem {
  uint8_t ring[WShape<D>::kStages * WShape<D>::kTile];
  uint8_t q[2 * WShape<D>::kQTile];
  float minus_lse[2][kChunkRows];          // in log2 units; -inf: the row adds nothing
  uint32_t adds[2][kChunkRows / 32];       // rows that add something, a bit each
  uint64_t kfull[WShape<D>::kStages], kempty[WShape<D>::kStages];
  uint64_t qfull[2], qempty[2], sfull[2][2], sempty[2][2], drain;   // s: [group][buffer]
  int warp_sum[kThreads / 32], start_b, start_pre;
  uint32_t tmem_base, abort_flag;
};

#define MLA_TMEM_LD_32x32b_X16(taddr, r)                                                          \
  asm volatile(                                                                                   \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14," \
      "%15}, [%16];"                                                                              \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),       \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),   \
        "=r"(r[14]), "=r"(r[15])                                                                  \
      : "r"(taddr))

// Warp 0: K tiles by TMA, boxes of box_rows rows and 64 dims; the lanes look up the
// rows of 32 boxes together and a batch ahead.
template <int D>
__device__ __forceinline__ void load_k_tma(WSmem<D>& sm, const WeightParams& p, const CUtensorMap* map, Walk<kWhole> w) {
  using C = WShape<D>;
  const int lane = threadIdx.x & 31;
  const int R = p.box_rows, shift = __ffs(R) - 1, boxes = kKeys >> shift, batch_tiles = 32 / boxes;
  const bool paged = p.block_table != nullptr;
  const uint32_t ring = smem_u32(sm.ring);
  Ring<C::kStages> at;
  int issued = 0;
  Segment s;
  while (w.next(p, s)) {
    const int end = min(s.S, (s.tile0 + s.n) * kKeys);
    auto key_of = [&](int j) { return (s.tile0 + j) * kKeys + lane * R; };
    auto entry_of = [&](int j) { return paged && key_of(j) < end ? table_entry(p, s.b, key_of(j)) : 0; };
    const int batch = paged ? 0 : s.b;
    int row = 0, entry = entry_of(0), first = 0;
    for (int j = 0; j < s.n; ++j, first = (first + boxes) & 31) {
      if (first == 0) {
        row = !paged ? key_of(j) : (key_of(j) < end ? pool_row(p, entry, key_of(j)) : 0);
        entry = entry_of(j + batch_tiles);
      }
      const int key0 = (s.tile0 + j) * kKeys;
      const uint32_t bar = smem_u32(&sm.kfull[at.stage]), dst = ring + at.stage * C::kTile + (j & 1) * (kKeys * 128);
      if ((j & 1) == 0) {
        if (!wait(sm, sm.kempty[at.stage], at.phase ^ 1, p)) goto out;
        const int n = min(min(2, s.n - j) * boxes, (s.S - key0 + R - 1) >> shift);   // boxes of this tile and the next
        if (p.test_stall && issued == 0 && blockIdx.x == 0) goto out;                // this load never comes
        arrive_expect_elect(bar, n * R * D * 2);
        ++issued;
      }
      const int n = min(boxes, (s.S - key0 + R - 1) >> shift);
      for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, first + i);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_box_elect(dst + c * (kTileKeys * 128) + i * R * 128, map, r, c, s.head, batch, bar);
      }
      if ((j & 1) || j == s.n - 1) at.advance();
    }
  }
out:
  for (int n = issued - 1; n >= 0 && n >= issued - C::kStages; --n)
    mbar_wait(smem_u32(&sm.kfull[n % C::kStages]), (n / C::kStages) & 1, kWaitNs / 2);
}

// Warp 0 where no box fits the pages: rows copied 16 bytes a lane, a stage at a time.
template <int D>
__device__ __forceinline__ void load_k_gather(WSmem<D>& sm, const WeightParams& p, Walk<kWhole> w) {
  using C = WShape<D>;
  constexpr int kUnits = D / 8, kPer = 32 / kUnits;
  constexpr int kAhead = C::kStages - 1 < 4 ? C::kStages - 1 : 4;   // stages in flight
  const int lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(sm.ring);
  const bool withheld = p.test_stall && blockIdx.x == 0;
  Ring<C::kStages> at, landed;
  int started = 0;
  auto publish = [&]() {
    fence_proxy_async_smem();
    if (!withheld) mbar_arrive(smem_u32(&sm.kfull[landed.stage]));
    landed.advance();
  };
  Segment s;
  while (w.next(p, s)) {
    const uint8_t* const head = p.k + s.head * p.k_stride[2] + (lane % kUnits) * 16;
    auto entry_of = [&](int j, int e) {                    // of the step's 32-key quarter e
      const int key = (s.tile0 + j) * kKeys + e * 32 + lane;
      return j + (e >> 1) < s.n && key < s.S ? table_entry(p, s.b, key) : 0;
    };
    int next[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) next[e] = entry_of(0, e);
    for (int j = 0; j < s.n; j += 2, at.advance()) {
      int rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = (s.tile0 + j) * kKeys + e * 32 + lane;
        rows[e] = j + (e >> 1) < s.n && key < s.S ? pool_row(p, next[e], key) : -1;
        next[e] = entry_of(j + 2, e);
      }
      if (!wait(sm, sm.kempty[at.stage], at.phase ^ 1, p)) goto out;
      const uint32_t dst = ring + at.stage * C::kTile + (lane % kUnits >> 3) * (kTileKeys * 128);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          const int r = i * kPer + lane / kUnits, tile_row = e * 32 + r;
          const int row = __shfl_sync(0xFFFFFFFFu, rows[e], r);
          cp_async_16(dst + tile_row * 128 + (((lane & 7) ^ (tile_row & 7)) << 4), head + (row < 0 ? 0 : row) * p.k_stride[1],
                      row >= 0);
        }
      cp_async_commit();
      if (++started >= kAhead) {
        cp_async_wait<kAhead - 1>();
        publish();
      }
    }
  }
  cp_async_wait<0>();
  for (int n = min(started, kAhead - 1); n > 0; --n) publish();
  return;
out:
  cp_async_wait<0>();
}

// Warps 2 and 3: chunks of query rows, every second row pair each, and their lse.
template <int D>
__device__ __forceinline__ void load_q(WSmem<D>& sm, const WeightParams& p, Walk<kWhole> w, int half) {
  using C = WShape<D>;
  constexpr int kUnits = D / 8, kPer = 32 / kUnits;
  const int lane = threadIdx.x & 31, all_rows = p.q_len * p.G;
  int loads = 0;
  Segment s;
  while (w.next(p, s)) {
    const int times = p.chunks == 1 ? 1 : (s.n + 1) / 2 * p.chunks;
    for (int x = 0, c = 0; x < times; ++x, c = c + 1 == p.chunks ? 0 : c + 1, ++loads) {
      const int buf = loads & 1;
      if (!wait(sm, sm.qempty[buf], ((loads >> 1) & 1) ^ 1, p)) return;
      const int N = min(kChunkRows, p.chunk_rows);
      const uint32_t tile = smem_u32(sm.q) + buf * C::kQTile;
      float lse[2] = {CUDART_INF_F, CUDART_INF_F};
      for (int r0 = half * 32; r0 < N; r0 += 64) {
        // A row a lane: its address and its lse, which is looked at once the copies are under way.
        const int R = c * kChunkRows + r0 + lane, i = p.by_G.of(R);
        const int head = s.head * p.G + (R - i * p.G);
        long long off = -1;
        if (R < all_rows) {
          lse[r0 >= 64] = p.given_lse[(static_cast<long long>(s.b) * p.q_len + i) * p.H + head];
          off = s.b * p.q_stride[0] + i * p.q_stride[1] + head * p.q_stride[2];
        }
#pragma unroll
        for (int e = 0; e < 32 / kPer; ++e) {
          const int r = e * kPer + lane / kUnits, u = lane % kUnits, row = r0 + r;
          const long long o = __shfl_sync(0xFFFFFFFFu, off, r);
          cp_async_16(tile + (u >> 3) * (kChunkRows * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4),
                      p.q + (o < 0 ? 0 : o) + u * 16, o >= 0);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r0 = half * 32 + 64 * k;
        if (r0 >= N) break;
        const bool adds = !isinf(lse[k]);
        sm.minus_lse[buf][r0 + lane] = adds ? -lse[k] * 1.4426950408889634f : -CUDART_INF_F;
        const uint32_t adding = __ballot_sync(0xFFFFFFFFu, adds);
        if (lane == 0) sm.adds[buf][r0 / 32] = adding;
        // Rows that add nothing may hold anything (those past the last are zeros already).
        const bool there = c * kChunkRows + r0 + lane < all_rows;
        for (unsigned rest = ~adding & __ballot_sync(0xFFFFFFFFu, there); rest; rest &= rest - 1u) {
          const int row = r0 + __ffs(rest) - 1;
          if (lane < kUnits)
            *reinterpret_cast<uint4*>(sm.q + buf * C::kQTile + (lane >> 3) * (kChunkRows * 128) + row * 128 + (lane & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.qfull[buf]));
    }
  }
}

// Warp 1: S = K Q^T of every two tiles and chunk.
template <int D, bool kBf16>
__device__ __forceinline__ void products(WSmem<D>& sm, const WeightParams& p, uint32_t tmem, Walk<kWhole> w) {
  using C = WShape<D>;
  const uint32_t id = idesc<kBf16>(static_cast<uint32_t>(p.chunk_rows), 0);
  const uint32_t ring = smem_u32(sm.ring), q = smem_u32(sm.q);
  Ring<C::kStages> at;
  int loads = 0, step = 0, done[2] = {0, 0};
  Segment s;
  while (w.next(p, s)) {
    for (int j = 0; j < s.n; j += 2, ++step, at.advance()) {
      const int g = step & 1;
      if (!wait(sm, sm.kfull[at.stage], at.phase, p)) return;
      for (int c = 0; c < p.chunks; ++c) {
        const int buf = loads & 1, b = done[g] & 1;
        const bool first_use = p.chunks > 1 || j == 0, last_use = p.chunks > 1 || j + 2 >= s.n;
        if (first_use && !wait(sm, sm.qfull[buf], (loads >> 1) & 1, p)) return;
        if (!wait(sm, sm.sempty[g][b], ((done[g] >> 1) & 1) ^ 1, p)) return;
        tc_fence_after();
        const uint32_t d = tmem + (2 * g + b) * kChunkRows;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss_elect(d, sdesc_sw128(ring + at.stage * C::kTile + (k >> 2) * (kTileKeys * 128) + (k & 3) * 32, 16, 1024),
                       sdesc_sw128(q + buf * C::kQTile + (k >> 2) * (kChunkRows * 128) + (k & 3) * 32, 16, 1024), id, k > 0);
        mma_commit_elect(smem_u32(&sm.sfull[g][b]));
        if (c == p.chunks - 1) mma_commit_elect(smem_u32(&sm.kempty[at.stage]));
        if (last_use) {
          mma_commit_elect(smem_u32(&sm.qempty[buf]));
          ++loads;
        }
        ++done[g];
      }
    }
  }
}

// Of kN columns from row `first` on those whose drafts see a key (`seen`: the drafts).
template <int kN>
__device__ __forceinline__ uint32_t seen_columns(const WeightParams& p, uint64_t seen, int first) {
  uint32_t columns = 0;
  const int last = min(p.by_G.of(first + kN - 1), p.q_len - 1);
#pragma unroll 1
  for (int i = p.by_G.of(first); i <= last; ++i) {
    const int lo = max(i * p.G - first, 0), hi = min((i + 1) * p.G - first, kN);
    if (seen >> i & 1ull) columns |= (~0u >> (32 - (hi - lo))) << lo;
  }
  return columns;
}

// kN columns: their sum of 2^(s a + minus_lse).  kEdge: of the rows whose drafts see the
// key and that add something (s may be anything in the others).
template <int kN, bool kEdge>
__device__ __forceinline__ float add_columns(const WeightParams& p, uint32_t s_t, const float* minus, uint32_t adds,
                                             int first_row, uint64_t seen) {
  uint32_t sr[kN];
  if constexpr (kN == 32) MLA_TMEM_LD_32x32b_X32(s_t, sr);
  else MLA_TMEM_LD_32x32b_X16(s_t, sr);
  uint32_t columns = 0;
  if constexpr (kEdge) columns = adds & seen_columns<kN>(p, seen, first_row);
  tmem_ld_wait();
  const uint64_t a2 = f2pack(p.scale_log2, p.scale_log2);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < kN; c += 4) {
    const float4 m = *reinterpret_cast<const float4*>(minus + c);
    float x[4];
    f2unpack(ffma2(f2pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), a2, f2pack(m.x, m.y)), x[0], x[1]);
    f2unpack(ffma2(f2pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), a2, f2pack(m.z, m.w)), x[2], x[3]);
    if constexpr (kEdge) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!(columns >> (c + e) & 1u)) x[e] = -CUDART_INF_F;
    }
    sum[0] = fadd2(sum[0], f2pack(ex2(x[0]), ex2(x[1])));
    sum[1] = fadd2(sum[1], f2pack(ex2(x[2]), ex2(x[3])));
  }
  float s0, s1, s2, s3;
  f2unpack(sum[0], s0, s1);
  f2unpack(sum[1], s2, s3);
  return (s0 + s1) + (s2 + s3);
}

template <bool kEdge>
__device__ __forceinline__ float add_chunk(const WeightParams& p, uint32_t s_t, const float* minus, const uint32_t* adds,
                                           int first_row, uint64_t seen) {
  float sum = 0.f;
  int c = 0;
#pragma unroll 1
  for (; c + 32 <= p.chunk_rows; c += 32)
    sum += add_columns<32, kEdge>(p, s_t + c, minus + c, adds[c / 32], first_row + c, seen);
  if (c < p.chunk_rows) sum += add_columns<16, kEdge>(p, s_t + c, minus + c, adds[c / 32], first_row + c, seen);
  return sum;
}

// Warps 4..11: group g takes every second step, a key a thread.
template <int D>
__device__ __forceinline__ void add_up(WSmem<D>& sm, const WeightParams& p, uint32_t tmem, Walk<kWhole> w, int g, int wq,
                                       int lane) {
  const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
  const int r = wq * 32 + lane, words = (p.q_len + 31) >> 5;
  int loads = 0, step = 0, done = 0;
  Segment s;
  while (w.next(p, s)) {
    const int prefix = s.S - p.q_len;
    for (int j = 0; j < s.n; j += 2, ++step) {
      const bool mine = (step & 1) == g;
      const int key0 = (s.tile0 + j) * kKeys, key = key0 + r;
      const bool valid = mine && key < s.S && (r < kKeys || j + 1 < s.n);
      float* const at = p.weights + (static_cast<long long>(s.b) * p.Hkv + s.head) * p.Smax + key;
      float sum = 0.f, old = 0.f;
      uint64_t seen = ~0ull;                               // drafts that see this key
      if (valid) old = *at;
      const bool edge = __any_sync(0xFFFFFFFFu, valid && key >= prefix);
      if (edge) {
        // A lane loads the masks of two drafts (one read after the other took 0.4 us each).
        const uint32_t* const rows = p.mask + static_cast<size_t>(s.b) * p.q_len * words;
        uint32_t word[2][2] = {};                          // [draft lane or 32 + lane][keys 0 .. 31 or 32 ..]
        if (lane < p.q_len) {
          word[0][0] = rows[lane * words];
          if (words > 1) word[0][1] = rows[lane * words + 1];
        }
        if (words > 1 && 32 + lane < p.q_len) {
          word[1][0] = rows[(32 + lane) * words];
          word[1][1] = rows[(32 + lane) * words + 1];
        }
        const int draft = key - prefix;                    // (may be any number)
        uint64_t drafts = 0;
        for (int i = 0; i < p.q_len; ++i) {
          const uint32_t lo = __shfl_sync(0xFFFFFFFFu, i < 32 ? word[0][0] : word[1][0], i & 31);
          const uint32_t hi = __shfl_sync(0xFFFFFFFFu, i < 32 ? word[0][1] : word[1][1], i & 31);
          drafts |= static_cast<uint64_t>((draft & 32 ? hi : lo) >> (draft & 31) & 1u) << i;
        }
        if (valid && key >= prefix) seen = drafts;
      }
      for (int c = 0; c < p.chunks; ++c) {
        const int buf = loads & 1;
        const bool first_use = p.chunks > 1 || j == 0, last_use = p.chunks > 1 || j + 2 >= s.n;
        if (first_use && !wait(sm, sm.qfull[buf], (loads >> 1) & 1, p)) return;
        if (mine) {
          const int b = done & 1;
          if (!wait(sm, sm.sfull[g][b], (done >> 1) & 1, p)) return;
          tc_fence_after();
          const uint32_t s_t = tmem + lanes + (2 * g + b) * kChunkRows;
          float x = 0.f;
          bool careful = edge;
          if (!edge) {
            x = add_chunk<false>(p, s_t, sm.minus_lse[buf], sm.adds[buf], c * kChunkRows, seen);
            // A key that is not finite gives NaN in the rows that add nothing, too (0 times it):
            // once more, without them.
            careful = __any_sync(0xFFFFFFFFu, valid && x != x);
          }
          if (careful) x = add_chunk<true>(p, s_t, sm.minus_lse[buf], sm.adds[buf], c * kChunkRows, seen);
          sum += x;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.sempty[g][b]));
          ++done;
        }
        if (last_use) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.qempty[buf]));
          ++loads;
        }
      }
      if (valid) *at = old + sum;
    }
  }
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap map_k, const WeightParams p) {
  using C = WShape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  WSmem<D>& sm = *reinterpret_cast<WSmem<D>*>(smem_raw);
  if (smem_u32(smem_raw) & 1023) {
    grid_dependency_wait();
    if (threadIdx.x == 0) atomicOr(p.status, kBitTimeout);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 3) {
    for (int i = lane; i < C::kStages; i += 32) {
      mbar_init(smem_u32(&sm.kfull[i]), p.box_rows ? 1 : 32);
      mbar_init(smem_u32(&sm.kempty[i]), 1);
    }
    if (lane >= 16 && lane < 20) {
      mbar_init(smem_u32(&sm.sfull[(lane >> 1) & 1][lane & 1]), 1);
      mbar_init(smem_u32(&sm.sempty[(lane >> 1) & 1][lane & 1]), 4);
    }
    if (lane == 20 || lane == 21) {
      mbar_init(smem_u32(&sm.qfull[lane & 1]), 2);
      mbar_init(smem_u32(&sm.qempty[lane & 1]), 1 + 8);
    }
    if (lane == 22) {
      mbar_init(smem_u32(&sm.drain), 1);
      sm.abort_flag = 0;
    }
    fence_mbarrier_init_cluster();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  if (tid == 0 && p.box_rows) tma_prefetch_desc(&map_k);
  grid_dependency_wait();
  if (tid == 0) grid_launch_dependents();

  // This CTA's run (as in the attention kernel).
  const int all = p.by_members.of(gridDim.x), team = p.by_members.of(blockIdx.x);
  const int member = static_cast<int>(blockIdx.x) - team * p.members;
  int len, total, start_b = 0, start_pre = 0;
  if (p.B <= 32) {
    // Every warp by itself, a stream a lane.
    int work = 0;
    if (lane < p.B) {
      work = stream_tiles<kWhole>(p, lane, len) * p.head_sets;
      if (blockIdx.x == 0 && warp == 0 && len != 0 && (len < p.q_len || len > p.Smax)) atomicOr(p.status, kBitSeqLen);
    }
    int inc = work;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
    }
    total = __shfl_sync(0xFFFFFFFFu, inc, 31);
    const Runs runs(p, total, all);
    if (team < runs.teams && total > 0) {
      start_b = __ffs(__ballot_sync(0xFFFFFFFFu, inc > runs.start(team))) - 1;
      start_pre = __shfl_sync(0xFFFFFFFFu, inc - work, start_b);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    // Each thread sums a run of streams, then a scan over threads; the thread whose
    // streams hold the first tile says which.
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int sum = 0;
    bool off = false;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      sum += stream_tiles<kWhole>(p, b, len) * p.head_sets;
      off |= len != 0 && (len < p.q_len || len > p.Smax);
    }
    if (off && blockIdx.x == 0) atomicOr(p.status, kBitSeqLen);
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) sm.warp_sum[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i == warp) before = total;
      total += sm.warp_sum[i];
    }
    const Runs runs(p, total, all);
    const int t0 = team < runs.teams ? runs.start(team) : total;
    before += inc - sum;
    if (t0 >= before && t0 < before + sum) {
      int b = b0;
      while (true) {
        const int n = stream_tiles<kWhole>(p, b, len) * p.head_sets;
        if (t0 < before + n) break;
        before += n;
        ++b;
      }
      sm.start_b = b;
      sm.start_pre = before;
    }
    __syncthreads();
    if (t0 < total) {
      start_b = sm.start_b;
      start_pre = sm.start_pre;
    }
  }
  const uint32_t tmem = sm.tmem_base;
  const Runs runs(p, total, all);
  const int t0 = team < runs.teams ? runs.start(team) : total;
  const Walk<kWhole> walk(p, member, t0, team < runs.teams ? runs.start(team + 1) : total, start_b, start_pre);

  if (warp == 0) {
    if (p.box_rows == 0) load_k_gather<D>(sm, p, walk);
    else load_k_tma<D>(sm, p, &map_k, walk);
  } else if (warp == 1) {
    products<D, kBf16>(sm, p, tmem, walk);
    drain_products(sm.drain);
  } else if (warp < 4) {
    load_q<D>(sm, p, walk, warp - 2);
  } else {
    add_up<D>(sm, p, tmem, walk, (warp - 4) >> 2, warp & 3, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using Fn = void (*)(CUtensorMap, WeightParams);
std::mutex g_mutex;
bool g_ready[64][4];

template <int D, bool kBf16>
int pick(int dev, int n, Fn* fn) {
  static_assert(sizeof(WSmem<D>) <= 232448, "one CTA's shared memory");
  *fn = weights_kernel<D, kBf16>;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_ready[dev][n]) {
    if (cudaFuncSetAttribute(*fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(WSmem<D>))) !=
        cudaSuccess) {
      cudaGetLastError();
      return MLA_ERR_LAUNCH;
    }
    g_ready[dev][n] = true;
  }
  return MLA_OK;
}

int run(const Call& c, const float* lse, float* out) {
  if (!shape_ok(c.B, c.q_len, c.H, c.Hkv, c.D) || c.Smax < 1 || c.Smax >= (1 << 24) ||
      static_cast<long long>((c.Smax + kKeys - 1) / kKeys) * c.Hkv >= (1ll << 31) / (c.B > 0 ? c.B : 1))
    return MLA_ERR_SHAPE;
  if ((c.dtype != MLA_BF16 && c.dtype != MLA_FP16) || !std::isfinite(c.scale)) return MLA_ERR_ARG;
  if (c.B == 0) return MLA_OK;
  if (!c.q || !c.k || !c.seq_lens || !c.mask || !lse || !out) return MLA_ERR_NULLPTR;
  if (!aligned_to(c.q, 16) || !aligned_to(c.k, 16) || !aligned_to(lse, 4) || !aligned_to(out, 4) ||
      !aligned_to(c.seq_lens, 4) || !aligned_to(c.mask, 4))
    return MLA_ERR_ALIGN;
  WeightParams p = {};
  const bool paged = c.table != nullptr;
  const long long rows = paged ? c.pool_rows : c.Smax;
  const int batches = paged ? 1 : c.B;
  const long long q_sizes[3] = {c.B, c.q_len, c.H}, k_sizes[3] = {batches, rows, c.Hkv};
  int st = byte_strides(c.strides, q_sizes, c.D, p.q_stride);
  if (st == MLA_OK) st = byte_strides(c.strides ? c.strides + 3 : nullptr, k_sizes, c.D, p.k_stride);
  if (st != MLA_OK) return st;
  DeviceCommon d;
  st = device_common(&d);
  if (st != MLA_OK) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_UNSUPPORTED_DEVICE;
  Fn fn;
  const bool bf16 = c.dtype == MLA_BF16;
  size_t smem;
  if (c.D == 128) {
    smem = sizeof(WSmem<128>);
    st = bf16 ? pick<128, true>(dev, 0, &fn) : pick<128, false>(dev, 1, &fn);
  } else {
    smem = sizeof(WSmem<64>);
    st = bf16 ? pick<64, true>(dev, 2, &fn) : pick<64, false>(dev, 3, &fn);
  }
  if (st != MLA_OK) return st;
  const int grid = cta_count(d);
  const int box = box_rows(c), heads = heads_side_by_side(p.k_stride, c.Hkv, 1, grid);
  CUtensorMap map = {};
  const CUtensorMapL2promotion promotion = c.D == 128 || heads > 1 || p.k_stride[1] == 2 * c.D
                                               ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                               : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  if (box != 0 && encode(d, &map, c.k, c, p.k_stride, rows, batches, box, 1, promotion) != MLA_OK) return MLA_ERR_LAUNCH;
  p.q = static_cast<const uint8_t*>(c.q);
  p.k = static_cast<const uint8_t*>(c.k);
  p.seq_lens = c.seq_lens;
  p.mask = c.mask;
  p.block_table = c.table;
  p.given_lse = lse;
  p.weights = out;
  p.status = d.status_word;
  p.B = c.B;
  p.q_len = c.q_len;
  p.H = c.H;
  p.Hkv = c.Hkv;
  p.G = c.H / c.Hkv;
  p.Smax = c.Smax;
  p.groups = p.group_members = p.group_sets = 1;
  p.members = p.head_members = heads;
  p.head_sets = c.Hkv / heads;
  p.by_members = Divisor(heads);
  p.by_group_members = p.by_group_sets = Divisor(1);
  p.by_G = Divisor(p.G);
  p.max_blocks = c.max_blocks;
  p.page = Divisor(paged ? c.page : 1);
  p.pool_pages = paged ? static_cast<int>(c.pool_rows / c.page) : 0;
  p.box_rows = box;
  p.test_stall = d.test_stall;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  const int all_rows = c.q_len * p.G;
  p.chunks = (all_rows + kChunkRows - 1) / kChunkRows;
  p.chunk_rows = p.chunks > 1 ? kChunkRows : (all_rows + 15) / 16 * 16;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, map, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

}  // namespace weights
}  // namespace gqa
}  // namespace mla

extern "C" {

int mla_gqa_attn_weights(const void* q, const void* k, const int64_t* strides, const int32_t* seq_lens,
                         const uint32_t* tree_mask, const float* lse, int B, int q_len, int H, int Hkv, int D, int Smax,
                         int dtype, float scale, float* weights, cudaStream_t stream) {
  mla::gqa::Call c = {};
  c.q = q;
  c.k = k;
  c.strides = strides;
  c.seq_lens = seq_lens;
  c.mask = tree_mask;
  c.B = B;
  c.q_len = q_len;
  c.H = H;
  c.Hkv = Hkv;
  c.D = D;
  c.Smax = Smax;
  c.dtype = dtype;
  c.scale = scale;
  c.stream = stream;
  return mla::gqa::weights::run(c, lse, weights);
}

int mla_gqa_attn_weights_paged(const void* q, const void* k_pool, const int64_t* strides, long long pool_rows,
                               const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                               const uint32_t* tree_mask, const float* lse, int B, int q_len, int H, int Hkv, int D,
                               int dtype, float scale, float* weights, cudaStream_t stream) {
  if (page_size < 1 || max_blocks < 1 || static_cast<long long>(max_blocks) * page_size >= (1ll << 24) ||
      pool_rows < 1 || pool_rows % page_size != 0 || pool_rows >= (1ll << 31))
    return MLA_ERR_SHAPE;
  if (B > 0 && !block_table) return MLA_ERR_NULLPTR;
  if (!mla::aligned_to(block_table, 4)) return MLA_ERR_ALIGN;
  mla::gqa::Call c = {};
  c.q = q;
  c.k = k_pool;
  c.strides = strides;
  c.seq_lens = seq_lens;
  c.mask = tree_mask;
  c.B = B;
  c.q_len = q_len;
  c.H = H;
  c.Hkv = Hkv;
  c.D = D;
  c.Smax = max_blocks * page_size;
  c.dtype = dtype;
  c.scale = scale;
  c.stream = stream;
  c.table = block_table;
  c.max_blocks = max_blocks;
  c.page = page_size;
  c.pool_rows = pool_rows;
  return mla::gqa::weights::run(c, lse, weights);
}

}  // extern "C"
