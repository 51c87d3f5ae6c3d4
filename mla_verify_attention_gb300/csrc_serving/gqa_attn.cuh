// Verify attention with grouped query heads on sm_103a: the kernels behind
// mla_gqa_verify_attn and mla_gqa_verify_attn_paged (include/mla_verify_attn.h).
//
// Mathematics.  The G = H / Hkv query heads of a key head and the q_len drafts
// of a stream are the rows of one dense product: S = Q K^T over the stream's
// keys, tree mask on the last q_len of them, online softmax (running max m,
// sum l, in log2 units), O = P V.  Keys and values are read once.
//
// What bounds it.  A key costs 4 D bytes and 4 D flops a row, so up to ~290
// rows (measured bf16 rate over measured copy rate) the cache read is the
// floor: the kernel is built to keep ~160 KB of loads in flight on every SM
// and to let nothing else take longer than the tile's share of bandwidth
// (32 KB at D = 128: ~1,500 cycles).
//
// Measured (GPU time, bf16 D = 128 unless said, loads first: share of the
// measured copy rate): 64 streams of 8k keys, one token, 8 heads a key head 317
// us, 6.8 TB/s (100 %); the same at D = 64, 16k keys 325 us (98 %); one stream
// of 64k keys, 9 drafts 50 us, 5.4 TB/s (79 %: ~6.5 us of start and end and ~4 us
// of merge around the stream); 16 streams x 1,024 rows over 8k keys 197 us, 1,395
// TFLOP/s (71 % of the measured bf16 rate: the chain of a tile through products,
// softmax and products again, not any one of them).
//
// Split.  The work is a sequence of 64-key tiles: streams, then key heads,
// then keys.  Every CTA (or team of CTAs, one a group of 128 rows) of one
// persistent wave takes an equal run of that sequence, computed on the device
// from seq_lens, so that ragged batches balance to one tile and nothing is
// planned on the host.  A (stream, head, row group) unit that lies within one run
// is written to `out`; one that is cut leaves unnormalised partials (at most two a
// CTA, which bounds the workspace by the grid) that the combine kernels merge in
// order.
//
// CTA.  A warp each loads K and V tiles (TMA boxes in the 128-byte swizzle), a
// warp each issues the two products (tcgen05.mma), eight softmax warps in two groups take the key tiles in
// turn, each with an accumulator O (128 rows) of its own in tensor memory; their
// (m, l, O) are merged when the unit's run ends.  More rows than 128 are taken
// by as many CTAs side by side, which share the cache reads through L2.  (Two
// row tiles a CTA, one a group, read the cache half as often but were slower:
// 264 rows over 16k keys 44 us against 32, 1,024 rows 45 against 39.)
// S is double-buffered per group in tensor memory (2 x 64 columns); P replaces
// S in place and is the A operand of O += P V.  O is only rescaled when a
// row's max grows by more than 2^8.
//
// Rounding.  P enters the product in v's type, for the tensor cores take both
// operands in one; the sums l stay unrounded fp32.  Against 64 bits out is then
// off by 2.3e-3 in bf16 and 2.9e-4 in fp16 (2-norm, relative), where the rounding
// of the result alone, which an exact P would leave, is 1.7e-3 and 2.1e-4.  P in
// two terms would remove the rest for a second product a tile.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <cstdint>

#include "fp4_format.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace gqa {

constexpr int kKeys = 64;                  // keys a tile
constexpr int kRows = 128;                 // rows a group's accumulator (MMA M)
constexpr int kThreads = 384;              // 4 control warps + 2 x 4 softmax warps
// Fewest tiles a team takes: below that, fewer teams share a short call's work.
constexpr int kMinTiles = 2;
constexpr float kLazy = 8.0f;              // log2 units a row's max may grow before O is rescaled
constexpr uint64_t kWaitNs = 2000000000ull;

// What the kernel attends over: a stream's whole cache, its first keys and a
// sliding window (see Window below), or a whole cache held in 4 bits (gqa_fp4.cu).
enum Mode { kWhole, kWindow, kFp4 };

struct Params {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  long long q_stride[3], k_stride[3], v_stride[3];   // bytes: batch, draft / row, head
  const int32_t* seq_lens;
  const uint32_t* mask;
  const int32_t* block_table;      // null: contiguous caches
  void* out;
  float* lse;
  int4* desc;                      // [grid] cut units: {stream, head * groups + group, first slot, parts}
  float2* part_ml;                 // [2 * grid][part_rows]
  float4* part_o;                  // [2 * grid][part_rows][D / 4]
  unsigned int* status;
  int B, q_len, H, Hkv, G, Smax, groups, part_rows;
  int members, head_members, group_members;   // CTAs a team: key heads x row groups side by side
  int head_sets, group_sets;       // ... and one after the other
  int desc_units;                  // entries of `desc`: one a unit, or one a CTA
  int whole;                       // units are not cut (short caches): the work is counted in units
  int max_blocks, pool_pages;
  Divisor page, by_members, by_group_members, by_group_sets, by_G;
  int box_rows;                    // rows a TMA box: 64 or a divisor that no page boundary cuts; 0: gather
  int test_stall;
  float scale_log2;
  int window, sinks;               // kWindow
  int steps_at;                    // kFp4: where a row's steps begin
  float v_factor;
};

template <int D, Mode kMode>
struct Shape {
  static constexpr int kThreads = kMode == kFp4 ? 512 : gqa::kThreads;
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kKeys * D * 2;          // bytes of a K or V tile
  static constexpr int kQTile = kRows * D * 2;
  // 160 KB of K and V tiles, or 96 KB in 16 bits and 54 or 72 KB in 4.
  static constexpr int kStages = (kMode == kFp4 ? 3 : 5) * (D == 128 ? 1 : 2);
  static constexpr int kRing = 2 * kStages * kTile;
  static constexpr int kCodes = kKeys * D / 2, kSteps = kKeys * 16;          // bytes of a tile in 4 bits
  static constexpr int kPacked = D == 128 ? 6 : 14;    // stages of them
};

// What only some forms have.
template <int D, Mode kMode>
struct Extra {};
template <int D>
struct Extra<D, kFp4> {
  using C = Shape<D, kFp4>;
  __align__(1024) uint8_t codes[2][C::kPacked][C::kCodes];   // [K, V]
  uint8_t steps[2][C::kPacked][C::kSteps];             // 16 bytes a row, this head's among them
  float q_unit[2][kRows];                              // what a row of Q was divided by
  uint64_t packed_full[2][C::kPacked], packed_empty[2][C::kPacked];
};

template <int D, Mode kMode>
struct __align__(1024) Smem {
  using C = Shape<D, kMode>;
  uint8_t q[2 * C::kQTile];                            // this segment's rows and the next one's
  uint8_t ring[C::kRing];                              // stage s: K tile, V tile
  float2 ml[2][kRows];
  uint64_t kfull[C::kStages], kempty[C::kStages];
  uint64_t vfull[C::kStages], vempty[C::kStages];
  uint64_t sfull[2][2], pfull[2][2], pvdone[2][2];     // [group][buffer]
  // (qfree: one a segment parity.  The products can be through with a short
  // segment before a softmax warp asks for the one before it.)
  uint64_t qfull, qfree[2], ofull, ofree, mlx, drain[2];
  int warp_sum[C::kThreads / 32], start_b, start_pre;
  uint32_t tmem_base, abort_flag;
  Extra<D, kMode> extra;
};

// ------------------------------------------------------------ instructions

template <bool kBf16>
__host__ __device__ constexpr uint32_t idesc(uint32_t N, uint32_t b_mn) {
  return (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// Shared-memory matrix descriptors (128-byte swizzle, 1 KB between groups of
// eight rows) have a constant upper half; the lower half holds the address and,
// for V, the distance between 64-wide chunks.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// The products are issued by one elected lane of a converged warp: the operands
// then move to uniform registers once, not lane by lane (a single-lane loop
// took 1.5 times as long).  A tile's products and the commits that follow them
// are one block, with one election.

// S = Q K^T of one tile, A and B K-major in shared memory: D / 64 chunks of four
// K = 16 steps; then the commits to `bar0`, `bar1` and, at the end, `bar2`.
#define MLA_QK_CHUNK(ao, bo, first)                                                                   \
  " add.u32 x, %1, " #ao ";\n add.u32 y, %2, " #bo ";\n mov.b64 a, {x, %8};\n mov.b64 b, {y, %8};\n" \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " #first ";\n"                              \
  " add.u32 x, %1, " #ao " + 2;\n add.u32 y, %2, " #bo " + 2;\n mov.b64 a, {x, %8};\n mov.b64 b, {y, %8};\n" \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n"                                       \
  " add.u32 x, %1, " #ao " + 4;\n add.u32 y, %2, " #bo " + 4;\n mov.b64 a, {x, %8};\n mov.b64 b, {y, %8};\n" \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n"                                       \
  " add.u32 x, %1, " #ao " + 6;\n add.u32 y, %2, " #bo " + 6;\n mov.b64 a, {x, %8};\n mov.b64 b, {y, %8};\n" \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n"
#define MLA_COMMIT(pred, bar) \
  " @" #pred " tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [" #bar "];\n"
#define MLA_QK_BODY(chunks)                                                                                        \
  asm volatile("{\n .reg .pred e, z, c;\n .reg .b32 x, y;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n" \
               " setp.ne.and.b32 c, %7, 0, e;\n setp.ne.b32 z, 0, 0;\n" chunks                                       \
               MLA_COMMIT(e, %4) MLA_COMMIT(e, %5) MLA_COMMIT(c, %6) "}" ::"r"(d),                                  \
               "r"(a), "r"(b), "r"(id), "r"(bar0), "r"(bar1), "r"(bar2), "r"(static_cast<uint32_t>(end)),           \
               "n"(kDescHi)                                                                                         \
               : "memory")
template <int kChunks>
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t bar0, uint32_t bar1,
                                         uint32_t bar2, bool end) {
  // Chunks lie 16 KB (Q, 128 rows) and 8 KB (K, 64 keys) apart: 1024 and 512 descriptor units.
  static_assert(kRows * 128 >> 4 == 1024 && kKeys * 128 >> 4 == 512, "chunk distances");
  if (kChunks == 1) MLA_QK_BODY(MLA_QK_CHUNK(0, 0, z));
  else MLA_QK_BODY(MLA_QK_CHUNK(0, 0, z) MLA_QK_CHUNK(1024, 512, 1));
}

// O (+)= P V over 64 keys: P in tensor memory (8 columns a K = 16 step), V
// MN-major in shared memory (16 rows of 128 bytes a step); then the commits.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t bar0,
                                         uint32_t bar1, uint32_t bar2, bool end) {
  asm volatile(
      "{\n .reg .pred e, p, c;\n .reg .b32 x, y;\n .reg .b64 b;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.and.b32 c, %8, 0, e;\n mov.b64 b, {%2, %9};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n"
      " add.u32 x, %1, 8;\n add.u32 y, %2, 128;\n mov.b64 b, {y, %9};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n"
      " add.u32 x, %1, 16;\n add.u32 y, %2, 256;\n mov.b64 b, {y, %9};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n"
      " add.u32 x, %1, 24;\n add.u32 y, %2, 384;\n mov.b64 b, {y, %9};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n" MLA_COMMIT(e, %5) MLA_COMMIT(e, %6)
      MLA_COMMIT(c, %7) "}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(bar0), "r"(bar1), "r"(bar2),
      "r"(static_cast<uint32_t>(end)), "n"(kDescHi)
      : "memory");
}

// One box of a cache by the elected lane of a converged warp.
__device__ __forceinline__ void tma_box_elect(uint32_t dst, const CUtensorMap* map, int row, int chunk, int head,
                                              int batch, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(head), "r"(batch), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_expect_elect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar), "r"(bytes)
      : "memory");
}

// 16 bytes to shared memory, or 16 zero bytes when !full.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (kBf16) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------ waits

// Bounded; gives up at once when another warp of the CTA has.
template <class S>
__device__ __forceinline__ bool wait_loop(S& sm, uint32_t bar, uint32_t parity, const Params& p) {
  for (int i = 0; i < 64; ++i)       // (reading the timer takes longer than most waits)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile uint32_t*>(&sm.abort_flag)) return false;
    if (globaltimer_ns() - t0 > kWaitNs) {
      atomicOr(p.status, kBitTimeout);
      *reinterpret_cast<volatile uint32_t*>(&sm.abort_flag) = 1u;
      return false;
    }
  }
}
constexpr long long kWaitCycles = 4000000000ll;    // two seconds at 2 GHz
// Out of line, except where warps have register counts of their own (a call's
// registers cannot be allocated there).
template <class S>
__device__ __noinline__ bool wait_call(S& sm, uint32_t bar, uint32_t parity, const Params& p) {
  return wait_loop(sm, bar, parity, p);
}
template <class S>
struct InlineWaits {
  static constexpr bool value = false;
};
template <int D>
struct InlineWaits<Smem<D, kFp4>> {
  static constexpr bool value = true;
};
template <class S>
__device__ __forceinline__ bool wait_slow(S& sm, uint32_t bar, uint32_t parity, const Params& p) {
  if constexpr (InlineWaits<S>::value) {
    // Little code, for it stands at every wait: with the loop above here instead, one stream
    // of 64k keys in 4 bits, 9 drafts took 52 us, not 41.
    const long long t0 = clock64();
    while (!*reinterpret_cast<volatile uint32_t*>(&sm.abort_flag)) {
      if (mbar_try_wait(bar, parity)) return true;
      if (clock64() - t0 > kWaitCycles) {
        atomicOr(p.status, kBitTimeout);
        *reinterpret_cast<volatile uint32_t*>(&sm.abort_flag) = 1u;
      }
    }
    return false;
  } else {
    return wait_call(sm, bar, parity, p);
  }
}
// By a whole converged warp; the result is warp-uniform.
template <class S>
__device__ __forceinline__ bool wait(S& sm, uint64_t& bar, uint32_t parity, const Params& p) {
  bool ok = mbar_try_wait(smem_u32(&bar), parity);
  if (!ok) ok = wait_slow(sm, smem_u32(&bar), parity, p);
  return __all_sync(0xFFFFFFFFu, ok);
}

// For two barriers at once: half the lanes ask for each.  A lane has then only
// seen what is ordered before its own barrier; __syncwarp orders that before what
// any lane does next (a vote alone orders no memory).
template <class S>
__device__ __forceinline__ bool wait2(S& sm, uint64_t& bar0, uint32_t parity0, uint64_t& bar1, uint32_t parity1,
                                      const Params& p) {
  const bool odd = (threadIdx.x & 1) != 0;
  const uint32_t bar = odd ? smem_u32(&bar1) : smem_u32(&bar0), parity = odd ? parity1 : parity0;
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = wait_slow(sm, bar, parity, p);
  ok = __all_sync(0xFFFFFFFFu, ok);
  __syncwarp();
  return ok;
}

// ------------------------------------------------------------ work

// With a window a draft sees the last `window` of the keys that its mask shows
// it, and those in the first `sinks` rows of the cache.  Prefix keys from `sinks`
// to `start` = prefix - window are seen by no draft, whatever its mask; whole
// tiles of them are skipped: of the stream's tiles, `first` lie before the gap.
// (A draft whose mask shows n drafts sees the prefix from prefix - window + n:
// the n - 1 keys or fewer between are left to the mask.)
struct Window {
  int start, first, gap;
  __device__ __forceinline__ Window(const Params& p, int S) {
    start = max(0, S - p.q_len - p.window);
    first = (min(p.sinks, start) + kKeys - 1) / kKeys;
    gap = max(0, start / kKeys - first);
  }
};

// Key tiles of stream b that are read; 0 for an unused stream and for one whose length is out of range.
template <Mode kMode>
__device__ __forceinline__ int stream_tiles(const Params& p, int b, int& S) {
  S = p.seq_lens[b];
  if (S < p.q_len || S > p.Smax) return 0;
  const int nt = (S + kKeys - 1) / kKeys;
  if constexpr (kMode == kWindow) return nt - Window(p, S).gap;
  return nt;
}

// Its work a unit: tiles, or with p.whole the unit itself.
__device__ __forceinline__ int stream_work(const Params& p, int nt) { return p.whole ? (nt > 0 ? 1 : 0) : nt; }

// A CTA's part of one unit.
struct Segment {
  int b, S, head, group, tile0, n, nt;   // tiles tile0 .. tile0 + n - 1 of the unit's nt
  int start, first, gap;                 // kWindow
  // First key of the segment's tile j.
  template <Mode kMode>
  __device__ __forceinline__ int key(int j) const {
    int t = tile0 + j;
    if constexpr (kMode == kWindow) t += t < first ? 0 : gap;
    return t * kKeys;
  }
};

// The teams' runs of a total of work: equal, the first `more` one longer.
// (Divisions are by products where the divisor is the call's: an integer
// division by a variable cost a call half a microsecond at its start.)
struct Runs {
  int teams, each, more;
  __device__ __forceinline__ Runs(const Params& p, int total, int all) {
    teams = max(1, min(p.whole ? total : total / kMinTiles, all));
    each = total / teams;
    more = total - each * teams;
  }
  __device__ __forceinline__ int start(int team) const { return team * each + min(team, more); }
  __device__ __forceinline__ int team_of(int t) const {
    const int longer = more * (each + 1);
    return t < longer ? t / (each + 1) : more + (t - longer) / each;
  }
};

// Walks a CTA's run of work [t, t1); every role walks it on its own.  The row
// groups of a key head, and key heads whose rows interleave in the cache, are
// taken side by side by the CTAs of a team, which have the same run: they read
// the same tiles at the same time, so that the caches come from HBM once (one
// after the other, 1,024 rows a head over 8k keys read them four times at 5.2
// TB/s) and in whole rows.  A group that does not exist is skipped.
template <Mode kMode>
struct Walk {
  int t, t1, pre;                          // pre: work before stream b
  int b, S, nt, head0, group0;
  __device__ __forceinline__ Walk(const Params& p, int member, int t0, int t1_, int b0, int pre0)
      : t(t0), t1(t1_), pre(pre0), b(b0), S(0), nt(0) {
    head0 = p.by_group_members.of(member);
    group0 = member - head0 * p.group_members;
    if (t < t1) nt = stream_tiles<kMode>(p, b, S);
  }
  __device__ __forceinline__ bool next(const Params& p, Segment& s) {
    const int units = p.head_sets * p.group_sets;
    while (t < t1) {
      while (t >= pre + stream_work(p, nt) * units) {
        pre += stream_work(p, nt) * units;
        nt = stream_tiles<kMode>(p, ++b, S);
      }
      const int local = t - pre, work = stream_work(p, nt);
      const int u = local < work ? 0 : local / work;
      const int head_set = p.by_group_sets.of(u);
      s.b = b;
      s.S = S;
      s.nt = nt;
      if constexpr (kMode == kWindow) {
        const Window w(p, S);
        s.start = w.start;
        s.first = w.first;
        s.gap = w.gap;
      }
      s.tile0 = local - u * work;
      s.head = head_set * p.head_members + head0;
      s.group = (u - head_set * p.group_sets) * p.group_members + group0;
      const int n = min(t1 - t, work - s.tile0);
      s.n = p.whole ? nt : n;
      t += n;
      if (s.group < p.groups) return true;
    }
    return false;
  }
};

__device__ __forceinline__ int rows_of_group(const Params& p, int group) {
  return min(kRows, p.q_len * p.G - group * kRows);
}

// Keys k0 .. k0 + 63 that a row with draft mask `mask64` sees: those before the
// drafts, np of which lie in the tile (np < 64, may be negative), then its drafts.
__device__ __forceinline__ uint64_t visible(uint64_t mask64, int np) {
  if (np > 0) return ((1ull << np) - 1ull) | mask64 << np;
  return -np < 64 ? mask64 >> (-np) : 0ull;
}

// Of keys k0 .. k0 + 63, those from row `from` of the cache to row `to`.
__device__ __forceinline__ uint64_t between(int k0, int from, int to) {
  const int lo = max(from - k0, 0), hi = min(to - k0, kKeys);
  if (lo >= hi) return 0ull;
  return (~0ull >> (kKeys - (hi - lo))) << lo;
}

// The drafts of stream b that any of its drafts sees, by a whole converged warp;
// `word`: the lane's draft's mask, where one word holds it.
__device__ __forceinline__ uint64_t seen_drafts(const Params& p, int b, uint32_t word, int lane) {
  if (p.q_len <= 32) return __reduce_or_sync(0xFFFFFFFFu, word) & (~0u >> (32 - p.q_len));
  const uint32_t* rows = p.mask + static_cast<size_t>(b) * p.q_len * 2;
  uint32_t lo = 0, hi = 0;
  for (int i = lane; i < p.q_len; i += 32) {
    lo |= rows[2 * i];
    hi |= rows[2 * i + 1];
  }
  lo = __reduce_or_sync(0xFFFFFFFFu, lo);
  hi = __reduce_or_sync(0xFFFFFFFFu, hi) & (~0u >> (64 - p.q_len));
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// ------------------------------------------------------------ loads

// Pool row of a key of stream b, in two steps: the table's entry is loaded well
// before its value is looked at (a check straight after the load waited for it, a
// tile: 64 streams of 8k keys on 4-row pages took 610 us).
__device__ __forceinline__ int table_entry(const Params& p, int b, int key) {
  return p.block_table[static_cast<size_t>(b) * p.max_blocks + p.page.of(key)];
}
// A page outside the pool is reported, and page 0 read.
__device__ __forceinline__ int pool_row(const Params& p, int page, int key) {
  if (page < 0 || page >= p.pool_pages) {
    atomicOr(p.status, kBitPage);
    page = 0;
  }
  const int size = static_cast<int>(p.page.d);
  return page * size + (key - p.page.of(key) * size);
}

// Position in a ring of stages.
template <int kStages>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Warps 0 (K) and 2 (V): tiles by TMA.  A tile is one box of 64 rows, or boxes
// of box_rows rows and 64 dims when pages are shorter than a tile.  (One warp
// for both took longer to issue a tile's copies than the memory to deliver them.)
// With a window, boxes without a key that a draft may see are left out.
template <int D, Mode kMode>
__device__ __forceinline__ void load_tma(Smem<D, kMode>& sm, const Params& p, const CUtensorMap* map, Walk<kMode> w, bool is_v) {
  using C = Shape<D, kMode>;
  const int lane = threadIdx.x & 31;
  uint64_t* const full = is_v ? sm.vfull : sm.kfull;
  uint64_t* const empty = is_v ? sm.vempty : sm.kempty;
  const uint32_t ring = smem_u32(sm.ring) + (is_v ? C::kTile : 0);
  // Boxes along the keys.  The lanes look up the rows of 32 of them, `batch_tiles`
  // tiles, together and a batch ahead.
  const int R = p.box_rows, shift = __ffs(R) - 1, boxes = kKeys >> shift, batch_tiles = 32 / boxes;
  const bool paged = p.block_table != nullptr;
  Ring<C::kStages> at;
  int issued = 0;
  Segment s;
  while (w.next(p, s)) {
    const int end = min(s.S, (s.tile0 + s.n) * kKeys);
    auto key_of = [&](int j) {
      if constexpr (kMode == kWindow) return s.template key<kMode>(j + (lane >> (6 - shift))) + (lane & (boxes - 1)) * R;
      return (s.tile0 + j) * kKeys + lane * R;
    };
    auto wanted = [&](int j) {
      const int key = key_of(j);
      if constexpr (kMode == kWindow)
        return j + (lane >> (6 - shift)) < s.n && key < s.S && (key < p.sinks || key + R > s.start);
      return key < end;
    };
    auto entry_of = [&](int j) { return paged && wanted(j) ? table_entry(p, s.b, key_of(j)) : 0; };
    const int batch = paged ? 0 : s.b;
    int row = 0, entry = entry_of(0), first = 0;           // `first`: lane of the tile's first box
    uint32_t wanted_lanes = 0;                             // (kWindow)
    for (int j = 0; j < s.n; ++j, at.advance(), first = (first + boxes) & 31) {
      if (first == 0) {
        row = !paged ? key_of(j) : (wanted(j) ? pool_row(p, entry, key_of(j)) : 0);
        if constexpr (kMode == kWindow) wanted_lanes = __ballot_sync(0xFFFFFFFFu, wanted(j));
        entry = entry_of(j + batch_tiles);
      }
      if (!wait(sm, empty[at.stage], at.phase ^ 1, p)) goto out;
      const uint32_t bar = smem_u32(&full[at.stage]), dst = ring + at.stage * 2 * C::kTile;
      if (p.test_stall && is_v && issued == 0 && blockIdx.x == 0) goto out;       // this load never comes
      if (R == kKeys) {
        arrive_expect_elect(bar, C::kTile);
        tma_box_elect(dst, map, __shfl_sync(0xFFFFFFFFu, row, first), 0, s.head, batch, bar);
      } else {
        int n = min(boxes, (s.S - s.template key<kMode>(j) + R - 1) >> shift);     // boxes with keys of the stream
        int left_out = 0;
        if constexpr (kMode == kWindow) left_out = n - __popc(wanted_lanes >> first & ((1u << n) - 1u));
        arrive_expect_elect(bar, (n - left_out) * R * D * 2);
        for (int i = 0; i < n; ++i) {
          if (kMode == kWindow && !(wanted_lanes >> (first + i) & 1u)) continue;
          const int r = __shfl_sync(0xFFFFFFFFu, row, first + i);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_box_elect(dst + c * (kKeys * 128) + i * R * 128, map, r, c, s.head, batch, bar);
        }
      }
      ++issued;
    }
  }
out:
  // The copies issued must have landed before the CTA may end.
  for (int n = issued - 1; n >= 0 && n >= issued - C::kStages; --n)
    mbar_wait(smem_u32(&full[n % C::kStages]), (n / C::kStages) & 1, kWaitNs / 2);
}

// Warps 0 (K) and 2 (V) when no TMA box fits the pages (page_size not a
// multiple of 8): rows copied 16 bytes a lane, into the layout the boxes would
// leave; rows past the stream are zeros.  A lane looks up the pages of two rows
// of the next tile while it copies this one.
template <int D, Mode kMode>
__device__ __forceinline__ void load_gather(Smem<D, kMode>& sm, const Params& p, Walk<kMode> w, bool is_v) {
  using C = Shape<D, kMode>;
  constexpr int kUnits = D / 8;                // 16-byte units a row
  constexpr int kPer = 32 / kUnits;            // rows a warp copies at once
  constexpr int kAhead = C::kStages - 1 < 8 ? C::kStages - 1 : 8;   // stages in flight
  constexpr int kTablesAhead = 6;              // tiles
  const int lane = threadIdx.x & 31;
  uint64_t* const full = is_v ? sm.vfull : sm.kfull;
  uint64_t* const empty = is_v ? sm.vempty : sm.kempty;
  const uint32_t ring = smem_u32(sm.ring) + (is_v ? C::kTile : 0);
  const uint8_t* const pool = is_v ? p.v : p.k;
  const long long row_stride = is_v ? p.v_stride[1] : p.k_stride[1];
  const long long head_stride = is_v ? p.v_stride[2] : p.k_stride[2];
  const bool withheld = p.test_stall && is_v && blockIdx.x == 0;
  Ring<C::kStages> at, landed;
  int started = 0;
  auto publish = [&]() {                       // the oldest tile's copies of this lane have landed
    fence_proxy_async_smem();
    if (!withheld) mbar_arrive(smem_u32(&full[landed.stage]));
    landed.advance();
  };
  Segment s;
  while (w.next(p, s)) {
    auto key_of = [&](int j, int half) { return s.template key<kMode>(j) + half * 32 + lane; };
    auto wanted = [&](int key) {
      if constexpr (kMode == kWindow) return key < s.S && (key < p.sinks || key >= s.start);
      return key < s.S;
    };
    auto entry_of = [&](int j, int half) {
      return j < s.n && wanted(key_of(j, half)) ? table_entry(p, s.b, key_of(j, half)) : 0;
    };
    auto row_of = [&](int j, int half, int entry) {        // -1 past the stream, or in the gap
      return wanted(key_of(j, half)) ? pool_row(p, entry, key_of(j, half)) : -1;
    };
    auto prefetch = [&](int j) {               // the table's entries for tile j, soon to be looked up
      const int key = s.template key<kMode>(j) + lane * 2;
      if (j < s.n && key < s.S)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.block_table + static_cast<size_t>(s.b) * p.max_blocks +
                                                      p.page.of(key)));
    };
    for (int j = 1; j < kTablesAhead; ++j) prefetch(j);
    const uint8_t* const head = pool + s.head * head_stride + (lane % kUnits) * 16;
    int lo_next = entry_of(0, 0), hi_next = entry_of(0, 1);
    for (int j = 0; j < s.n; ++j, at.advance()) {
      prefetch(j + kTablesAhead);
      const int lo = row_of(j, 0, lo_next), hi = row_of(j, 1, hi_next);
      lo_next = entry_of(j + 1, 0);
      hi_next = entry_of(j + 1, 1);
      if (!wait(sm, empty[at.stage], at.phase ^ 1, p)) goto out;
      const uint32_t dst = ring + at.stage * 2 * C::kTile + (lane % kUnits >> 3) * (kKeys * 128);
#pragma unroll
      for (int e = 0; e < kKeys / kPer; ++e) {
        const int r = e * kPer + lane / kUnits;                     // row of the tile
        const int row = __shfl_sync(0xFFFFFFFFu, e * kPer < 32 ? lo : hi, r & 31);
        cp_async_16(dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4), head + (row < 0 ? 0 : row) * row_stride, row >= 0);
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

// ------------------------------------------------------------ loads of a cache in 4 bits
//
// Warps 0 (K) and 2 (V) bring a tile's codes and steps into a ring in 4 bits, by TMA or,
// where pages are not a multiple of eight rows, row by row; two more warps each (12 and
// 13, 14 and 15) turn them into the 16-bit tiles of the products, a tile each in turn.
// (A code times its step is exact in fp16, whatever the type of Q; the pools' factors go
// to the scale and to the result.)  The 16-byte units of a row's codes are swizzled, as
// TMA does, so that eight lanes that read a unit of eight rows, and then write eight rows of
// a tile, meet no bank twice.
// Measured (GPU time, bf16, D = 128): one stream of 64k keys, 9 drafts of 8 heads a key
// head 39.9 us, 64 streams of 1k to 32k keys, 5 tokens 353 us: ~1,000 cycles a tile of
// 64 keys, most of them the softmax's, whose warps, the unpacking and the products' share
// the instruction cache (16-bit caches: 860 cycles).  The kernel spills: 72 bytes stored, 360
// loaded, in a thread's 128 registers at launch (168 and 88 by role).
struct Fp4Maps {
  CUtensorMap codes[2], steps[2];              // K, V: boxes of D / 2 and of 16 bytes
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
               : "memory");
}

template <int D>
__device__ __forceinline__ int code_unit(int row, int u) {
  return row * (D / 32) + (u ^ (D == 128 ? row >> 1 & 3 : row >> 2 & 1));
}

// 4, 8 or 16 bytes to shared memory, or as many zero bytes when !full.
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool full) {
  static_assert(kBytes == 4 || kBytes == 8, "");
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(full ? kBytes : 0)
               : "memory");
}

// A box a lane, looked up together and a tile ahead.
template <int D>
__device__ __forceinline__ void load_packed_boxes(Smem<D, kFp4>& sm, const Params& p, const Fp4Maps& maps, Walk<kFp4> w,
                                                  bool is_v) {
  using C = Shape<D, kFp4>;
  const int lane = threadIdx.x & 31, R = p.box_rows, shift = __ffs(R) - 1;
  const CUtensorMap* const codes = &maps.codes[is_v];
  const CUtensorMap* const steps = &maps.steps[is_v];
  const uint32_t dst = smem_u32(sm.extra.codes[is_v]) + lane * R * (D / 2);
  const uint32_t dst_steps = smem_u32(sm.extra.steps[is_v]) + lane * R * 16;
  Ring<C::kPacked> at;
  int issued = 0;
  Segment s;
  while (w.next(p, s)) {
    const int end = min(s.S, (s.tile0 + s.n) * kKeys), step_x = (p.steps_at + s.head * (D / 16)) & ~15;
    auto entry_of = [&](int key) { return lane * R < kKeys && key < end ? table_entry(p, s.b, key) : 0; };
    int key = s.tile0 * kKeys + lane * R;
    int next = entry_of(key);
    for (int k0 = s.tile0 * kKeys; k0 < end; k0 += kKeys, key += kKeys, at.advance()) {
      const int n = min(kKeys, end - k0) + R - 1 >> shift;   // boxes
      const int row = lane < n ? pool_row(p, next, key) : 0;
      next = entry_of(key + kKeys);
      if (!wait(sm, sm.extra.packed_empty[is_v][at.stage], at.phase ^ 1, p)) goto out;
      const uint32_t bar = smem_u32(&sm.extra.packed_full[is_v][at.stage]);
      if (p.test_stall && is_v && issued == 0 && blockIdx.x == 0) goto out;         // this load never comes
      arrive_expect_elect(bar, n * R * (D / 2 + 16));
      __syncwarp();
      if (lane < n) {
        tma_rows(dst + at.stage * C::kCodes, codes, s.head * (D / 2), row, bar);
        tma_rows(dst_steps + at.stage * C::kSteps, steps, step_x, row, bar);
      }
      ++issued;
    }
  }
out:
  for (int n = issued - 1; n >= 0 && n >= issued - C::kPacked; --n)
    mbar_wait(smem_u32(&sm.extra.packed_full[is_v][n % C::kPacked]), (n / C::kPacked) & 1, kWaitNs / 2);
}

template <int D>
__device__ __forceinline__ void load_packed_rows(Smem<D, kFp4>& sm, const Params& p, Walk<kFp4> w, bool is_v) {
  using C = Shape<D, kFp4>;
  constexpr int kUnits = D / 32, kPer = 32 / kUnits;     // 16-byte units of a row's codes, rows a warp copies at once
  const int lane = threadIdx.x & 31;
  const uint8_t* const pool = is_v ? p.v : p.k;
  const long long row_stride = is_v ? p.v_stride[1] : p.k_stride[1];
  const uint32_t full = smem_u32(sm.extra.packed_full[is_v]);
  // (The swizzle of a row is that of row + kPer.)
  const uint32_t dst = smem_u32(sm.extra.codes[is_v]) + code_unit<D>(lane / kUnits, lane % kUnits) * 16;
  const uint32_t dst_steps = smem_u32(sm.extra.steps[is_v]) + lane * 16;
  const bool withheld = p.test_stall && is_v && blockIdx.x == 0;
  constexpr int kEntries = 3;                            // tiles whose table entries are under way
  Ring<C::kPacked> at;
  Segment s;
  while (w.next(p, s)) {
    const int end = min(s.S, (s.tile0 + s.n) * kKeys);
    auto entry_of = [&](int key) { return key < end ? table_entry(p, s.b, key) : 0; };
    const uint8_t* const codes = pool + s.head * (D / 2) + (lane % kUnits) * 16;
    const uint8_t* const steps = pool + p.steps_at + s.head * (D / 16);
    const int step_rest = s.head * (D / 16) & 15;
    int key = s.tile0 * kKeys + lane;
    int next[kEntries][2];                               // of this tile and those behind it
#pragma unroll
    for (int e = 0; e < kEntries; ++e)
#pragma unroll
      for (int h = 0; h < 2; ++h) next[e][h] = entry_of(key + e * kKeys + 32 * h);
    for (; key - lane < end; key += kKeys, at.advance()) {
      int row[2];                                        // -1 past the stream
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row[h] = key + 32 * h < end ? pool_row(p, next[0][h], key + 32 * h) : -1;
#pragma unroll
        for (int e = 1; e < kEntries; ++e) next[e - 1][h] = next[e][h];
        next[kEntries - 1][h] = entry_of(key + kEntries * kKeys + 32 * h);
      }
      if (!wait(sm, sm.extra.packed_empty[is_v][at.stage], at.phase ^ 1, p)) goto out;
#pragma unroll
      for (int e = 0; e < kKeys / kPer; ++e) {
        const int r = __shfl_sync(0xFFFFFFFFu, row[e * kPer >= 32], (e * kPer & 31) + lane / kUnits);
        cp_async_16(dst + at.stage * C::kCodes + e * 512, codes + max(r, 0) * row_stride, r >= 0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        cp_async_small<D / 16>(dst_steps + at.stage * C::kSteps + h * 512 + step_rest, steps + max(row[h], 0) * row_stride,
                               row[h] >= 0);
      if (!withheld)                                     // arrives when this lane's copies have
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full + at.stage * 8) : "memory");
    }
  }
out:
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One of the two warps of K or V: every second tile.
template <int D>
__device__ __forceinline__ void unpack_tiles(Smem<D, kFp4>& sm, const Params& p, Walk<kFp4> w, bool is_v, int half) {
  using C = Shape<D, kFp4>;
  constexpr int kUnits = D / 32;               // 16-byte units of a row's codes: 32 values
  constexpr int kTimes = kKeys * kUnits / 32;  // units a lane
  const int lane = threadIdx.x & 31;
  uint64_t* const full = is_v ? sm.vfull : sm.kfull;
  uint64_t* const empty = is_v ? sm.vempty : sm.kempty;
  // Unit u of row row0 + e * 32 / kUnits.
  const int u = lane >> 3 & (kUnits - 1), row0 = (lane >> 3) / kUnits * 8 + (lane & 7);
  Ring<C::kPacked> from;
  Ring<C::kStages> to;
  int turn = 0;
  Segment s;
  while (w.next(p, s)) {
    for (int j = 0; j < s.n; ++j, from.advance(), to.advance(), turn ^= 1) {
      if (turn != half) continue;
      if (!wait(sm, sm.extra.packed_full[is_v][from.stage], from.phase, p)) return;
      const uint8_t* const codes = sm.extra.codes[is_v][from.stage];
      const uint8_t* const steps = sm.extra.steps[is_v][from.stage] + (s.head * (D / 16) & 15);
      if (!wait(sm, empty[to.stage], to.phase ^ 1, p)) return;
      uint8_t* const tile = sm.ring + to.stage * 2 * C::kTile + (is_v ? C::kTile : 0) + (u >> 1) * (kKeys * 128);
      // (A loop of few instructions, the next unit loaded ahead: unrolled further, it and the
      // softmax's code take turns in the instruction cache.  One stream of 64k keys, 9
      // drafts: 41.1, 39.7, 39.6 and 48.3 us with 1, 2, 4 and 8 units of its 8.)
      auto load = [&](int row, uint4& c, uint32_t& two) {
        c = *reinterpret_cast<const uint4*>(codes + code_unit<D>(row, u) * 16);
        two = *reinterpret_cast<const uint16_t*>(steps + row * 16 + u * 2);
      };
      uint4 next;
      uint32_t next_two;
      load(row0, next, next_two);
#pragma unroll 2
      for (int e = 0; e < kTimes; ++e) {
        const int row = row0 + e * (32 / kUnits);
        const uint32_t words[4] = {next.x, next.y, next.z, next.w}, step2 = fp4::from_e4m3x2(next_two);
        if (e + 1 < kTimes) load(row + 32 / kUnits, next, next_two);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t step = __byte_perm(step2, step2, i < 2 ? 0x1010 : 0x3232);
          uint32_t h[4];
          fp4::from_e2m1x8(words[i], h);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[y]), *reinterpret_cast<const __half2*>(&step));
            h[y] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(tile + row * 128 + ((((u & 1) * 4 + i) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.extra.packed_empty[is_v][from.stage]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full[to.stage]));
    }
  }
}

// ------------------------------------------------------------ products

// A segment's tiles are taken by the two softmax groups in turn.  Issuing one
// tile's products takes a warp several hundred cycles (waits, descriptors,
// commits), as long as the tensor pipe needs for them; S = Q K^T and O += P V
// are therefore issued by a warp each, and run apart by as many tiles as there
// are S buffers.  (One product of 128 keys for both groups at a time gained 7 %
// at D = 64 and lost as much or more with 264 and 1,024 rows, whose groups then
// wait for each other; three S buffers a group, where tensor memory has room,
// gained nothing.)

// Warp 1: S of every tile.
template <int D, bool kBf16, Mode kMode>
struct ProductsQk {
  using C = Shape<D, kMode>;
  static constexpr uint32_t kId = idesc<kBf16 && kMode != kFp4>(kKeys, 0);
  Smem<D, kMode>& sm;
  const Params& p;
  uint32_t tmem, q0, k0;
  Ring<C::kStages> at;
  int done[2] = {0, 0};                        // tiles of each group so far
  __device__ __forceinline__ ProductsQk(Smem<D, kMode>& sm_, const Params& p_, uint32_t tmem_)
      : sm(sm_), p(p_), tmem(tmem_), q0(desc_lo(smem_u32(sm_.q), 16)), k0(desc_lo(smem_u32(sm_.ring), 16)) {}

  template <int g>
  __device__ __forceinline__ bool tile(int seg, bool last) {
    const int b = done[g] & 1;
    if (!wait2(sm, sm.pvdone[g][b], ((done[g] >> 1) & 1) ^ 1, sm.kfull[at.stage], at.phase, p)) return false;
    tc_fence_after();
    issue_qk<C::kChunks>(tmem + 256 + (2 * g + b) * kKeys, q0 + (seg & 1) * (C::kQTile >> 4),
                         k0 + at.stage * (2 * C::kTile >> 4), kId, smem_u32(&sm.sfull[g][b]),
                         smem_u32(&sm.kempty[at.stage]), smem_u32(&sm.qfree[seg & 1]), last);
    ++done[g];
    at.advance();
    return true;
  }

  __device__ __forceinline__ void run(Walk<kMode> w) {
    int seg = 0;
    Segment s;
    while (w.next(p, s)) {
      if (!wait(sm, sm.qfull, seg & 1, p)) return;
      for (int j = 0; j < s.n; j += 2) {
        if (!tile<0>(seg, j == s.n - 1)) return;
        if (j + 1 < s.n && !tile<1>(seg, j == s.n - 2)) return;
      }
      ++seg;
    }
  }
};

// Warp 3: O += P V of every tile.
template <int D, bool kBf16, Mode kMode>
struct ProductsPv {
  using C = Shape<D, kMode>;
  static constexpr uint32_t kId = idesc<kBf16 && kMode != kFp4>(D, 1);
  Smem<D, kMode>& sm;
  const Params& p;
  uint32_t tmem, v0;
  Ring<C::kStages> at;
  int done[2] = {0, 0};
  __device__ __forceinline__ ProductsPv(Smem<D, kMode>& sm_, const Params& p_, uint32_t tmem_)
      : sm(sm_), p(p_), tmem(tmem_), v0(desc_lo(smem_u32(sm_.ring) + C::kTile, kKeys * 128)) {}

  // `first`: the group's first of the segment, O starts at 0.
  template <int g>
  __device__ __forceinline__ bool tile(bool first, bool last) {
    const int b = done[g] & 1;
    if (!wait2(sm, sm.pfull[g][b], (done[g] >> 1) & 1, sm.vfull[at.stage], at.phase, p)) return false;
    tc_fence_after();
    issue_pv(tmem + g * D, tmem + 256 + (2 * g + b) * kKeys, v0 + at.stage * (2 * C::kTile >> 4), kId, first ? 0u : 1u,
             smem_u32(&sm.pvdone[g][b]), smem_u32(&sm.vempty[at.stage]), smem_u32(&sm.ofull), last);
    ++done[g];
    at.advance();
    return true;
  }

  __device__ __forceinline__ void run(Walk<kMode> w) {
    int seg = 0;
    Segment s;
    while (w.next(p, s)) {
      // The last segment's results have been read out of both accumulators.
      if (seg > 0 && !wait(sm, sm.ofree, (seg - 1) & 1, p)) return;
      for (int j = 0; j < s.n; j += 2) {
        if (!tile<0>(j == 0, j == s.n - 1)) return;
        if (j + 1 < s.n && !tile<1>(j == 0, j == s.n - 2)) return;
      }
      ++seg;
    }
  }
};

// ------------------------------------------------------------ softmax

// A warp's 32 rows of 64 bytes, one a lane, turned in `buf` (2 KB, 16-byte
// units XOR-swizzled by row pair) so that four lanes then write one row's 64
// bytes: row 8 i + lane / 4 to dst[i] (null: nothing), in units of 16 bytes.
// (Stored straight from the lanes' rows, every store touched 32 lines.)
__device__ __forceinline__ void store_rows(uint8_t* buf, const uint4* v, uint8_t* const* dst, int lane) {
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = v[e];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2);
    const uint4 x = *reinterpret_cast<const uint4*>(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
    if (dst[i] != nullptr) *reinterpret_cast<uint4*>(dst[i]) = x;
  }
}

// Starts the copies of a segment's Q rows into a swizzled tile, by all softmax
// warps: each group half the rows of each warp's 32.
template <int D, bool kBf16, Mode kMode>
__device__ __forceinline__ void start_q(Smem<D, kMode>& sm, const Params& p, const Segment& s, int seg, int g, int wq,
                                        int lane) {
  using C = Shape<D, kMode>;
  constexpr int kUnits = D / 8;                            // 16-byte units a row
  constexpr int kPer = 32 / kUnits;                        // rows a warp copies at once
  const int rows = rows_of_group(p, s.group);
  const int R = s.group * kRows + wq * 32 + lane;
  const int i = p.by_G.of(R);
  // Each lane knows its row's address; the lanes that copy a row ask for it.
  const long long base = wq * 32 + lane < rows ? s.b * p.q_stride[0] + i * p.q_stride[1] +
                                                     (s.head * p.G + (R - i * p.G)) * p.q_stride[2]
                                               : 0;
  const uint32_t tile = smem_u32(sm.q) + (seg & 1) * C::kQTile;
  const int r0 = g * 16 + lane / kUnits, u = lane % kUnits;
  if constexpr (kMode == kFp4 && kBf16) {
    // The products are fp16's (a code times its step is not always bf16's): a row's
    // largest magnitude is brought to 2^14 by a power of two, which leaves every
    // value down to 2^-28 of it as it is.
    uint4 v[16 / kPer];
#pragma unroll
    for (int e = 0; e < 16 / kPer; ++e) {
      const long long off = __shfl_sync(0xFFFFFFFFu, base, r0 + e * kPer);
      v[e] = wq * 32 + r0 + e * kPer < rows ? *reinterpret_cast<const uint4*>(p.q + off + u * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 16 / kPer; ++e) {
      const int row = wq * 32 + r0 + e * kPer;
      uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w}, top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
      top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
      for (int x = 1; x < kUnits; x <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      const int exponent = min(max(127 + 14 + 127 - static_cast<int>(top >> 7), 1), 253);   // of the power of two
      const float times = __uint_as_float(static_cast<uint32_t>(exponent) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack2<false>(bf16lo_to_f32(w[i]) * times, bf16hi_to_f32(w[i]) * times);
      *reinterpret_cast<uint4*>(sm.q + (seg & 1) * C::kQTile + (u >> 3) * (kRows * 128) + row * 128 +
                                (((u & 7) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      if (u == 0) sm.extra.q_unit[seg & 1][row] = __uint_as_float(static_cast<uint32_t>(254 - exponent) << 23);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16 / kPer; ++e) {
      const long long off = __shfl_sync(0xFFFFFFFFu, base, r0 + e * kPer);
      const int row = wq * 32 + r0 + e * kPer;
      if (row < rows)
        cp_async_16(tile + (u >> 3) * (kRows * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4), p.q + off + u * 16, true);
    }
    cp_async_commit();
  }
}
// The copies have landed: hands the tile to the products.
template <int D, Mode kMode>
__device__ __forceinline__ void finish_q(Smem<D, kMode>& sm, int lane) {
  cp_async_wait<0>();
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&sm.qfull));
}

// Warps 4..11: group g = 0, 1, warp wq of the group, one row a thread.
template <int D, bool kBf16, Mode kMode>
__device__ __forceinline__ void softmax(Smem<D, kMode>& sm, const Params& p, uint32_t tmem, Walk<kMode> w, int g, int wq,
                                        int lane) {
  using C = Shape<D, kMode>;
  // fp16 weights are kept 2^7 larger: the largest, 2^(8 + 7), is in range and
  // the smallest that is not rounded to a subnormal is 2^-14 / 2^7 of a row's
  // largest weight or more.  bf16 has fp32's range.
  constexpr bool kBf16P = kBf16 && kMode != kFp4;
  constexpr float kShift = kBf16P ? 0.f : 7.f;
  const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
  const int r = wq * 32 + lane;
  const uint32_t o_t = tmem + lanes + g * D;
  float a = p.scale_log2;
  const bool pos = a > 0.f;
  float a_eff = pos ? a : 1.f;
  int kt = 0, seg = 0, n = 0;                              // n: tiles of this group so far
  Segment s, next;
  bool more = w.next(p, s);
  if (more) {
    start_q<D, kBf16, kMode>(sm, p, s, 0, g, wq, lane);
    finish_q<D, kMode>(sm, lane);
  }
  for (; more; s = next) {
    more = w.next(p, next);
    if (more) {
      // The next segment's Q lands while this one's tiles are worked on.
      if (seg > 0 && !wait(sm, sm.qfree[(seg - 1) & 1], ((seg - 1) >> 1) & 1, p)) return;
      start_q<D, kBf16, kMode>(sm, p, next, seg + 1, g, wq, lane);
    }
    const int rows = rows_of_group(p, s.group);
    const int R = s.group * kRows + r;                     // row of the stream and head: draft * G + head in group
    const bool valid = r < rows;
    const bool warp_valid = wq * 32 < rows;
    const int i = p.by_G.of(R);
    const int head = s.head * p.G + (R - i * p.G);
    uint64_t mask64 = 0;
    uint32_t word = 0;
    if (p.q_len <= 32 && lane < p.q_len) word = p.mask[static_cast<size_t>(s.b) * p.q_len + lane];
    if (valid) {
      const int words = (p.q_len + 31) >> 5;
      const uint32_t* mrow = p.mask + (static_cast<size_t>(s.b) * p.q_len + i) * words;
      mask64 = mrow[0];
      if (words > 1) mask64 |= static_cast<uint64_t>(mrow[1]) << 32;
      if (p.q_len < 64) mask64 &= (1ull << p.q_len) - 1ull;
    }
    const int prefix = s.S - p.q_len;
    // With a window: prefix keys from `sinks` to `hide` are hidden from this row,
    // and of more drafts than the window holds the first ones that are no sinks.
    int hide = 0, hide_most = 0;
    if constexpr (kMode == kWindow) {
      const int n_seen = __popcll(mask64);
      hide = prefix - min(prefix, max(0, p.window - n_seen));
      hide_most = prefix - min(prefix, max(0, p.window - p.q_len));
      uint64_t last = mask64;
      for (int x = n_seen; x > p.window; --x) last &= last - 1ull;
      mask64 = last | (mask64 & between(prefix, 0, p.sinks));
    }
    if constexpr (kMode == kFp4 && kBf16) {
      if (!wait(sm, sm.qfull, seg & 1, p)) return;
      a = p.scale_log2 * sm.extra.q_unit[seg & 1][r];
      a_eff = pos ? a : 1.f;
    }
    float m = -CUDART_INF_F, l = 0.f;
    for (int j = g; j < s.n; j += 2, ++n) {
      const int buf = n & 1;
      const uint32_t s_t = tmem + lanes + 256 + (2 * g + buf) * kKeys;
      const int k0 = s.template key<kMode>(j);
      const bool edge = kMode == kWindow && k0 < hide_most && k0 + kKeys > p.sinks;   // some row's window starts here
      if (!wait(sm, sm.sfull[g][buf], (n >> 1) & 1, p)) return;
      if (warp_valid) {
        tc_fence_after();
        uint32_t sr[64];
        MLA_TMEM_LD_32x32b_X32(s_t, sr);
        MLA_TMEM_LD_32x32b_X32(s_t + 32, (sr + 32));
        tmem_ld_wait();
        if (!pos) {
#pragma unroll
          for (int c = 0; c < 64; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * a);
        }
        if (k0 + kKeys > prefix || edge) {
          uint64_t vis = kMode == kWindow && k0 + kKeys <= prefix ? ~0ull : visible(mask64, prefix - k0);
          if constexpr (kMode == kWindow) vis &= ~between(k0, p.sinks, hide);
          const uint32_t lo = static_cast<uint32_t>(vis), hi = static_cast<uint32_t>(vis >> 32);
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(((c < 32 ? lo : hi) >> (c & 31)) & 1u)) sr[c] = __float_as_uint(-CUDART_INF_F);
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(sr[e]);
#pragma unroll
        for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a_eff;
        const bool grow = mt > m + kLazy;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float alpha = grow ? ex2(m - mt) : 1.f;    // 0 when nothing was visible before
          if (grow) m = mt;
          l *= alpha;
          if (j > g) {
            // O holds tiles up to the previous one of this group, once its product is done.
            if (!wait(sm, sm.pvdone[g][(n - 1) & 1], ((n - 1) >> 1) & 1, p)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              MLA_TMEM_LD_32x32b_X32(o_t + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              MLA_TMEM_ST_32x32b_X32(o_t + c, o);
            }
          }
        }
        const float msub = m == -CUDART_INF_F ? 0.f : m - kShift;
        const uint64_t a2 = f2pack(a_eff, a_eff), m2 = f2pack(-msub, -msub);
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t pw[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x0, x1;
          f2unpack(ffma2(f2pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), a2, m2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          sum[c & 1] = fadd2(sum[c & 1], f2pack(p0, p1));
          pw[c] = pack2<kBf16P>(p0, p1);
        }
        MLA_TMEM_ST_32x32b_X32(s_t, pw);
        float s0, s1, s2, s3;
        f2unpack(sum[0], s0, s1);
        f2unpack(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tmem_st_wait();
        tc_fence_before();
      }
      if (k0 + kKeys > prefix || (kMode == kWindow && k0 < s.start && k0 + kKeys > p.sinks)) {
        // Rows past the stream, drafts that none sees (a batch padded to one q_len)
        // and keys in the gap may hold anything: P is 0 there, but 0 * NaN is not.
        uint64_t used = k0 + kKeys > prefix ? visible(seen_drafts(p, s.b, word, lane), prefix - k0) : ~0ull;
        if constexpr (kMode == kWindow) used &= ~between(k0, p.sinks, s.start);
        const uint32_t lo = static_cast<uint32_t>(used), hi = static_cast<uint32_t>(used >> 32);
        if ((lo & hi) != ~0u) {
          const int stage = (kt + j) % C::kStages;
          if (!wait(sm, sm.vfull[stage], ((kt + j) / C::kStages) & 1, p)) return;
          // Each thread one 16-byte column of every kRows / (D / 8)-th row.
          constexpr int kStep = kRows / (D / 8);
          const int u = r % (D / 8), row0 = r / (D / 8);
          uint8_t* const at = sm.ring + stage * 2 * C::kTile + C::kTile + (u >> 3) * (kKeys * 128) + (u & 7) * 16 + row0 * 128;
#pragma unroll
          for (int row = 0; row < kKeys; row += kStep)
            if (!(((row < 32 ? lo : hi) >> ((row & 31) + row0)) & 1u))
              *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.pfull[g][buf]));
    }

    // ---- end of the segment.  The next one's Q is handed over first: its
    // products then start while this one's results are written.
    if (more) {
      if (!wait(sm, sm.qfull, seg & 1, p)) return;         // (a group without a tile has not seen it)
      finish_q<D, kMode>(sm, lane);
    }
    const bool direct = s.n == s.nt;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (seg > 0 ? 1 : 0);
    const long long out_row = (static_cast<long long>(s.b) * p.q_len + i) * p.H + head;
    float m_off = m == -CUDART_INF_F ? -CUDART_INF_F : m - kShift;
    // The groups' accumulators: their weights, from both maxima and sums.  (Not
    // before the last segment's, in the same place, have been read.)
    if (seg > 0 && !wait(sm, sm.ofree, (seg - 1) & 1, p)) return;
    sm.ml[g][r] = make_float2(m_off, l);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.mlx));
    if (!wait(sm, sm.mlx, seg & 1, p)) return;
    const float2 ml0 = sm.ml[0][r], ml1 = sm.ml[1][r];
    m_off = fmaxf(ml0.x, ml1.x);
    float w0 = ml0.x == -CUDART_INF_F ? 0.f : ex2(ml0.x - m_off);
    float w1 = ml1.x == -CUDART_INF_F ? 0.f : ex2(ml1.x - m_off);
    l = w0 * ml0.y + w1 * ml1.y;
    if (!wait(sm, sm.ofull, seg & 1, p)) return;
    if (warp_valid) {
      tc_fence_after();
      if (direct) {
        const float inv = l == 0.f ? 0.f : 1.f / l;        // (a NaN stays one)
        w0 *= inv;
        w1 *= inv;
      }
      if constexpr (kMode == kFp4) {
        w0 *= p.v_factor;
        w1 *= p.v_factor;
      }
      const int c0 = g * (D / 2), c1 = c0 + D / 2;         // each group writes half the columns
      // The products are through with this segment's Q: the first 2 KB of the
      // rows that this warp itself copies are free to turn the results in.
      uint8_t* const buf = sm.q + (seg & 1) * C::kQTile + (wq * 32 + g * 16) * 128;
      uint8_t* dst[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 8 * e + (lane >> 2);
        const long long orow = __shfl_sync(0xFFFFFFFFu, out_row, row);
        const size_t part_row = static_cast<size_t>(slot) * p.part_rows + wq * 32 + row;
        uint8_t* const to = direct ? static_cast<uint8_t*>(p.out) + (orow * D + c0) * 2
                                   : reinterpret_cast<uint8_t*>(p.part_o + part_row * (D / 4) + c0 / 4);
        dst[e] = wq * 32 + row < rows ? to + (lane & 3) * 16 : nullptr;
      }
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t x0[32];
        float o[32];
        MLA_TMEM_LD_32x32b_X32(tmem + lanes + c, x0);
        if (s.n > 1) {
          uint32_t x1[32];
          MLA_TMEM_LD_32x32b_X32(tmem + lanes + D + c, x1);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = w0 * __uint_as_float(x0[e]) + w1 * __uint_as_float(x1[e]);
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = w0 * __uint_as_float(x0[e]);
        }
        uint4 v[4];
        if (direct) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = make_uint4(pack2<kBf16>(o[8 * e], o[8 * e + 1]), pack2<kBf16>(o[8 * e + 2], o[8 * e + 3]),
                              pack2<kBf16>(o[8 * e + 4], o[8 * e + 5]), pack2<kBf16>(o[8 * e + 6], o[8 * e + 7]));
          store_rows(buf, v, dst, lane);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = make_uint4(__float_as_uint(o[16 * h + 4 * e]), __float_as_uint(o[16 * h + 4 * e + 1]),
                                __float_as_uint(o[16 * h + 4 * e + 2]), __float_as_uint(o[16 * h + 4 * e + 3]));
            store_rows(buf, v, dst, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (h == 0 && dst[e] != nullptr) dst[e] += 64;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (dst[e] != nullptr) dst[e] += 64;
      }
      if (valid && g == 0) {
        if (direct)
          p.lse[out_row] = l == 0.f ? -CUDART_INF_F : (m_off + log2f(l)) * 0.6931471805599453f;
        else
          p.part_ml[static_cast<size_t>(slot) * p.part_rows + r] = make_float2(m_off, l);
      }
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.ofree));
    kt += s.n;
    ++seg;
  }
}

// ------------------------------------------------------------ kernel

// This warp's products are done (or its CTA may not end).
__device__ __forceinline__ void drain_products(uint64_t& bar) {
  mma_commit_elect(smem_u32(&bar));
  mbar_wait(smem_u32(&bar), 0, kWaitNs);
  __syncwarp();
}

// Tells the merge about the units that start in this CTA's run: a cut one goes
// on in the teams after this one (parts > 0), a whole one is none of its
// business (0).  With p.desc_units there is an entry a unit, else one a CTA, for
// the only unit that can be cut, its last.  Written before the first wait, so
// that the merge finds it whatever becomes of the loads.
template <Mode kMode>
__device__ __forceinline__ void note_cut_units(const Params& p, Walk<kMode> w, const Runs& runs) {
  const int cta = static_cast<int>(blockIdx.x);
  int4 d = make_int4(0, 0, 0, 0);
  Segment s;
  for (int seg = 0; w.next(p, s); ++seg) {
    if (s.tile0 != 0) continue;
    const int hg = s.head * p.groups + s.group;
    if (s.n < s.nt) {
      const int last = runs.team_of(w.t1 - s.n + s.nt - 1);   // the team that has the unit's last tile
      d = make_int4(s.b, hg, 2 * cta + (seg > 0 ? 1 : 0), last - p.by_members.of(cta) + 1);
    }
    if (p.desc_units) p.desc[s.b * p.Hkv * p.groups + hg] = d;
  }
  if (!p.desc_units) p.desc[cta] = d;
}

template <int D, bool kBf16, Mode kMode>
__device__ __forceinline__ void run_cta(const CUtensorMap* map_k, const CUtensorMap* map_v, const Fp4Maps* maps, const Params& p) {
  using S = Smem<D, kMode>;
  using C = Shape<D, kMode>;
  constexpr int kThreads = C::kThreads;
  // Shared memory is full to the last KB: the tiles' alignment is asked for, and
  // checked, instead of made with a spare KB.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  if (smem_u32(smem_raw) & 1023) {
    grid_dependency_wait();
    if (threadIdx.x == 0) {
      atomicOr(p.status, kBitTimeout);
      p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);          // (an entry a unit: there are no more than CTAs)
    }
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 3) {
    const uint32_t loaders = kMode == kFp4 || p.box_rows ? 1 : 32;
    for (int i = lane; i < C::kStages; i += 32) {
      mbar_init(smem_u32(&sm.kfull[i]), loaders);
      mbar_init(smem_u32(&sm.vfull[i]), loaders);
      mbar_init(smem_u32(&sm.kempty[i]), 1);
      mbar_init(smem_u32(&sm.vempty[i]), 1);
    }
    if (lane >= 16 && lane < 20) {
      const int g = (lane >> 1) & 1, i = lane & 1;
      mbar_init(smem_u32(&sm.sfull[g][i]), 1);
      mbar_init(smem_u32(&sm.pfull[g][i]), 4);
      mbar_init(smem_u32(&sm.pvdone[g][i]), 1);
    }
    if (lane == 20) {
      mbar_init(smem_u32(&sm.qfull), 8);
      mbar_init(smem_u32(&sm.qfree[0]), 1);
      mbar_init(smem_u32(&sm.qfree[1]), 1);
    }
    if (lane == 21) {
      mbar_init(smem_u32(&sm.ofull), 1);
      mbar_init(smem_u32(&sm.ofree), 8);
      mbar_init(smem_u32(&sm.mlx), 8);
    }
    if constexpr (kMode == kFp4) {
      for (int i = lane; i < 2 * C::kPacked; i += 32) {
        mbar_init(smem_u32(&sm.extra.packed_full[0][i]), p.box_rows ? 1 : 32);
        mbar_init(smem_u32(&sm.extra.packed_empty[0][i]), 1);
      }
    }
    if (lane == 22) {
      mbar_init(smem_u32(&sm.drain[0]), 1);
      mbar_init(smem_u32(&sm.drain[1]), 1);
      sm.abort_flag = 0;
    }
    fence_mbarrier_init_cluster();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  if (kMode != kFp4 && tid == 0 && p.box_rows) {
    tma_prefetch_desc(map_k);
    tma_prefetch_desc(map_v);
  }
  grid_dependency_wait();                                  // nothing of the caller's was touched so far
  if (tid == 0) grid_launch_dependents();

  // ---- this CTA's run of work: it starts in stream `start_b`, before which
  // lie `start_pre` tiles (or units).
  const int units = p.head_sets * p.group_sets;
  const int all = p.by_members.of(gridDim.x), team = p.by_members.of(blockIdx.x);
  const int member = static_cast<int>(blockIdx.x) - team * p.members;
  int len, total, start_b = 0, start_pre = 0;
  if (p.B <= 32) {
    // Every warp by itself, a stream a lane.
    int work = 0;
    if (lane < p.B) {
      work = stream_work(p, stream_tiles<kMode>(p, lane, len)) * units;
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
    // Each thread sums a run of streams, then a scan over threads; the thread
    // whose streams hold the first tile says which.
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int sum = 0;
    bool off = false;                  // (reported after the loop: an atomic in it would hold up the next loads)
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      sum += stream_work(p, stream_tiles<kMode>(p, b, len)) * units;
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
        const int n = stream_work(p, stream_tiles<kMode>(p, b, len)) * units;
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
  const Walk<kMode> walk(p, member, t0, team < runs.teams ? runs.start(team + 1) : total, start_b, start_pre);

  if constexpr (kMode == kFp4) {
    // 512 threads of 128 registers: the softmax warps take 168, the others 88.
    if (warp >= 4 && warp < 12) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      softmax<D, kBf16, kMode>(sm, p, tmem, walk, (warp - 4) >> 2, warp & 3, lane);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      if (warp >= 12) {
        unpack_tiles<D>(sm, p, walk, warp >= 14, warp & 1);
      } else if (warp == 0 || warp == 2) {
        if (p.box_rows == 0) load_packed_rows<D>(sm, p, walk, warp == 2);
        else load_packed_boxes<D>(sm, p, *maps, walk, warp == 2);
      } else if (warp == 1) {
        ProductsQk<D, kBf16, kMode>(sm, p, tmem).run(walk);
        drain_products(sm.drain[0]);
      } else {
        if (lane == 0 && !p.whole) note_cut_units(p, walk, runs);
        __syncwarp();
        ProductsPv<D, kBf16, kMode>(sm, p, tmem).run(walk);
        drain_products(sm.drain[1]);
      }
    }
  } else if (warp == 0 || warp == 2) {
    if (p.box_rows == 0) load_gather<D, kMode>(sm, p, walk, warp == 2);
    else load_tma<D, kMode>(sm, p, warp == 2 ? map_v : map_k, walk, warp == 2);
  } else if (warp == 1) {
    ProductsQk<D, kBf16, kMode>(sm, p, tmem).run(walk);
    drain_products(sm.drain[0]);
  } else if (warp == 3) {
    if (lane == 0 && !p.whole) note_cut_units(p, walk, runs);
    __syncwarp();
    ProductsPv<D, kBf16, kMode>(sm, p, tmem).run(walk);
    drain_products(sm.drain[1]);
  } else if (warp >= 4) {
    softmax<D, kBf16, kMode>(sm, p, tmem, walk, (warp - 4) >> 2, warp & 3, lane);
  }
  // Streams without keys.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (stream_tiles<kMode>(p, b, len) != 0) continue;
    if (p.desc_units && !p.whole)
      for (int u = tid; u < p.Hkv * p.groups; u += kThreads) p.desc[b * p.Hkv * p.groups + u] = make_int4(0, 0, 0, 0);
    const long long rows = static_cast<long long>(p.q_len) * p.H;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + b * rows * (D * 2));
    for (long long x = tid; x < rows * (D / 8); x += kThreads) o[x] = make_uint4(0, 0, 0, 0);
    for (long long x = tid; x < rows; x += kThreads) p.lse[b * rows + x] = -CUDART_INF_F;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBf16, Mode kMode>
__global__ void __launch_bounds__(Shape<D, kMode>::kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params p) {
  run_cta<D, kBf16, kMode>(&map_k, &map_v, nullptr, p);
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(Shape<D, kFp4>::kThreads, 1) attn_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Params p) {
  run_cta<D, kBf16, kFp4>(nullptr, nullptr, &maps, p);
}

// Merges the partials of the cut units.  A unit's parts are the first one's slot
// and the first slots of the same member of the teams after it.  A block takes
// kR rows of a unit; kP part groups of threads share the parts, a thread one
// row's four columns of several parts at a time (weights, sums and values loaded
// together), and the groups' results are put together through shared memory.
// Everything is added in a fixed order.  The call is a chain of a few reads
// that depend on each other (~1.5 us after the split kernel has ended), so there
// is as little else in it as there can be.  Two shapes:
//   few units, many parts: two rows and four part groups; block (x, y) takes
//     chunk x of the unit of entry y;
//   many units, few parts: one part group; every block first lists the cut units
//     (all entries read at once) and takes chunks of them in turn (a block a chunk
//     and entry were 9,728 that mostly found nothing to do).  With no more chunks
//     than blocks at a time a chunk is eight rows and a thread loads eight parts
//     at once (264 rows over 16k keys 32.6 -> 31.9 us against four).  With more,
//     what counts are blocks an SM and instructions a byte: three parts at once,
//     and sixteen rows with eight columns a thread (1,024 rows in two parts each:
//     48.7 us; four columns 50.3; and four parts at once 51.0, eight 53.6).
constexpr int kMaxParts = 320;               // CTAs of the split kernel at most
constexpr int kMergeUnits = 8;               // rows x part groups of a block, four columns a thread
constexpr int kMergeParts = 4;               // part groups when there are many parts
// kAtOnce: parts a thread loads at once; kV: its columns, in fours, D / kV apart.
template <int D, bool kBf16, int kP, int kAtOnce, int kV>
__device__ __forceinline__ void merge_rows(const Params& p, const int4 d, int chunk) {
  constexpr int kLanes = D / 4 / kV;                       // threads a row
  constexpr int kR = kMergeUnits * kV / kP;
  constexpr int kGroup = kLanes * kR;                      // threads a part group
  __shared__ float4 sums[kP > 1 ? kP - 1 : 1][kV][kGroup];
  __shared__ float2 stats[kP > 1 ? kP - 1 : 1][kR];
  const int tid = threadIdx.x, c4 = tid % kLanes, r = tid / kLanes % kR, group = tid / kGroup, t = tid % kGroup;
  const int parts = d.w, rr = chunk * kR + r;
  const int head = d.y / p.groups, R = (d.y - head * p.groups) * kRows + rr;
  const bool valid = rr < kRows && R < p.q_len * p.G;
  // Row rr of part k >= 1 lies in slot 2 * (CTA of part 0 + k * members).
  const size_t row_k = static_cast<size_t>(2 * (d.z >> 1)) * p.part_rows + rr;
  const size_t row_0 = static_cast<size_t>(d.z) * p.part_rows + rr;
  const size_t step = static_cast<size_t>(2 * p.members) * p.part_rows;
  float4 o[kV] = {};
  float m = -CUDART_INF_F, l = 0.f;
  auto scale = [&](float keep) {
    l *= keep;
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = make_float4(o[v].x * keep, o[v].y * keep, o[v].z * keep, o[v].w * keep);
  };
  auto add = [&](float w, const float4& x, int v) {
    o[v].x += w * x.x;
    o[v].y += w * x.y;
    o[v].z += w * x.z;
    o[v].w += w * x.w;
  };
  for (int k0 = group; valid && k0 < parts; k0 += kAtOnce * kP) {
    float4 x[kAtOnce][kV] = {};
    float2 y[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int k = k0 + e * kP;
      y[e] = make_float2(-CUDART_INF_F, 0.f);
      if (k < parts) {
        const size_t row = k ? row_k + k * step : row_0;
        y[e] = __ldcg(p.part_ml + row);
#pragma unroll
        for (int v = 0; v < kV; ++v) x[e][v] = __ldcg(p.part_o + row * (D / 4) + v * kLanes + c4);
      }
    }
    float top = m;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) top = fmaxf(top, y[e].x);
    scale(m == -CUDART_INF_F ? 0.f : ex2(m - top));
    m = top;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const float w = y[e].x == -CUDART_INF_F ? 0.f : ex2(y[e].x - m);
      l += w * y[e].y;
#pragma unroll
      for (int v = 0; v < kV; ++v) add(w, x[e][v], v);
    }
  }
  if (kP > 1) {
    if (group) {
#pragma unroll
      for (int v = 0; v < kV; ++v) sums[group - 1][v][t] = o[v];
      if (c4 == 0) stats[group - 1][r] = make_float2(m, l);
    }
    __syncthreads();
    if (group) return;
    float top = m;
#pragma unroll
    for (int g = 0; g < kP - 1; ++g) top = fmaxf(top, stats[g][r].x);
    scale(m == -CUDART_INF_F ? 0.f : ex2(m - top));
    m = top;
#pragma unroll
    for (int g = 0; g < kP - 1; ++g) {
      const float2 y = stats[g][r];
      const float w = y.x == -CUDART_INF_F ? 0.f : ex2(y.x - m);
      l += w * y.y;
#pragma unroll
      for (int v = 0; v < kV; ++v) add(w, sums[g][v][t], v);
    }
  }
  if (!valid) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;              // (a NaN stays one)
  const int i = p.by_G.of(R);
  const long long row = (static_cast<long long>(d.x) * p.q_len + i) * p.H + head * p.G + (R - i * p.G);
#pragma unroll
  for (int v = 0; v < kV; ++v)
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * (D * 2))[v * kLanes + c4] =
        make_uint2(pack2<kBf16>(o[v].x * inv, o[v].y * inv), pack2<kBf16>(o[v].z * inv, o[v].w * inv));
  if (c4 == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(D / 4 * kMergeUnits) combine_many_parts(const Params p, int) {
  grid_dependency_wait();
  const int4 d = __ldcg(p.desc + blockIdx.y);
  if (d.w != 0) merge_rows<D, kBf16, kMergeParts, 8, 1>(p, d, blockIdx.x);
}

template <int D, bool kBf16, int kAtOnce, int kV>
__global__ void __launch_bounds__(D / 4 * kMergeUnits) combine_many_units(const Params p, int entries) {
  static_assert(kMergeUnits * kV <= 16, "a partial's rows are a multiple of 16");
  constexpr int kThreadsM = D / 4 * kMergeUnits, kWarps = kThreadsM / 32;
  __shared__ int4 cut[kMaxParts];
  __shared__ int warp_cut[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5;
  grid_dependency_wait();
  int n_cut = 0;
  for (int base = 0; base < entries; base += kThreadsM) {
    const int4 d = base + tid < entries ? __ldcg(p.desc + base + tid) : make_int4(0, 0, 0, 0);
    const unsigned ballot = __ballot_sync(0xFFFFFFFFu, d.w != 0);
    if ((tid & 31) == 0) warp_cut[warp] = __popc(ballot);
    __syncthreads();
    int at = n_cut;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp && d.w != 0) cut[at + __popc(ballot & ((1u << (tid & 31)) - 1u))] = d;
      at += warp_cut[w];
    }
    n_cut = at;
    __syncthreads();
  }
  const int chunks = p.part_rows / (kMergeUnits * kV);
  for (int item = blockIdx.x; item < n_cut * chunks; item += gridDim.x) {
    const int u = item / chunks;
    merge_rows<D, kBf16, 1, kAtOnce, kV>(p, cut[u], item - u * chunks);
  }
}

}  // namespace gqa
}  // namespace mla
