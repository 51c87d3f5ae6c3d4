// Attention over a cache held in 4 bits for few query rows a key head (decoding, short
// drafts): the other kernel behind mla_gqa_verify_attn_fp4_paged.
//
// Mathematics.  That of the attention kernel (gqa_attn.cuh), turned around: S^T = K Q^T
// and O^T = V^T P with the keys, then the dimensions, as the 16 rows of a warp's
// mma.sync and 8 query rows as its columns, so that 8 rows cost a sixteenth of the 128
// that a tcgen05 product has.  Codes become fp16 in the registers of the lanes that
// feed the product: nothing is written back to shared memory.
//   K: lane 4 g + c holds keys g and g + 8 of 16, and a contiguous quarter c of their
//      dimensions: 16 bytes (8 at D = 64).  The order of the dimensions in a
//      product is free if Q has the same: a lane's quarter of a row of Q as it lies.
//   V: lane 4 g + c holds dimensions 16 g .. 16 g + 15 (8 at D = 64) of keys 2 c, 2 c + 1,
//      2 c + 8, 2 c + 9; the halves of two keys' bytes are interleaved before they
//      are converted, so that a pair of keys lies in a register as the product wants.
// S^T's layout is P's but for a transpose of 8 x 8 (movmatrix).  The keys' order in
// shared memory is permuted (`order`) so that K's and V's reads collide as little as the
// rows' pitch allows.
//
// What bounds it: 1,152 bytes a key of 8 heads at D = 128, 23 bytes a cycle and SM, and as
// much the instructions: 268 a warp for 16 keys of a head and eight rows (70 conversions,
// 64 fp16 products, 16 mma.sync), 1.6 a cycle and SM with two warps a scheduler.  A fifth
// of the stalls are instruction fetch: the body stands twice (with and without hidden
// keys), each time unrolled over 32 keys.  Spills: 52 bytes stored, 108 loaded with 25 to
// 32 rows at D = 128, 8 and 52 with 9 to 16 at D = 64, none in the other forms.
// Measured (GPU time, bf16, D = 128, 64 streams of 1k to 32k keys, 8 key heads, 16-row
// pages): one token of 8 heads a key head 134 us, 5.0 TB/s (74 % of the measured copy
// rate); 2, 3, 4 tokens 174, 227, 285 us.
//
// Split.  Equal runs of 64-key tiles as in the attention kernel, but a CTA takes all (up
// to eight) key heads of a run: whole rows of the cache come in by TMA boxes of eight rows
// or more (a bulk copy a row took 64 cycles each, 2.6 TB/s in all; boxes of eight 7.1),
// or, where pages are not a multiple of eight rows, by four warps' 16-byte copies.
// Eight other warps are shared out among the heads; those of one head take 16 or 32 keys
// in turn and are put together at a unit's end.  (16 warps of 16 keys: 173 us against
// 150, for registers and instructions; 12 warps on four heads 181.)  The heads of a CTA
// count as a team's members for the merge.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "gqa_attn.cuh"
#include "gqa_host.h"
#include "mla_verify_attn.h"

namespace mla {
namespace gqa {
namespace few {

constexpr int kMostStages = 8;
constexpr int kLoaders = 4;                // warps that load

struct FewParams : Params {
  int heads, head_warps;           // key heads a CTA, warps a head
  // A stage: stage_keys rows of K, then of V (stage_bytes / 2 behind).  Whole rows where a CTA
  // has all heads; else (split) the heads' codes, then their steps, which begin at a
  // multiple of 16 bytes.
  int stage_keys, stages, stage_bytes, split;
  int code_pitch, step_pitch;      // bytes between rows
  int code_bytes, step_bytes;      // copied of a row (step_bytes: split)
  int row_end;                     // bytes of a pool row
  uint32_t order;                  // key of row i of 8, four bits each
  Divisor by_units;                // 16-byte units of a row
};

// kN: query rows in eights; with more of them a warp takes fewer keys at a time.
constexpr int kWarps = 8;
template <int kN>
struct Shape8 {
  static constexpr int kThreads = 32 * (kWarps + kLoaders);
  static constexpr int kTogether = kN <= 2 ? 2 : 1;        // sixteens of keys
  // 384 threads of 168 registers: with more rows the loaders leave some to the others,
  static constexpr int kMore = kN > 1 ? 224 : 0, kLess = 56;
  // and Q stays in shared memory, in the order in which a warp's lanes take it.
  static constexpr bool kSharedQ = kN >= 3;
};

// A warp's place in its run, kept in shared memory between the ends of segments: the
// stages want all registers.
struct Place {
  Walk<kWhole> walk;
  Segment s;
  int seg;
};

template <int kN>
struct __align__(128) Head {
  uint64_t full[kMostStages], empty[kMostStages], meet[kWarps];
  float2 ml[kWarps][8 * kN];
  Place place[kWarps];
  uint64_t mask[kWarps][8 * kN + 1];       // what each row's draft sees of the drafts; all of them
  int warp_sum[kWarps + kLoaders], start_b, start_pre;
  uint32_t abort_flag;
};

}  // namespace few
template <int kN>
struct InlineWaits<few::Head<kN>> {
  static constexpr bool value = true;
};
namespace few {

template <int D>
constexpr int kSumPitch = D + 4;           // floats a row of the warps' sums
template <int D, int kN>
constexpr int kQBytes = Shape8<kN>::kSharedQ ? kWarps * kN * 32 * (D / 2) : 0;
template <int D>
constexpr int kSums = kWarps * 8 * kSumPitch<D> * 4;

__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at));
  return r;
}
// kWords 32-bit words.
template <int kWords>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* w) {
  if constexpr (kWords == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (kWords == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t low2(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t x) { return __byte_perm(x, x, 0x3232); }

struct Maps {
  CUtensorMap codes[2], steps[2];            // of K and V
};

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
               : "memory");
}

// The first loader: a box of K and one of V a lane.
template <int kN>
__device__ __forceinline__ void load_boxes(Head<kN>& sm, const FewParams& p, const Maps& maps, uint32_t ring, int each, Walk<kWhole> w) {
  const int lane = threadIdx.x & 31, R = p.box_rows;
  int stage = 0, issued = 0;
  uint32_t phase = 0;
  Segment s;
  while (w.next(p, s)) {
    const int begin = s.tile0 * kKeys, end = min(s.S, (s.tile0 + s.n) * kKeys);
    const int code_x = p.split ? s.head * each : 0;                          // in 8 bytes
    const int step_x = (p.steps_at + ((s.head * each) & ~15)) >> 3;
    auto entry_of = [&](int k0) {
      const int key = k0 + lane * R;
      return lane * R < p.stage_keys && key < end ? table_entry(p, s.b, key) : 0;
    };
    int next = entry_of(begin);
    for (int k0 = begin; k0 < end; k0 += p.stage_keys) {
      const int n = (min(p.stage_keys, end - k0) + R - 1) / R;               // boxes
      const int row = lane < n ? pool_row(p, next, k0 + lane * R) : 0;
      next = entry_of(k0 + p.stage_keys);
      if (!wait(sm, sm.empty[stage], phase ^ 1, p)) goto out;
      const uint32_t bar = smem_u32(&sm.full[stage]);
      if (p.test_stall && blockIdx.x == 0 && issued == 0) goto out;          // this load never comes
      if (lane == 0) mbar_arrive_expect_tx(bar, 2 * n * R * (p.code_bytes + p.step_bytes));
      __syncwarp();
      if (lane < n) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t dst = ring + stage * p.stage_bytes + v * (p.stage_bytes >> 1);
          tma_box(dst + lane * R * p.code_pitch, &maps.codes[v], code_x, row, bar);
          if (p.split)
            tma_box(dst + p.stage_keys * p.code_pitch + lane * R * p.step_pitch, &maps.steps[v], step_x, row, bar);
        }
      }
      ++issued;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
out:
  for (int n = issued - 1; n >= 0 && n >= issued - p.stages; --n)
    mbar_wait(smem_u32(&sm.full[n % p.stages]), (n / p.stages) & 1, kWaitNs / 2);
}

// All loaders where no box fits the pages: a quarter of a stage's rows each, 16 bytes a lane.
template <int kN>
__device__ __forceinline__ void load_rows(Head<kN>& sm, const FewParams& p, uint32_t ring, int each, Walk<kWhole> w, int loader) {
  const int lane = threadIdx.x & 31, units = static_cast<int>(p.by_units.d), code_units = p.code_bytes >> 4;
  const int keys = p.stage_keys / kLoaders, first = loader * keys;           // (no more than 64)
  int stage = 0;
  uint32_t phase = 0;
  Segment s;
  while (w.next(p, s)) {
    const int begin = s.tile0 * kKeys, end = min(s.S, (s.tile0 + s.n) * kKeys);
    const int code_at = p.split ? s.head * each * 8 : 0, step_at = p.steps_at + ((s.head * each) & ~15);
    auto entry_of = [&](int k0, int h) {
      const int r = h * 32 + lane, key = k0 + first + r;
      return r < keys && key < end ? table_entry(p, s.b, key) : 0;
    };
    int next[2] = {entry_of(begin, 0), entry_of(begin, 1)};
    for (int k0 = begin; k0 < end; k0 += p.stage_keys) {
      const int n = min(keys, end - k0 - first);                             // rows (none: negative)
      int row[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row[h] = h * 32 + lane < n ? pool_row(p, next[h], k0 + first + h * 32 + lane) : 0;
        next[h] = entry_of(k0 + p.stage_keys, h);
      }
      if (!wait(sm, sm.empty[stage], phase ^ 1, p)) goto out;
      const uint32_t dst = ring + stage * p.stage_bytes;
      for (int x = lane; x - lane < n * units; x += 32) {
        const int r = p.by_units.of(x), u = x - r * units;
        const int lo = __shfl_sync(0xFFFFFFFFu, row[0], r & 31), hi = __shfl_sync(0xFFFFFFFFu, row[1], r & 31);
        if (x >= n * units) continue;
        const long long at = r < 32 ? lo : hi;
        const int key = first + r;
        const bool step = u >= code_units;
        // (Of a split row's steps, those behind the row's end are not there.)
        const int from = step ? step_at + (u - code_units) * 16 : code_at + u * 16;
        const uint32_t to = dst + (step ? p.stage_keys * p.code_pitch + key * p.step_pitch + (u - code_units) * 16
                                        : key * p.code_pitch + u * 16);
        const bool there = !step || from < p.row_end;
        cp_async_16(to, p.k + at * p.k_stride[1] + (there ? from : 0), there);
        cp_async_16(to + (p.stage_bytes >> 1), p.v + at * p.v_stride[1] + (there ? from : 0), there);
      }
      if (!(p.test_stall && blockIdx.x == 0))
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.full[stage])) : "memory");
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
out:
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// All warps of a head are here; false: some wait has run out.
template <int kN>
__device__ __forceinline__ bool meet(Head<kN>& sm, const FewParams& p, int head, uint32_t& times) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.meet[head]));
  return wait(sm, sm.meet[head], times++ & 1u, p);
}

// The drafts that draft i of stream b sees.
__device__ __forceinline__ uint64_t mask_of(const Params& p, int b, int i) {
  const int words = (p.q_len + 31) >> 5;
  const uint32_t* const row = p.mask + (static_cast<size_t>(b) * p.q_len + i) * words;
  uint64_t m = row[0];
  if (words > 1) m |= static_cast<uint64_t>(row[1]) << 32;
  return m;
}
// Whether a key of the run is one that drafts with this mask see.
__device__ __forceinline__ bool among(uint64_t mask, int key, int prefix, int end) {
  return key < end && (key < prefix || (mask >> (key - prefix) & 1ull));
}

template <int D, bool kBf16, int kN>
__device__ __forceinline__ void attend(Head<kN>& sm, const FewParams& p, uint8_t* shared_q, uint32_t ring, float* sums, int warp,
                                       int lane) {
  constexpr int kTiles = D / 16;             // of 16 dimensions (or rows of O^T)
  constexpr int kQ = D / 8;                  // registers of a row of Q a lane
  constexpr int kS = Shape8<kN>::kTogether;
  constexpr bool kTwo = kN <= 2;
  constexpr float kShift = 7.f;              // (see the attention kernel's softmax)
  constexpr float kNothing = -FLT_MAX;       // no score is smaller
  const int g = lane >> 2, c = lane & 3;
  const int head_local = warp / p.head_warps, j = warp - head_local * p.head_warps;
  const int rows = p.q_len * p.G;
  const bool several = kN == 1 && p.head_warps > 1;        // warps of a head (more rows: always one, see few_rows)
  const int key_g = p.order >> (4 * g) & 7, key_c = p.order >> (8 * c) & 7, key_c1 = p.order >> (8 * c + 4) & 7;
  // Where this lane reads, from a stage's start and of the first 16 keys: K's codes (and
  // their steps, from where the head's steps are), the same of V, and from there to
  // the second key's.
  const int k_codes = key_g * p.code_pitch + head_local * (D / 2) + c * (D / 8), k_steps = key_g * p.step_pitch + c * (D / 64);
  const int v_codes = (p.stage_bytes >> 1) + key_c * p.code_pitch + head_local * (D / 2) + g * (D / 16);
  const int v_steps = (p.stage_bytes >> 1) + key_c * p.step_pitch + (D == 128 ? g : g >> 1);
  int stage = 0;
  uint32_t phase = 0, met = 0;
  while (true) {
    Segment s;
    {
      Walk<kWhole> w = sm.place[warp].walk;
      if (!w.next(p, s)) return;
      __syncwarp();
      if (lane == 0) {
        sm.place[warp].walk = w;
        sm.place[warp].s = s;
        ++sm.place[warp].seg;
      }
    }
    const int begin = s.tile0 * kKeys, end = min(s.S, (s.tile0 + s.n) * kKeys), prefix = s.S - p.q_len;
    if (end > prefix) {
      const uint64_t used =
          seen_drafts(p, s.b, p.q_len <= 32 && lane < p.q_len ? p.mask[static_cast<size_t>(s.b) * p.q_len + lane] : 0u, lane);
      if (lane == 0) sm.mask[warp][8 * kN] = used;
      if (lane < 8 * kN) sm.mask[warp][lane] = mask_of(p, s.b, p.by_G.of(min(lane, rows - 1)));   // (rows past the last: its)
      __syncwarp();
    }
    // ---- rows of Q: row 8 t + g, this lane's quarter; in fp16, brought to its range
    // by a power of two where they are bf16.
    constexpr bool kSharedQ = Shape8<kN>::kSharedQ;
    uint4* const q_at = reinterpret_cast<uint4*>(shared_q) + warp * kN * (kQ / 4) * 32 + lane;
    uint32_t q[kSharedQ ? 1 : kN][kQ];
    float a[kN][2];                          // scale of rows 8 t + 2 c, + 1
    // ms: what a row's exponents are taken off, its maximum less kShift; kNothing
    // until it has seen a key.
    float ms[kN][2], l[kN][2], o[kN][kTiles][4];
#pragma unroll
    for (int t = 0; t < kN; ++t) {
      const int R = 8 * t + g, i = p.by_G.of(R);
      float unit = 1.f;
      const uint8_t* const src =
          p.q + s.b * p.q_stride[0] + i * p.q_stride[1] + ((s.head + head_local) * p.G + (R - i * p.G)) * p.q_stride[2] + c * (D / 2);
      uint32_t* const q_t = q[kSharedQ ? 0 : t];
#pragma unroll
      for (int e = 0; e < kQ / 4; ++e) {
        const uint4 x = R < rows ? reinterpret_cast<const uint4*>(src)[e] : make_uint4(0, 0, 0, 0);
        q_t[4 * e] = x.x;
        q_t[4 * e + 1] = x.y;
        q_t[4 * e + 2] = x.z;
        q_t[4 * e + 3] = x.w;
      }
      if (kBf16) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kQ; ++e) top = __vmaxu2(top, q_t[e] & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int exponent = min(max(127 + 14 + 127 - static_cast<int>(top >> 7), 1), 253);
        const float by = __uint_as_float(static_cast<uint32_t>(exponent) << 23);
        unit = __uint_as_float(static_cast<uint32_t>(254 - exponent) << 23);
#pragma unroll
        for (int e = 0; e < kQ; ++e) q_t[e] = pack2<false>(bf16lo_to_f32(q_t[e]) * by, bf16hi_to_f32(q_t[e]) * by);
      }
      if constexpr (kSharedQ) {
#pragma unroll
        for (int e = 0; e < kQ / 4; ++e)
          q_at[(t * (kQ / 4) + e) * 32] = make_uint4(q_t[4 * e], q_t[4 * e + 1], q_t[4 * e + 2], q_t[4 * e + 3]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        a[t][e] = p.scale_log2 * __shfl_sync(0xFFFFFFFFu, unit, (2 * c + e) * 4);
        ms[t][e] = kNothing;
        l[t][e] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][x][e] = 0.f;
    }
    // Of the stage's row 0: this head's steps.
    const int steps_at = (p.split ? p.stage_keys * p.code_pitch + ((s.head * (D / 16)) & 15) : p.steps_at) + head_local * (D / 16);

    // ---- the run's stages
    const int code_next = (key_c1 - key_c) * p.code_pitch, step_next = (key_c1 - key_c) * p.step_pitch;
    auto keys = [&](auto at_edge, uint32_t codes, uint32_t steps, int k0) {
      constexpr bool kEdge = decltype(at_edge)::value;
      // Everything of the 16 kS keys that this lane has: K's codes and steps of two keys,
      // V's of four, a sixteen.
      uint32_t wk[kS][2][D / 32], sk[kS][2], wv[kS][2][2][D / 64], sv[kS][2][2];
#pragma unroll
      for (int i = 0; i < kS; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t c0 = codes + (16 * i + 8 * h) * p.code_pitch, s0 = steps + (16 * i + 8 * h) * p.step_pitch;
          lds<D / 32>(c0 + k_codes, wk[i][h]);
          sk[i][h] = D == 128 ? lds_u16(s0 + k_steps) : lds_u8(s0 + k_steps);
          lds<D / 64>(c0 + v_codes, wv[i][h][0]);
          lds<D / 64>(c0 + v_codes + code_next, wv[i][h][1]);
          sv[i][h][0] = lds_u8(s0 + v_steps);
          sv[i][h][1] = lds_u8(s0 + v_steps + step_next);
        }
      }
      // S^T = K Q^T (two sums where there are few: a product waits for the last one's)
      float x[kS][kN][4];
#pragma unroll
      for (int i = 0; i < kS; ++i) {
        const uint32_t sa = fp4::from_e4m3x2(sk[i][0]), sb = fp4::from_e4m3x2(sk[i][1]);
        float x2[kTwo ? kN : 1][4] = {};
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][t][e] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t ha[4], hb[4];
          fp4::from_e2m1x8(wk[i][0][e], ha);
          fp4::from_e2m1x8(wk[i][1][e], hb);
          const uint32_t fa = e < 2 ? low2(sa) : high2(sa), fb = e < 2 ? low2(sb) : high2(sb);
          uint32_t qe[kN][4];
#pragma unroll
          for (int t = 0; t < kN; ++t) {
            if constexpr (kSharedQ) {
              const uint4 v = q_at[(t * (kQ / 4) + e) * 32];
              qe[t][0] = v.x, qe[t][1] = v.y, qe[t][2] = v.z, qe[t][3] = v.w;
            } else {
#pragma unroll
              for (int z = 0; z < 4; ++z) qe[t][z] = q[t][4 * e + z];
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t f[4] = {times(ha[2 * y], fa), times(hb[2 * y], fb), times(ha[2 * y + 1], fa),
                                   times(hb[2 * y + 1], fb)};
#pragma unroll
            for (int t = 0; t < kN; ++t) mma(kTwo && y ? x2[kTwo ? t : 0] : x[i][t], f, qe[t][2 * y], qe[t][2 * y + 1]);
          }
        }
#pragma unroll
        for (int t = 0; kTwo && t < kN; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][t][e] += x2[kTwo ? t : 0][e];
      }
      // Softmax: x[i][t][0..1] are key g's scores of rows 2 c, 2 c + 1, [2..3] key g + 8's.
      uint32_t hidden = 0;
      if constexpr (kEdge) {
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t mask = sm.mask[warp][8 * t + 2 * c + e];
#pragma unroll
            for (int i = 0; i < kS; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!among(mask, k0 + 16 * i + key_g + 8 * h, prefix, end)) hidden |= 1u << ((i * kN + t) * 4 + 2 * h + e);
          }
      }
      float y[kS][kN][4];
      auto shifted = [&]() {
#pragma unroll
        for (int i = 0; i < kS; ++i)
#pragma unroll
          for (int t = 0; t < kN; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[i][t][e] = fmaf(x[i][t][e], a[t][e & 1], -ms[t][e & 1]);
              if (kEdge && (hidden >> ((i * kN + t) * 4 + e) & 1u)) y[i][t][e] = -CUDART_INF_F;
            }
      };
      shifted();
      float most = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kS; ++i)
#pragma unroll
        for (int t = 0; t < kN; ++t)
          most = fmaxf(most, fmaxf(fmaxf(y[i][t][0], y[i][t][1]), fmaxf(y[i][t][2], y[i][t][3])));
      if (__any_sync(0xFFFFFFFFu, most > kLazy + kShift)) {
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < kS; ++i)
#pragma unroll
              for (int z = e; z < 4; z += 2)
                if (!kEdge || !(hidden >> ((i * kN + t) * 4 + z) & 1u)) top = fmaxf(top, x[i][t][z] * a[t][e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            if (top - ms[t][e] > kLazy + kShift) {
              const float alpha = ex2(ms[t][e] - (top - kShift));      // 0 when nothing was visible before
              ms[t][e] = top - kShift;
              l[t][e] *= alpha;
#pragma unroll
              for (int z = 0; z < kTiles; ++z) {
                o[t][z][e] *= alpha;
                o[t][z][e + 2] *= alpha;
              }
            }
          }
        shifted();
      }
      // O^T += V^T P: two pairs of keys, 2 c and 2 c + 1 and those 8 behind.
#pragma unroll
      for (int i = 0; i < kS; ++i) {
        uint32_t pb[kN][2], scale[2];
#pragma unroll
        for (int t = 0; t < kN; ++t) {
          const float p0 = ex2(y[i][t][0]), p1 = ex2(y[i][t][1]), p2 = ex2(y[i][t][2]), p3 = ex2(y[i][t][3]);
          l[t][0] += p0 + p2;
          l[t][1] += p1 + p3;
          pb[t][0] = transposed(pack2<false>(p0, p1));
          pb[t][1] = transposed(pack2<false>(p2, p3));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (kEdge) {
            // Rows past the run, and drafts that none sees, may hold anything.
            if (!among(sm.mask[warp][8 * kN], k0 + 16 * i + 8 * h + key_c, prefix, end)) sv[i][h][0] = 0;
            if (!among(sm.mask[warp][8 * kN], k0 + 16 * i + 8 * h + key_c1, prefix, end)) sv[i][h][1] = 0;
          }
          scale[h] = fp4::from_e4m3x2(sv[i][h][0] | sv[i][h][1] << 8);
        }
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          // Tiles 4 e and 4 e + 1: the even dimensions of the eight; then the odd ones.
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            uint32_t v2[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = wv[i][h][0][e], a1 = wv[i][h][1][e];
              fp4::from_e2m1x8(odd ? (a0 >> 4 & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u)
                                   : (a0 & 0x0F0F0F0Fu) | (a1 << 4 & 0xF0F0F0F0u), v2[h]);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t f[4] = {times(v2[0][2 * z], scale[0]), times(v2[0][2 * z + 1], scale[0]),
                                     times(v2[1][2 * z], scale[1]), times(v2[1][2 * z + 1], scale[1])};
#pragma unroll
              for (int t = 0; t < kN; ++t) mma(o[t][4 * e + 2 * odd + z], f, pb[t][0], pb[t][1]);
            }
          }
        }
      }
    };
    for (int k1 = begin; k1 < end; k1 += p.stage_keys) {
      if (!wait(sm, sm.full[stage], phase, p)) return;
      const uint32_t base = ring + stage * p.stage_bytes;
      const int last = min(k1 + p.stage_keys, end);
      for (int k0 = k1 + 16 * kS * j; k0 < last; k0 += 16 * kS * p.head_warps) {
        const uint32_t codes = base + (k0 - k1) * p.code_pitch, steps = base + (k0 - k1) * p.step_pitch + steps_at;
        if (k0 + 16 * kS > min(prefix, end)) keys(std::true_type(), codes, steps, k0);
        else keys(std::false_type(), codes, steps, k0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[stage]));
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }

    // ---- the unit's end: the warps of a head are put together.
    __syncwarp();
    s = sm.place[warp].s;
    const int head = s.head + head_local;
    const bool direct = s.n == s.nt;
    const int slot = 2 * (static_cast<int>(blockIdx.x) * p.heads + head_local) + (sm.place[warp].seg > 1 ? 1 : 0);
    float w_mine[kN][2], m_all[kN][2], l_all[kN][2];
#pragma unroll
    for (int t = 0; t < kN; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], d);
        if (l[t][e] == 0.f) ms[t][e] = -CUDART_INF_F;
        m_all[t][e] = ms[t][e];
        l_all[t][e] = l[t][e];
        w_mine[t][e] = 1.f;
        if (several && g == 0) sm.ml[warp][8 * t + 2 * c + e] = make_float2(ms[t][e], l[t][e]);
      }
    if (several) {
      if (!meet(sm, p, head_local, met)) return;
#pragma unroll
      for (int t = 0; t < kN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -CUDART_INF_F, sum = 0.f;
          for (int x = 0; x < p.head_warps; ++x) top = fmaxf(top, sm.ml[head_local * p.head_warps + x][8 * t + 2 * c + e].x);
          for (int x = 0; x < p.head_warps; ++x) {
            const float2 y = sm.ml[head_local * p.head_warps + x][8 * t + 2 * c + e];
            sum += (y.x == -CUDART_INF_F ? 0.f : ex2(y.x - top)) * y.y;
          }
          w_mine[t][e] = ms[t][e] == -CUDART_INF_F ? 0.f : ex2(ms[t][e] - top);
          m_all[t][e] = top;
          l_all[t][e] = sum;
        }
    }
    // Eight rows at a time.
#pragma unroll
    for (int t = 0; t < kN; ++t) {
      if (8 * t >= rows) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e, i = p.by_G.of(row);
        const long long out_row = (static_cast<long long>(s.b) * p.q_len + i) * p.H + head * p.G + (row - i * p.G);
        float by = w_mine[t][e] * p.v_factor;
        if (direct) by *= l_all[t][e] == 0.f ? 0.f : 1.f / l_all[t][e];       // (a NaN stays one)
        if (j == 0 && g == 0 && row < rows) {
          if (direct)
            p.lse[out_row] = l_all[t][e] == 0.f ? -CUDART_INF_F : (m_all[t][e] + log2f(l_all[t][e])) * 0.6931471805599453f;
          else
            p.part_ml[static_cast<size_t>(slot) * p.part_rows + row] = make_float2(m_all[t][e], l_all[t][e]);
        }
        // Dimensions g D / 8 .. of row `row`, in order.
        float v[2 * kTiles];
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
          const int at = (y >> 2) * 8 + (y & 1) * 4 + (y >> 1 & 1);
          v[at] = o[t][y][e] * by;
          v[at + 2] = o[t][y][e + 2] * by;
        }
        if (several) {
          float4* const to = reinterpret_cast<float4*>(sums + (warp * 8 + 2 * c + e) * kSumPitch<D> + g * (D / 8));
#pragma unroll
          for (int y = 0; y < D / 32; ++y) to[y] = make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
        } else if (row < rows) {
          if (direct) {
            uint4* const to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (out_row * D + g * (D / 8)) * 2);
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
              to[y] = make_uint4(pack2<kBf16>(v[8 * y], v[8 * y + 1]), pack2<kBf16>(v[8 * y + 2], v[8 * y + 3]),
                                 pack2<kBf16>(v[8 * y + 4], v[8 * y + 5]), pack2<kBf16>(v[8 * y + 6], v[8 * y + 7]));
          } else {
            float4* const to = p.part_o + (static_cast<size_t>(slot) * p.part_rows + row) * (D / 4) + g * (D / 32);
#pragma unroll
            for (int y = 0; y < D / 32; ++y) to[y] = make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
          }
        }
      }
      if (several) {
        if (!meet(sm, p, head_local, met)) return;
        const int here = min(8, rows - 8 * t);
        for (int x = j * 32 + lane; x < here * (D / 4); x += 32 * p.head_warps) {
          const int r = x / (D / 4), col = x % (D / 4), row = 8 * t + r;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int y = 0; y < p.head_warps; ++y) {
            const float4 v = *reinterpret_cast<const float4*>(sums + ((head_local * p.head_warps + y) * 8 + r) * kSumPitch<D> + col * 4);
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
          }
          if (direct) {
            const int i = p.by_G.of(row);
            const long long out_row = (static_cast<long long>(s.b) * p.q_len + i) * p.H + head * p.G + (row - i * p.G);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (out_row * D + col * 4) * 2) =
                make_uint2(pack2<kBf16>(sum.x, sum.y), pack2<kBf16>(sum.z, sum.w));
          } else {
            p.part_o[(static_cast<size_t>(slot) * p.part_rows + row) * (D / 4) + col] = sum;
          }
        }
        // (A next unit's warps meet before its sums take these ones' place.)
      }
    }
  }
}

template <int D, bool kBf16, int kN>
__global__ void __launch_bounds__(Shape8<kN>::kThreads, 1) few_kernel(const __grid_constant__ Maps maps, const FewParams p) {
  using C = Shape8<kN>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Head<kN>& sm = *reinterpret_cast<Head<kN>*>(smem_raw);
  float* const sums = reinterpret_cast<float*>(smem_raw + sizeof(Head<kN>));
  uint8_t* const shared_q = smem_raw + sizeof(Head<kN>) + (p.head_warps > 1 ? kSums<D> : 0);
  uint8_t* const ring = shared_q + kQBytes<D, kN>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    if (lane < p.stages) {
      mbar_init(smem_u32(&sm.full[lane]), p.box_rows ? 1 : 32 * kLoaders);
      mbar_init(smem_u32(&sm.empty[lane]), p.heads * p.head_warps);
    }
    if (lane < p.heads) mbar_init(smem_u32(&sm.meet[lane]), p.head_warps);
    if (lane == 0) sm.abort_flag = 0;
    fence_mbarrier_init_cluster();
    fence_proxy_async_smem();
  }
  grid_dependency_wait();
  if (tid == 0) grid_launch_dependents();

  // This CTA's run (as in the attention kernel, with a CTA a team).
  const int units = p.head_sets, team = blockIdx.x;
  const int per = (p.B + C::kThreads - 1) / C::kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int sum = 0, len;
  bool off = false;
  for (int b = b0; b < b1; ++b) {
    sum += stream_work(p, stream_tiles<kWhole>(p, b, len)) * units;
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
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWarps + kLoaders; ++i) {
    if (i == warp) before = total;
    total += sm.warp_sum[i];
  }
  const Runs runs(p, total, gridDim.x);
  const int t0 = team < runs.teams ? runs.start(team) : total;
  before += inc - sum;
  if (t0 >= before && t0 < before + sum) {
    int b = b0;
    while (true) {
      const int n = stream_work(p, stream_tiles<kWhole>(p, b, len)) * units;
      if (t0 < before + n) break;
      before += n;
      ++b;
    }
    sm.start_b = b;
    sm.start_pre = before;
  }
  __syncthreads();
  const bool any = t0 < total;
  const Walk<kWhole> walk(p, 0, t0, any ? runs.start(team + 1) : total, any ? sm.start_b : 0, any ? sm.start_pre : 0);

  if (warp >= kWarps) {
    if constexpr (C::kMore > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLess));
    if (warp == kWarps && lane == 0 && !p.whole) {
      // The merge's list: the units that start in this run and are cut (see note_cut_units).
      int4 d = make_int4(0, 0, 0, 0);
      Walk<kWhole> w = walk;
      Segment s;
      for (int seg = 0; w.next(p, s); ++seg) {
        if (s.tile0 != 0) continue;
        const bool cut = s.n < s.nt;
        const int parts = cut ? runs.team_of(w.t1 - s.n + s.nt - 1) - team + 1 : 0;
        if (cut) d = make_int4(s.b, s.head, 2 * team * p.heads + (seg > 0 ? 1 : 0), parts);
        if (p.desc_units)
          for (int h = 0; h < p.heads; ++h)
            p.desc[s.b * p.Hkv + s.head + h] = cut ? make_int4(s.b, s.head + h, d.z + 2 * h, parts) : make_int4(0, 0, 0, 0);
      }
      if (!p.desc_units) p.desc[team] = d;
    }
    __syncwarp();
    if (p.box_rows == 0) load_rows<kN>(sm, p, smem_u32(ring), D / 16, walk, warp - kWarps);
    else if (warp == kWarps) load_boxes<kN>(sm, p, maps, smem_u32(ring), D / 16, walk);
  } else {
    if constexpr (C::kMore > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMore));
    if (warp < p.heads * p.head_warps) {
      if (lane == 0) {
        sm.place[warp].walk = walk;
        sm.place[warp].seg = 0;
      }
      __syncwarp();
      attend<D, kBf16, kN>(sm, p, shared_q, smem_u32(ring), sums, warp, lane);
    }
  }
  // Streams without keys.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (stream_tiles<kWhole>(p, b, len) != 0) continue;
    if (p.desc_units && !p.whole)
      for (int u = tid; u < p.Hkv; u += C::kThreads) p.desc[b * p.Hkv + u] = make_int4(0, 0, 0, 0);
    const long long rows = static_cast<long long>(p.q_len) * p.H;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + b * rows * (D * 2));
    for (long long x = tid; x < rows * (D / 8); x += C::kThreads) o[x] = make_uint4(0, 0, 0, 0);
    for (long long x = tid; x < rows; x += C::kThreads) p.lse[b * rows + x] = -CUDART_INF_F;
  }
}

// The merge where each entry stands for a CTA's cut unit of every head (entries a
// head: combine_many_parts of the attention kernel).  A block lists the cut units,
// and takes chunks of eight rows of their heads in turn.
template <int D, bool kBf16>
__global__ void __launch_bounds__(D / 4 * kMergeUnits) combine_heads(const FewParams p, int entries) {
  constexpr int kThreadsM = D / 4 * kMergeUnits, kWarpsM = kThreadsM / 32;
  __shared__ int4 cut[kMaxParts];
  __shared__ int warp_cut[kWarpsM];
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
    for (int w = 0; w < kWarpsM; ++w) {
      if (w == warp && d.w != 0) cut[at + __popc(ballot & ((1u << (tid & 31)) - 1u))] = d;
      at += warp_cut[w];
    }
    n_cut = at;
    __syncthreads();
  }
  const int chunks = (p.q_len * p.G + kMergeUnits - 1) / kMergeUnits;
  for (int item = blockIdx.x; item < n_cut * p.heads * chunks; item += gridDim.x) {
    const int u = item / (p.heads * chunks), rest = item - u * p.heads * chunks, h = rest / chunks;
    int4 d = cut[u];
    d.y += h;
    d.z += 2 * h;
    merge_rows<D, kBf16, 1, 8, 1>(p, d, rest - h * chunks);
  }
}

// ------------------------------------------------------------ host

using Fn = void (*)(Maps, FewParams);
using MergeFn = void (*)(FewParams, int);
using PartsFn = void (*)(Params, int);
struct Variant {
  Fn attn;
  MergeFn merge;
  PartsFn parts, units;
  int threads, together, head_bytes, sum_bytes;
};
template <int D, bool kBf16, int kN>
Variant variant() {
  return {few_kernel<D, kBf16, kN>, combine_heads<D, kBf16>, combine_many_parts<D, kBf16>, combine_many_units<D, kBf16, 8, 1>,
          Shape8<kN>::kThreads, Shape8<kN>::kTogether, static_cast<int>(sizeof(Head<kN>)) + kQBytes<D, kN>, kSums<D>};
}

constexpr int kMostEights = 4;
constexpr int kSharedBytes = 232448;
constexpr int kStageBytes = 80 << 10;      // a stage, at most (40 KB: 150 us where 80 take 138)
constexpr int kStageKeys = 256;            // 32 boxes of eight rows, which is what a loader's lanes see to

std::mutex g_mutex;
bool g_ready[64][4][kMostEights];

// Key heads a CTA: the most that divide Hkv and leave no more than a quarter of the warps idle.
int heads_a_cta(int Hkv, int warps) {
  int best = 1;
  for (int h = 2; h <= warps && h <= Hkv; ++h)
    if (Hkv % h == 0 && 4 * h * (warps / h) >= 3 * warps) best = h;
  return best;
}

// Bytes of the longest run of steps that a CTA's heads have, from one multiple of 16 to another.
int most_step_bytes(int Hkv, int heads, int each) {
  int most = 0;
  for (int h = 0; h < Hkv; h += heads) {
    const int bytes = (((h + heads) * each + 15) & ~15) - ((h * each) & ~15);
    if (bytes > most) most = bytes;
  }
  return most;
}

}  // namespace few

// Whether this kernel can take a call, and whether it does: by its rows a key head, the
// sets of key heads that CTAs take apart (streams times Hkv / few_heads) and the keys that
// the table has room for.  GPU time here / with the tcgen05 kernel, us, D = 128, 8 heads
// a key head, 8 key heads, tables without spare room, pages of 64 rows unless said:
//   one stream of 1k, 4k, 16k, 64k, 256k keys (one CTA has all heads of a key):
//     one token  13.7 / 12.3, 14.3 / 13.4, 18.5 / 18.2, 30 / 38, 69 / 118
//     2 tokens   17 / 12, 17 / 14, 22 / 18, 35 / 38, 83 / 118
//     3          20 / 13, 21 / 14, 25 / 18, 42 / 38, 106 / 118 (of 128k 64 / 65; 16-row pages 64 / 84)
//     4          25 / 13, 25 / 14, 30 / 18, 50 / 38, 129 / 118 (of 128k 77 / 65; 16-row pages 77 / 84; D 64 48 / 63)
//   4 streams of 256, 1k, 4k, 16k, 64k keys:
//     one token  14.0 / 10.1, 14 / 19, 16 / 24, 29 / 42, 66 / 121
//     2 tokens   18 / 10, 18 / 19, 20 / 24, 36 / 43, 83 / 122
//     3          22 / 10, 21 / 19, 23 / 24, 43 / 43, 106 / 122
//     4          28 / 10, 29 / 19, 33 / 24, 58 / 43, 136 / 122 (16-row pages 58 / 49, 136 / 158 the last two)
//   32 streams of 64, 512, 4k, 16k: 2 tokens 11 / 16, 22 / 31, 54 / 76, 151 / 233; 3 13 / 16, 26 / 31, 67 / 78,
//     196 / 235; 4 16 / 16, 34 / 31, 85 / 79, 244 / 236 (16-row pages 84 / 93, 245 / 309 the last two)
//   64 streams of 64, 512, 4k, 16k: 4 tokens 16 / 29, 47 / 53, 144 / 148, 463 / 459; of 1k to 32k 287 / 356;
//   one token, one stream of 1k and 4k keys: 4 key heads 12 / 12, 12 / 14; one 9 / 11, 10 / 12.
// (A table with more room than its streams have keys is judged by its room: that costs up to
// the difference above, as 8 streams of 1k to 32k keys, 3 tokens, 58 / 50.)
bool few_can(int q_len, int H, int Hkv) {
  const long long rows = static_cast<long long>(q_len) * (H / Hkv);
  return rows <= 8 || (rows <= 8 * few::kMostEights && few_heads(Hkv) == few::kWarps);
}
bool few_rows(const Call& c) {
  if (!few_can(c.q_len, c.H, c.Hkv)) return false;
  const int rows = c.q_len * (c.H / c.Hkv), heads = few_heads(c.Hkv);
  const long long sets = static_cast<long long>(c.B) * (c.Hkv / heads), keys = sets * c.Smax;
  if (rows <= 8) return keys >= (sets == 1 && heads > 4 ? 1 << 14 : 1 << 11);
  if (sets >= (rows <= 24 ? 32 : 64)) return true;
  if (rows <= 16) return keys >= (sets == 1 ? 1 << 16 : 1 << 13);
  return (rows <= 24 || c.D == 64 || box_rows(c) < kKeys) && keys >= 1 << 17;
}
int few_heads(int Hkv) { return few::heads_a_cta(Hkv, few::kWarps); }

int run_few(const Call& c, const Params& shared, const DeviceCommon& d, int grid) {
  using namespace few;
  const int rows = c.q_len * (c.H / c.Hkv);
  const bool bf16 = c.dtype == MLA_BF16;
  static const Variant all[4][kMostEights] = {
      {variant<64, true, 1>(), variant<64, true, 2>(), variant<64, true, 3>(), variant<64, true, 4>()},
      {variant<64, false, 1>(), variant<64, false, 2>(), variant<64, false, 3>(), variant<64, false, 4>()},
      {variant<128, true, 1>(), variant<128, true, 2>(), variant<128, true, 3>(), variant<128, true, 4>()},
      {variant<128, false, 1>(), variant<128, false, 2>(), variant<128, false, 3>(), variant<128, false, 4>()}};
  const int type = (c.D == 128 ? 2 : 0) + (bf16 ? 0 : 1), eights = (rows + 7) / 8;
  const Variant& v = all[type][eights - 1];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MLA_ERR_UNSUPPORTED_DEVICE;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_ready[dev][type][eights - 1]) {
      if (cudaFuncSetAttribute(v.attn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes) != cudaSuccess) {
        cudaGetLastError();
        return MLA_ERR_LAUNCH;
      }
      g_ready[dev][type][eights - 1] = true;
    }
  }
  FewParams p = {};
  static_cast<Params&>(p) = shared;
  p.heads = heads_a_cta(c.Hkv, kWarps);
  p.head_warps = kWarps / p.heads;
  p.members = p.head_members = p.heads;
  p.head_sets = c.Hkv / p.heads;
  p.by_members = Divisor(p.heads);
  p.groups = p.group_members = p.group_sets = 1;
  p.by_group_members = p.by_group_sets = Divisor(1);
  p.split = p.heads != c.Hkv;
  p.row_end = fp4::row_bytes(c.Hkv, c.D);
  p.code_bytes = p.split ? p.heads * (c.D / 2) : p.row_end;
  p.step_bytes = p.split ? most_step_bytes(c.Hkv, p.heads, c.D / 16) : 0;
  p.code_pitch = p.code_bytes;
  p.step_pitch = p.split ? p.step_bytes : p.code_bytes;
  p.by_units = Divisor((p.code_bytes + p.step_bytes) / 16);
  // Rows 2 i and 2 i + 1 of K are read together, 64 bytes each, and rows 0, 2, 4 and 6 of
  // V, 32 bytes each: keys whose rows lie in different banks, as far as the pitch allows.
  p.order = p.code_pitch % 128 == 64 ? 0x67542310u : p.code_pitch % 64 == 32 ? 0x57463120u : 0x73625140u;
  const int key_bytes = 2 * (p.code_bytes + p.step_bytes);
  p.stage_keys = 16 * v.together * p.head_warps;
  const int fixed = v.head_bytes + (p.head_warps > 1 ? v.sum_bytes : 0), least = 16 * v.together * p.head_warps;
  while (2 * p.stage_keys <= kStageKeys && 2 * p.stage_keys * key_bytes <= kStageBytes) p.stage_keys *= 2;
  while (p.stage_keys > least && 2 * p.stage_keys * key_bytes > kSharedBytes - fixed) p.stage_keys /= 2;
  p.stage_bytes = p.stage_keys * key_bytes;
  const int stage = p.stage_bytes;
  p.stages = (kSharedBytes - fixed) / stage;
  if (p.stages > kMostStages) p.stages = kMostStages;
  if (p.stages < 2) return MLA_ERR_SHAPE;                  // (no number of heads gives less)
  // Boxes of at least eight rows (they begin at 128 bytes of shared memory) that neither
  // a page's nor a stage's end cuts.
  const int whole = p.stage_keys & -p.stage_keys, box = box_rows(c);
  p.box_rows = box < whole ? box : whole;
  Maps maps = {};
  for (int i = 0; i < 2 && p.box_rows; ++i) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.row_end) / 8, static_cast<cuuint64_t>(c.pool_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.pool_stride[i])};
    const cuuint32_t elem[2] = {1, 1};
    for (int part = 0; part <= p.split; ++part) {
      const cuuint32_t size[2] = {static_cast<cuuint32_t>(part ? p.step_bytes : p.code_bytes) / 8,
                                 static_cast<cuuint32_t>(p.box_rows)};
      if (d.encode(part ? &maps.steps[i] : &maps.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT64, 2,
                   const_cast<void*>(i ? c.v : c.k), dims, strides, size, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return MLA_ERR_LAUNCH;
    }
  }

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(v.threads, 1, 1);
  cfg.dynamicSmemBytes = fixed + p.stages * stage;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, v.attn, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  if (p.whole) return MLA_OK;
  const int entries = p.desc_units ? c.B * c.Hkv : grid, pairs = (rows + 1) / 2;
  cfg.blockDim = dim3(c.D / 4 * kMergeUnits, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cudaError_t err;
  if (p.desc_units && static_cast<long long>(entries) * pairs <= 3 * grid && grid / (c.B * p.head_sets) >= kManyParts) {
    cfg.gridDim = dim3(pairs, entries, 1);
    err = cudaLaunchKernelEx(&cfg, v.parts, static_cast<Params>(p), entries);
  } else {
    const long long chunks = static_cast<long long>(entries) * (p.desc_units ? 1 : p.heads) * ((rows + 7) / 8);
    cfg.gridDim = dim3(static_cast<unsigned>(chunks < 8 * grid ? chunks : 8 * grid), 1, 1);
    err = p.desc_units ? cudaLaunchKernelEx(&cfg, v.units, static_cast<Params>(p), entries)
                       : cudaLaunchKernelEx(&cfg, v.merge, p, entries);
  }
  if (err != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

}  // namespace gqa
}  // namespace mla
