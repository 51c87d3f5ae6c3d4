// Host side of mla_gqa_verify_attn, mla_gqa_verify_attn_window and their paged
// forms: argument checks, tensor maps and the two launches (attention, then the
// merge of the units that the even split of the work has cut).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "gqa_attn.cuh"
#include "gqa_host.h"
#include "internal.h"
#include "mla_verify_attn.h"

namespace mla {
namespace gqa {

constexpr int kMaxDevices = 64;
// Caches of at most so many keys are not cut: a CTA then takes whole units, and
// there is nothing to merge.  By the keys that the cache or table has room for,
// which is what the host knows.  9 drafts, 64 heads on 8 key heads, uncut / cut
// (room for one key more), us: one stream of 64 keys 5.9 / 8.4, of 256 7.0 / 10.6,
// of 512 8.8 / 10.9; 16 streams of 64 keys 7.7 / 13.0, of 512 10.4 / 19.0.
constexpr int kWholeKeys = 512;
// Row groups of a head that CTAs take side by side, at most.
constexpr int kMaxMembers = 16;

struct Plan {
  int groups;          // groups of 128 rows a key head
  int part_rows;       // rows of a partial, a multiple of 16
};

bool shape_ok(int B, int q, int H, int Hkv, int D) {
  return B >= 0 && B < (1 << 20) && q >= 1 && q <= 64 && H >= 1 && Hkv >= 1 && H % Hkv == 0 && (D == 64 || D == 128) &&
         static_cast<long long>(B) * q * H < (1ll << 31) && static_cast<long long>(q) * H < (1ll << 24);
}

Plan plan(int q, int H, int Hkv) {
  const int rows = q * (H / Hkv);
  Plan p;
  p.groups = (rows + kRows - 1) / kRows;
  p.part_rows = rows < kRows ? (rows + 15) / 16 * 16 : kRows;
  return p;
}

// One persistent CTA an SM.
int cta_count(const DeviceCommon& d) { return d.sms < kMaxParts ? d.sms : kMaxParts; }

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
  size_t ml, o, bytes;
};
Layout layout(const Plan& pl, int grid, int D) {
  Layout l;
  const size_t slots = 2 * static_cast<size_t>(grid);
  l.ml = round256(grid * sizeof(int4));
  l.o = round256(l.ml + slots * pl.part_rows * sizeof(float2));
  l.bytes = l.o + slots * pl.part_rows * D * sizeof(float);
  return l;
}

using CombineFn = void (*)(Params, int);

struct Variant {
  AttnFn attn;
  Fp4Fn fp4;                  // instead, kFp4
  CombineFn combine_parts, combine_few_chunks, combine_many_chunks;
  size_t smem;
  int threads;
};
template <int D, bool kBf16>
Variant variant() {
  constexpr size_t smem = sizeof(Smem<D, kWhole>);
  static_assert(smem <= 232448, "one CTA's shared memory");
  return {attn_kernel<D, kBf16, kWhole>, nullptr, combine_many_parts<D, kBf16>, combine_many_units<D, kBf16, 8, 1>,
          combine_many_units<D, kBf16, 3, 2>, smem, kThreads};
}

std::mutex g_ready_mutex;
bool g_ready[kMaxDevices][3][4];

// The kernels for these sizes, ready on the current device.
int pick(int D, int dtype, Mode mode, Variant* out) {
  static const Variant all[4] = {variant<64, true>(), variant<64, false>(), variant<128, true>(),
                                 variant<128, false>()};
  const int n = (D == 128 ? 2 : 0) + (dtype == MLA_FP16 ? 1 : 0);
  *out = all[n];
  if (mode == kWindow) out->attn = window_kernel(D, dtype == MLA_BF16);
  if (mode == kFp4) out->fp4 = fp4_kernel(D, dtype == MLA_BF16, &out->smem, &out->threads);
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_ready_mutex);
  if (!g_ready[dev][mode][n]) {
    const cudaFuncAttribute attribute = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const int bytes = static_cast<int>(out->smem);
    if ((mode == kFp4 ? cudaFuncSetAttribute(out->fp4, attribute, bytes) : cudaFuncSetAttribute(out->attn, attribute, bytes)) !=
        cudaSuccess) {
      cudaGetLastError();
      return MLA_ERR_LAUNCH;
    }
    g_ready[dev][mode][n] = true;
  }
  return MLA_OK;
}

// Byte strides of one tensor from element strides (or contiguous ones); a
// dimension of size 1 gets the contiguous stride.
int byte_strides(const int64_t* given, const long long* sizes, int D, long long* out) {
  long long whole = 2ll * D;
  for (int i = 2; i >= 0; --i) {
    out[i] = whole;
    if (given != nullptr && sizes[i] > 1) {
      if (given[i] < 8 || given[i] >= (1ll << 38)) return MLA_ERR_SHAPE;
      if (given[i] % 8) return MLA_ERR_ALIGN;
      out[i] = 2 * given[i];
    }
    whole *= sizes[i];
  }
  return MLA_OK;
}

// Rows a TMA box: whole 64-key tiles, or the largest power of two that no
// page boundary cuts, down to the 8 rows of a swizzle group; other page
// sizes are gathered row by row (0).
int box_rows(const Call& c) {
  if (c.table == nullptr) return kKeys;
  const int low = c.page & -c.page;
  return low >= kKeys ? kKeys : (low >= 8 ? low : 0);
}

// Heads side by side where a row of the cache holds them all: the most that
// leave fewer than 3 % of the CTAs without a team.
int heads_side_by_side(const long long* stride, int Hkv, int group_members, int grid) {
  int heads = 1;
  if (stride[2] < stride[1])
    for (int h = 2; h <= Hkv && h * group_members <= grid; ++h) {
      const int team = h * group_members;
      if (Hkv % h == 0 && 100 * (grid % team) < 3 * grid) heads = h;
    }
  return heads;
}

int encode(const DeviceCommon& d, CUtensorMap* map, const void* base, const Call& c, const long long* stride,
           long long rows, int batches, int box_rows, int box_chunks, CUtensorMapL2promotion promotion) {
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(c.D / 64),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(batches)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(stride[1]), 128, static_cast<cuuint64_t>(stride[2]),
                                 static_cast<cuuint64_t>(stride[0])};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_chunks), 1, 1};
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  const CUresult r =
      d.encode(map, c.dtype == MLA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
               const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_LAUNCH;
}

// The maps of pools held in 4 bits: rows of bytes, a box this many rows of a head's
// codes (in the swizzle that suits their width), or of 16 bytes that hold its steps.
int encode_fp4(const DeviceCommon& d, const Call& c, int rows, Fp4Maps* maps) {
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(fp4::row_bytes(c.Hkv, c.D)), static_cast<cuuint64_t>(c.pool_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.pool_stride[i])};
    const cuuint32_t codes[2] = {static_cast<cuuint32_t>(c.D / 2), static_cast<cuuint32_t>(rows)};
    const cuuint32_t steps[2] = {16, static_cast<cuuint32_t>(rows)}, elem[2] = {1, 1};
    void* const pool = const_cast<void*>(i ? c.v : c.k);
    if (d.encode(&maps->codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pool, dims, strides, codes, elem,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        d.encode(&maps->steps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pool, dims, strides, steps, elem,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

int run(const Call& c) {
  if (!shape_ok(c.B, c.q_len, c.H, c.Hkv, c.D) || c.Smax < 1 || c.Smax >= (1 << 24)) return MLA_ERR_SHAPE;
  if (c.mode == kWindow && (c.window < 1 || c.sinks < 0)) return MLA_ERR_SHAPE;
  if ((c.dtype != MLA_BF16 && c.dtype != MLA_FP16) || !std::isfinite(c.scale)) return MLA_ERR_ARG;
  const Plan pl = plan(c.q_len, c.H, c.Hkv);
  // The kernel counts the work, at most this, in 32 bits.
  if (static_cast<long long>((c.Smax + kKeys - 1) / kKeys) * c.Hkv * pl.groups >= (1ll << 31) / (c.B > 0 ? c.B : 1))
    return MLA_ERR_SHAPE;
  if (c.B == 0) return MLA_OK;
  if (!c.q || !c.k || !c.v || !c.seq_lens || !c.mask || !c.out || !c.lse) return MLA_ERR_NULLPTR;
  if (!aligned_to(c.q, 16) || !aligned_to(c.k, 16) || !aligned_to(c.v, 16) || !aligned_to(c.out, 16) ||
      !aligned_to(c.lse, 4) || !aligned_to(c.seq_lens, 4) || !aligned_to(c.mask, 4) ||
      (c.workspace && !aligned_to(c.workspace, 256)))
    return MLA_ERR_ALIGN;
  Params p = {};
  const bool paged = c.table != nullptr;
  const long long rows = paged ? c.pool_rows : c.Smax;
  const int batches = paged ? 1 : c.B;
  const long long q_sizes[3] = {c.B, c.q_len, c.H}, kv_sizes[3] = {batches, rows, c.Hkv};
  int st = byte_strides(c.strides, q_sizes, c.D, p.q_stride);
  if (c.mode == kFp4) {
    p.k_stride[1] = c.pool_stride[0];
    p.v_stride[1] = c.pool_stride[1];
    p.k_stride[2] = p.v_stride[2] = c.D / 2;
    p.steps_at = fp4::code_bytes(c.Hkv, c.D);
    p.v_factor = c.v_factor;
  } else {
    if (st == MLA_OK) st = byte_strides(c.strides ? c.strides + 3 : nullptr, kv_sizes, c.D, p.k_stride);
    if (st == MLA_OK) st = byte_strides(c.strides ? c.strides + 6 : nullptr, kv_sizes, c.D, p.v_stride);
  }
  if (st != MLA_OK) return st;

  DeviceCommon d;
  st = device_common(&d);
  if (st != MLA_OK) return st;
  const int grid = cta_count(d);
  const bool few = c.mode == kFp4 && few_rows(c);
  const Layout lay = layout(pl, few ? grid * few_heads(c.Hkv) : grid, c.D);
  if (!c.workspace || c.workspace_bytes < lay.bytes) return MLA_ERR_WORKSPACE;
  Variant var = {};
  if (!few) st = pick(c.D, c.dtype, c.mode, &var);
  if (st != MLA_OK) return st;

  const int box = box_rows(c);
  p.group_sets = (pl.groups + kMaxMembers - 1) / kMaxMembers;
  p.group_members = (pl.groups + p.group_sets - 1) / p.group_sets;
  const int heads = heads_side_by_side(p.k_stride, c.Hkv, p.group_members, grid);
  p.members = heads * p.group_members;
  p.head_members = heads;
  p.head_sets = c.Hkv / heads;
  p.by_members = Divisor(p.members);
  p.by_group_members = Divisor(p.group_members);
  p.by_group_sets = Divisor(p.group_sets);
  p.by_G = Divisor(c.H / c.Hkv);
  // Fetches of 256 bytes into L2 where the team wants all of them: also with 64
  // dims a head, if two heads or two rows lie side by side (64 streams of 16k
  // keys 347 -> 326 us; without teams such fetches cost 480 us against 397).
  const bool fetch_256 = c.D == 128 || heads > 1 || p.k_stride[1] == 2 * c.D;
  const CUtensorMapL2promotion promotion =
      fetch_256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  CUtensorMap map_k = {}, map_v = {};
  Fp4Maps fp4_maps = {};
  if (c.mode == kFp4 && !few && box != 0) {
    st = encode_fp4(d, c, box, &fp4_maps);
    if (st != MLA_OK) return st;
  }
  if (c.mode != kFp4 && box != 0 && (encode(d, &map_k, c.k, c, p.k_stride, rows, batches, box, box == kKeys ? c.D / 64 : 1, promotion) != MLA_OK ||
                   encode(d, &map_v, c.v, c, p.v_stride, rows, batches, box, box == kKeys ? c.D / 64 : 1, promotion) != MLA_OK))
    return MLA_ERR_LAUNCH;

  uint8_t* const ws = static_cast<uint8_t*>(c.workspace);
  p.q = static_cast<const uint8_t*>(c.q);
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.seq_lens = c.seq_lens;
  p.mask = c.mask;
  p.block_table = c.table;
  p.out = c.out;
  p.lse = c.lse;
  p.desc = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
  p.part_o = reinterpret_cast<float4*>(ws + lay.o);
  p.status = d.status_word;
  p.B = c.B;
  p.q_len = c.q_len;
  p.H = c.H;
  p.Hkv = c.Hkv;
  p.G = c.H / c.Hkv;
  p.Smax = c.Smax;
  p.groups = pl.groups;
  p.part_rows = pl.part_rows;
  const int rows_a_head = c.q_len * (c.H / c.Hkv);
  const long long units = static_cast<long long>(c.B) * c.Hkv * pl.groups;
  p.desc_units = units <= grid;
  long long most_tiles = (c.Smax + kKeys - 1) / kKeys;     // of a stream
  if (c.mode == kWindow) {
    const long long seen = (static_cast<long long>(c.sinks) + kKeys - 1) / kKeys +
                           (static_cast<long long>(c.window) + c.q_len + 2 * kKeys - 2) / kKeys;
    if (seen < most_tiles) most_tiles = seen;
  }
  p.whole = most_tiles <= kWholeKeys / kKeys;
  p.window = c.window;
  p.sinks = c.sinks;
  p.max_blocks = c.max_blocks;
  p.page = Divisor(paged ? c.page : 1);
  p.pool_pages = paged ? static_cast<int>(c.pool_rows / c.page) : 0;
  p.box_rows = box;
  p.test_stall = d.test_stall;
  p.scale_log2 = c.scale * 1.4426950408889634f;

  if (few) return run_few(c, p, d, grid);

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(var.threads, 1, 1);
  cfg.dynamicSmemBytes = var.smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((c.mode == kFp4 ? cudaLaunchKernelEx(&cfg, var.fp4, fp4_maps, p)
                      : cudaLaunchKernelEx(&cfg, var.attn, map_k, map_v, p)) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  if (p.whole) return MLA_OK;
  // The merge's shape: by the parts a cut unit has, about, if the blocks that
  // gives are not more than fit the device at once (three an SM).
  const int entries = p.desc_units ? static_cast<int>(units) : grid;
  const int pairs = ((rows_a_head < pl.part_rows ? rows_a_head : pl.part_rows) + 1) / 2;
  const bool many = p.desc_units && static_cast<long long>(entries) * pairs <= 3 * grid &&
                    (grid / p.members) / (static_cast<long long>(c.B) * p.head_sets * p.group_sets) >= kManyParts;
  CombineFn combine = var.combine_parts;
  if (many) {
    cfg.gridDim = dim3(pairs, entries, 1);
  } else {
    long long chunks = static_cast<long long>(entries) * (pl.part_rows / kMergeUnits);
    combine = var.combine_few_chunks;
    if (chunks > 5 * grid) {
      combine = var.combine_many_chunks;
      chunks /= 2;                                         // (twice the rows)
    }
    cfg.gridDim = dim3(static_cast<unsigned>(chunks < 8 * grid ? chunks : 8 * grid), 1, 1);
  }
  cfg.blockDim = dim3(c.D / 4 * kMergeUnits, 1, 1);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, combine, p, entries) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

}  // namespace gqa
}  // namespace mla

extern "C" {

size_t mla_gqa_workspace_size(int B, int q_len, int H, int Hkv, int D) {
  using namespace mla;
  if (!gqa::shape_ok(B, q_len, H, Hkv, D)) return 0;
  DeviceCommon d;
  if (device_common(&d) != MLA_OK) return 0;
  return gqa::layout(gqa::plan(q_len, H, Hkv), gqa::cta_count(d), D).bytes;
}

int mla_gqa_verify_attn(const void* q, const void* k, const void* v, const int64_t* strides,
                        const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len, int H,
                        int Hkv, int D, int Smax, int dtype, float scale, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const mla::gqa::Call c = {q, k, v, strides, seq_lens, tree_mask, B, q_len, H, Hkv, D, Smax, dtype, scale,
                            out, lse, workspace, workspace_bytes, stream, nullptr, 0, 0, 0, mla::gqa::kWhole, 0, 0};
  return mla::gqa::run(c);
}

int mla_gqa_verify_attn_window(const void* q, const void* k, const void* v, const int64_t* strides,
                               const int32_t* seq_lens, const uint32_t* tree_mask, int B, int q_len, int H,
                               int Hkv, int D, int Smax, int dtype, float scale, int window, int sinks,
                               void* out, float* lse, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  const mla::gqa::Call c = {q, k, v, strides, seq_lens, tree_mask, B, q_len, H, Hkv, D, Smax, dtype, scale,
                            out, lse, workspace, workspace_bytes, stream, nullptr, 0, 0, 0, mla::gqa::kWindow,
                            window, sinks};
  return mla::gqa::run(c);
}

}  // extern "C"

namespace mla {
namespace gqa {

// What the paged calls check before the others.
int run_paged(Call c, const int32_t* block_table, int max_blocks, int page_size, long long pool_rows) {
  if (page_size < 1 || max_blocks < 1 || static_cast<long long>(max_blocks) * page_size >= (1ll << 24) ||
      pool_rows < 1 || pool_rows % page_size != 0 || pool_rows >= (1ll << 31))
    return MLA_ERR_SHAPE;
  if (c.B > 0 && !block_table) return MLA_ERR_NULLPTR;
  if (!aligned_to(block_table, 4)) return MLA_ERR_ALIGN;
  c.table = block_table;
  c.max_blocks = max_blocks;
  c.page = page_size;
  c.pool_rows = pool_rows;
  c.Smax = max_blocks * page_size;
  return run(c);
}

}  // namespace gqa
}  // namespace mla

extern "C" {

int mla_gqa_verify_attn_paged(const void* q, const void* k_pool, const void* v_pool,
                              const int64_t* strides, long long pool_rows, const int32_t* block_table,
                              int max_blocks, int page_size, const int32_t* seq_lens,
                              const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D,
                              int dtype, float scale, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  const mla::gqa::Call c = {q, k_pool, v_pool, strides, seq_lens, tree_mask, B, q_len, H, Hkv, D, 0, dtype, scale,
                            out, lse, workspace, workspace_bytes, stream, nullptr, 0, 0, 0, mla::gqa::kWhole, 0, 0};
  return mla::gqa::run_paged(c, block_table, max_blocks, page_size, pool_rows);
}

size_t mla_gqa_fp4_workspace_size(int B, int q_len, int H, int Hkv, int D) {
  using namespace mla;
  if (!gqa::shape_ok(B, q_len, H, Hkv, D) || Hkv > MLA_FP4_MAX_HEADS) return 0;
  DeviceCommon d;
  if (device_common(&d) != MLA_OK) return 0;
  // (Whichever kernel takes the call: that is for the table's size to say.)
  const bool few = gqa::few_can(q_len, H, Hkv);
  return gqa::layout(gqa::plan(q_len, H, Hkv), gqa::cta_count(d) * (few ? gqa::few_heads(Hkv) : 1), D).bytes;
}

int mla_gqa_verify_attn_fp4_paged(const void* q, const int64_t* q_strides, const void* k_pool, long long k_pool_stride,
                                  const void* v_pool, long long v_pool_stride, long long pool_rows,
                                  const int32_t* block_table, int max_blocks, int page_size, const int32_t* seq_lens,
                                  const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D, int dtype,
                                  float scale, float k_factor, float v_factor, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  const long long row = static_cast<long long>(mla_gqa_fp4_row_bytes(Hkv, D)), limit = 1ll << 32;
  if (row == 0 || k_pool_stride < row || v_pool_stride < row || k_pool_stride > limit || v_pool_stride > limit)
    return MLA_ERR_SHAPE;
  if (!mla::fp4::factor_ok(k_factor) || !mla::fp4::factor_ok(v_factor) || !std::isfinite(scale) ||
      !std::isfinite(scale * k_factor))
    return MLA_ERR_ARG;
  if (k_pool_stride % 16 || v_pool_stride % 16) return MLA_ERR_ALIGN;
  mla::gqa::Call c = {q, k_pool, v_pool, q_strides, seq_lens, tree_mask, B, q_len, H, Hkv, D, 0, dtype, scale * k_factor,
                      out, lse, workspace, workspace_bytes, stream, nullptr, 0, 0, 0, mla::gqa::kFp4, 0, 0};
  c.pool_stride[0] = k_pool_stride;
  c.pool_stride[1] = v_pool_stride;
  c.v_factor = v_factor;
  return mla::gqa::run_paged(c, block_table, max_blocks, page_size, pool_rows);
}

int mla_gqa_verify_attn_window_paged(const void* q, const void* k_pool, const void* v_pool,
                                     const int64_t* strides, long long pool_rows, const int32_t* block_table,
                                     int max_blocks, int page_size, const int32_t* seq_lens,
                                     const uint32_t* tree_mask, int B, int q_len, int H, int Hkv, int D,
                                     int dtype, float scale, int window, int sinks, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const mla::gqa::Call c = {q, k_pool, v_pool, strides, seq_lens, tree_mask, B, q_len, H, Hkv, D, 0, dtype, scale,
                            out, lse, workspace, workspace_bytes, stream, nullptr, 0, 0, 0, mla::gqa::kWindow,
                            window, sinks};
  return mla::gqa::run_paged(c, block_table, max_blocks, page_size, pool_rows);
}

}  // extern "C"
