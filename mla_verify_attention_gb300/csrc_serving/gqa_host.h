// What the host sides of the grouped-head calls share; defined in gqa_attn.cu
// where nothing else is said.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_attn.cuh"
#include "internal.h"

namespace mla {
namespace gqa {

struct Call {
  const void *q, *k, *v;
  const int64_t* strides;
  const int32_t* seq_lens;
  const uint32_t* mask;
  int B, q_len, H, Hkv, D, Smax, dtype;
  float scale;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
  const int32_t* table;   // paged
  int max_blocks, page;
  long long pool_rows;
  Mode mode;
  int window, sinks;
  long long pool_stride[2];   // kFp4: bytes, K and V
  float v_factor;
};

bool shape_ok(int B, int q, int H, int Hkv, int D);
int byte_strides(const int64_t* given, const long long* sizes, int D, long long* out);
int box_rows(const Call& c);
int heads_side_by_side(const long long* stride, int Hkv, int group_members, int grid);
int encode(const DeviceCommon& d, CUtensorMap* map, const void* base, const Call& c, const long long* stride,
           long long rows, int batches, int box_rows, int box_chunks, CUtensorMapL2promotion promotion);
int cta_count(const DeviceCommon& d);

// Forms of the attention kernel that are compiled on their own.
using AttnFn = void (*)(CUtensorMap, CUtensorMap, Params);
AttnFn window_kernel(int D, bool bf16);    // gqa_window.cu
using Fp4Fn = void (*)(Fp4Maps, Params);
Fp4Fn fp4_kernel(int D, bool bf16, size_t* smem, int* threads);    // gqa_fp4.cu

// The kernel for few query rows a key head over a cache in 4 bits: whether it can take a
// call and whether it does, key heads a CTA, and its launches (gqa_fp4_few.cu).
bool few_can(int q_len, int H, int Hkv);
bool few_rows(const Call& c);
int few_heads(int Hkv);
int run_few(const Call& c, const Params& shared, const DeviceCommon& d, int grid);

// Parts a unit from which four part groups share the merge of a row.
constexpr int kManyParts = 8;

}  // namespace gqa
}  // namespace mla
