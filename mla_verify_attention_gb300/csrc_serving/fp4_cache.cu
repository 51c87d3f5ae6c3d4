// Rows into a cache held in 4 bits (mla_gqa_cache_append_fp4).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp4_format.cuh"
#include "internal.h"
#include "launch.h"
#include "mla_verify_attn.h"
#include "ptx.cuh"

namespace mla {
namespace fp4 {

// Mathematics.  For each 16 values x of a head, with the pool's factor f:
//   step = E4M3 nearest to min(448, max|x| / (6 f)),  d = step * f,
//   code = E2M1 nearest to x / d (both ties to even; all 0 where d is 0).
// max|x| / (6 f) is one IEEE division a group.  x / d is x times the correctly
// rounded 1 / d with one correction of its remainder, which rounds as the division does
// (Markstein's theorem; no operand leaves the normal range, see factor_ok): so a
// value halfway between two codes stays there, as in exact arithmetic.
//
// What bounds it: 2 bytes a value read, 9 / 16 written, 2 more where the values
// held are asked for; a lane takes eight values (16 bytes in, 4 out), a warp one row
// of K or V, four loads in flight a lane.
struct AppendParams {
  const uint8_t* src[2];
  long long src_stride[2];
  uint8_t* pool[2];
  long long pool_stride[2];
  uint8_t* held[2];                // null: not wanted
  long long held_stride[2];
  float factor[2];
  const int32_t* slots;
  unsigned int* status;
  long long pool_rows;
  int T, units, code_bytes;        // units: eight values
};

constexpr int kWarps = 8;
constexpr int kLoads = 4;

template <bool kBf16>
__device__ __forceinline__ float to_float(uint32_t half_bits) {
  if (kBf16) return __uint_as_float(half_bits << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(half_bits)));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  if (kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One lane's eight values; two lanes side by side share a step.
template <bool kBf16>
__device__ __forceinline__ void quantise(const uint4& v, float factor, float six_factor, uint32_t& codes, uint32_t& step,
                                         float& d) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // Magnitudes of 16-bit floats order as whole numbers do, NaN above all.
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  step = to_e4m3(__fdiv_rn(to_float<kBf16>(top), six_factor));
  d = __half2float(__ushort_as_half(static_cast<unsigned short>(from_e4m3x2(step) & 0xFFFFu))) * factor;
  codes = 0;
  if (!(d > 0.f)) return;                                  // nothing but 0, or NaN
  const float r = __frcp_rn(d), most = 8.f * d;            // (beyond 6 d all is one code; infinities end here)
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fminf(fmaxf(to_float<kBf16>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu), -most), most);
    const float q = a * r;
    x[e] = copysignf(__fmaf_rn(__fmaf_rn(-q, d, a), r, q), a);   // (-0 would lose its sign)
  }
  codes = to_e2m1x8(x);
}

template <bool kBf16>
__global__ void __launch_bounds__(32 * kWarps) append_fp4_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w >> 1);
  const bool second = w & 1u;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if (t >= p.T) return;
  const int slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.pool_rows) {
    if (lane == 0 && !second) atomicOr(p.status, kBitSlot);
    return;
  }
  const uint4* const src =
      reinterpret_cast<const uint4*>((second ? p.src[1] : p.src[0]) + t * (second ? p.src_stride[1] : p.src_stride[0]));
  uint8_t* const row = (second ? p.pool[1] : p.pool[0]) + slot * (second ? p.pool_stride[1] : p.pool_stride[0]);
  uint8_t* const held = second ? p.held[1] : p.held[0];
  const long long held_at = t * (second ? p.held_stride[1] : p.held_stride[0]);
  const float factor = second ? p.factor[1] : p.factor[0], six = 6.f * factor;
  for (int c = lane; c - lane < p.units; c += 32 * kLoads) {
    uint4 v[kLoads] = {};
#pragma unroll
    for (int e = 0; e < kLoads; ++e)
      if (c + 32 * e < p.units) v[e] = src[c + 32 * e];
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int u = c + 32 * e;
      if (u - lane >= p.units) break;                      // (the same for the whole warp)
      uint32_t codes, step;
      float d;
      quantise<kBf16>(v[e], factor, six, codes, step, d);
      if (u >= p.units) continue;
      reinterpret_cast<uint32_t*>(row)[u] = codes;
      if (!(u & 1)) row[p.code_bytes + (u >> 1)] = static_cast<uint8_t>(step);
      if (held != nullptr) {
        uint32_t h[4], o[4];
        from_e2m1x8(codes, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
          o[i] = pack<kBf16>(x.x * d, x.y * d);
        }
        reinterpret_cast<uint4*>(held + held_at)[u] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace fp4
}  // namespace mla

extern "C" {

size_t mla_gqa_fp4_row_bytes(int Hkv, int D) {
  if (Hkv < 1 || Hkv > MLA_FP4_MAX_HEADS || (D != 64 && D != 128)) return 0;
  return static_cast<size_t>(mla::fp4::row_bytes(Hkv, D));
}

int mla_gqa_cache_append_fp4(const void* k, long long k_stride, const void* v, long long v_stride, int Hkv, int D,
                             int dtype, float k_factor, float v_factor, void* k_pool, long long k_pool_stride,
                             void* v_pool, long long v_pool_stride, long long pool_rows, const int32_t* slots, int T,
                             void* k_held, long long k_held_stride, void* v_held, long long v_held_stride,
                             cudaStream_t stream) {
  using namespace mla;
  const long long row = static_cast<long long>(mla_gqa_fp4_row_bytes(Hkv, D)), limit = 1ll << 32;
  const long long wide = 2ll * Hkv * D;
  if (row == 0 || T < 0 || T >= (1 << 30) || pool_rows < 1 || pool_rows >= (1ll << 31) || k_pool_stride < row ||
      v_pool_stride < row || k_pool_stride > limit || v_pool_stride > limit || k_stride < 0 || v_stride < 0 ||
      k_stride > limit || v_stride > limit || (k_held && (k_held_stride < wide || k_held_stride > limit)) ||
      (v_held && (v_held_stride < wide || v_held_stride > limit)))
    return MLA_ERR_SHAPE;
  if ((dtype != MLA_BF16 && dtype != MLA_FP16) || !fp4::factor_ok(k_factor) || !fp4::factor_ok(v_factor)) return MLA_ERR_ARG;
  if (T == 0) return MLA_OK;
  if (!k || !v || !k_pool || !v_pool || !slots) return MLA_ERR_NULLPTR;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) ||
      !aligned_to(k_held, 16) || !aligned_to(v_held, 16) || !aligned_to(slots, 4) || k_stride % 16 || v_stride % 16 ||
      k_pool_stride % 16 || v_pool_stride % 16 || (k_held && k_held_stride % 16) || (v_held && v_held_stride % 16))
    return MLA_ERR_ALIGN;
  DeviceCommon d;
  const int st = device_common(&d);
  if (st != MLA_OK) return st;
  fp4::AppendParams p = {};
  const void* const src[2] = {k, v};
  void* const pool[2] = {k_pool, v_pool};
  void* const held[2] = {k_held, v_held};
  const long long strides[3][2] = {{k_stride, v_stride}, {k_pool_stride, v_pool_stride}, {k_held_stride, v_held_stride}};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = static_cast<const uint8_t*>(src[i]);
    p.src_stride[i] = strides[0][i];
    p.pool[i] = static_cast<uint8_t*>(pool[i]);
    p.pool_stride[i] = strides[1][i];
    p.held[i] = static_cast<uint8_t*>(held[i]);
    p.held_stride[i] = strides[2][i];
  }
  p.factor[0] = k_factor;
  p.factor[1] = v_factor;
  p.slots = slots;
  p.status = d.status_word;
  p.pool_rows = pool_rows;
  p.T = T;
  p.units = Hkv * (D / 8);
  p.code_bytes = fp4::code_bytes(Hkv, D);
  const unsigned blocks = static_cast<unsigned>((2ll * T + fp4::kWarps - 1) / fp4::kWarps);
  return launch_dependent(dtype == MLA_BF16 ? fp4::append_fp4_kernel<true> : fp4::append_fp4_kernel<false>, p, dim3(blocks),
                          32 * fp4::kWarps, 0, stream);
}

}  // extern "C"
