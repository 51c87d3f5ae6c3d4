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
// A quotient x / d is q = x r for an approximate reciprocal r (relative error e < 2^-22)
// and one correction by the remainder, q + (x - q d) r, both fused: off by e^2 before
// its one rounding.  Where f is a power of two, a quotient that is a number halfway
// between two codes or steps so comes out as that number, as in exact arithmetic, and one
// that is not lies 2^-19 or more away (x has 11 bits, a step 4, a border 3).  For another
// f, 6 f and step f are rounded to fp32 (2^-24) before the division and its quotient
// once more: one within 2^-22 of halfway may come out on either side.  The values are taken negative and
// their remainder as q d - x: its zero then leaves the sign of a q of -0.
//
// What bounds it: 2 bytes a value read, 9 / 16 written, 2 more where the values held are
// asked for, and as much the conversions and quotients: 32,251 tokens of 8 heads of 128
// with the values held 54.7 us, 5.5 TB/s (81 % of the measured copy rate), at 3.1
// instructions a cycle and SM.  A lane takes eight values (16 bytes in, 4 out), four
// loads in flight (2 or 8: 65, 62 us; values read before the slot is known: no change).
// A block takes as many rows of K or V as its threads' loads cover (a warp a row left
// half the lanes of a 16-unit row idle: 32k rows of one head 25.7 us).
struct AppendParams {
  const uint8_t* src[2];
  uint8_t* pool[2];
  uint8_t* held[2];                // null: not wanted
  uint32_t src_stride[2], pool_stride[2], held_stride[2];   // in 16 bytes
  float factor[2], by_six[2];      // 1 / (6 factor), rounded
  const int32_t* slots;
  unsigned int* status;
  long long pool_rows;
  int T, units, code_bytes;        // units: eight values
  int block_rows;
  Divisor by_units;
};

constexpr int kThreads = 128;
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

// A pair of values as fp32.
template <bool kBf16>
__device__ __forceinline__ uint64_t to_floats(uint32_t two) {
  if (kBf16) return f2pack(bf16lo_to_f32(two), bf16hi_to_f32(two));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
  return f2pack(f.x, f.y);
}
// a b for each half (a sum with -0 changes nothing).
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) { return ffma2(a, b, 0x8000000080000000ull); }

// One lane's eight values; two lanes side by side share a step.
template <bool kBf16>
__device__ __forceinline__ void quantise(const uint4& v, float factor, float six_factor, float by_six, uint32_t& codes,
                                         uint32_t& step, float& d) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // Magnitudes of 16-bit floats order as whole numbers do, NaN above all.
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  const float most = to_float<kBf16>(top), q = most * by_six;
  const float quotient = __fmaf_rn(-__fmaf_rn(q, six_factor, -most), by_six, q);
  step = to_e4m3(q < 1024.f ? quotient : q);               // (infinities and NaN have no remainder)
  d = __half2float(__ushort_as_half(static_cast<unsigned short>(from_e4m3x2(step) & 0xFFFFu))) * factor;
  codes = 0;
  if (!(d > 0.f)) return;                                  // nothing but 0, or NaN
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  const uint64_t minus_r2 = f2pack(-r, -r), d2 = f2pack(d, d);
  const bool beyond = most > 7.f * d;                      // of the largest step's reach: all one code
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint64_t minus = to_floats<kBf16>(w[e] ^ 0x80008000u);
    if (beyond) {
      float lo, hi;
      f2unpack(minus, lo, hi);
      minus = f2pack(fminf(fmaxf(lo, -7.f * d), 7.f * d), fminf(fmaxf(hi, -7.f * d), 7.f * d));
    }
    const uint64_t q2 = fmul2(minus, minus_r2);
    f2unpack(ffma2(ffma2(q2, d2, minus), minus_r2, q2), x[2 * e], x[2 * e + 1]);
  }
  codes = to_e2m1x8(x);
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) append_fp4_kernel(const AppendParams p) {
  const int tid = threadIdx.x;
  const bool second = blockIdx.y != 0;
  const int t0 = static_cast<int>(blockIdx.x) * p.block_rows, rows = min(p.block_rows, p.T - t0), all = rows * p.units;
  grid_dependency_wait();
  if (tid == 0) grid_launch_dependents();
  const uint8_t* const src = second ? p.src[1] : p.src[0];
  uint8_t* const pool = second ? p.pool[1] : p.pool[0];
  uint8_t* const held = second ? p.held[1] : p.held[0];
  const uint32_t src_stride = second ? p.src_stride[1] : p.src_stride[0];
  const uint32_t pool_stride = second ? p.pool_stride[1] : p.pool_stride[0];
  const uint32_t held_stride = second ? p.held_stride[1] : p.held_stride[0];
  auto row_of = [](auto* base, int row, uint32_t stride) {
    return base + static_cast<uint64_t>(static_cast<uint32_t>(row)) * stride * 16;
  };
  const float factor = second ? p.factor[1] : p.factor[0], six = 6.f * factor, by_six = second ? p.by_six[1] : p.by_six[0];
  for (int x0 = 0; x0 < all; x0 += kThreads * kLoads) {    // (the same for the whole block)
    uint4 v[kLoads] = {};
    int unit[kLoads], row[kLoads], slot[kLoads];
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int x = x0 + e * kThreads + tid, r = p.by_units.of(x);
      row[e] = t0 + r;
      unit[e] = x - r * p.units;
      slot[e] = x < all ? p.slots[row[e]] : -1;
    }
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      if (slot[e] >= p.pool_rows) {
        atomicOr(p.status, kBitSlot);
        slot[e] = -1;
      }
      if (slot[e] >= 0) v[e] = reinterpret_cast<const uint4*>(row_of(src, row[e], src_stride))[unit[e]];
    }
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      uint32_t codes, step;
      float d;
      quantise<kBf16>(v[e], factor, six, by_six, codes, step, d);  // (eight lanes side by side have one row)
      step |= __shfl_down_sync(0xFFFFFFFFu, step, 2) << 8;
      step |= __shfl_down_sync(0xFFFFFFFFu, step, 4) << 16;
      if (slot[e] < 0) continue;
      uint8_t* const to = row_of(pool, slot[e], pool_stride);
      reinterpret_cast<uint32_t*>(to)[unit[e]] = codes;
      if (!(unit[e] & 7)) *reinterpret_cast<uint32_t*>(to + p.code_bytes + (unit[e] >> 1)) = step;
      if (held != nullptr) {
        uint32_t h[4], o[4];
        from_e2m1x8(codes, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          f2unpack(fmul2(to_floats<false>(h[i]), f2pack(d, d)), lo, hi);
          o[i] = pack<kBf16>(lo, hi);
        }
        reinterpret_cast<uint4*>(row_of(held, row[e], held_stride))[unit[e]] = make_uint4(o[0], o[1], o[2], o[3]);
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
    p.src_stride[i] = static_cast<uint32_t>(strides[0][i] / 16);
    p.pool[i] = static_cast<uint8_t*>(pool[i]);
    p.pool_stride[i] = static_cast<uint32_t>(strides[1][i] / 16);
    p.held[i] = static_cast<uint8_t*>(held[i]);
    p.held_stride[i] = static_cast<uint32_t>(strides[2][i] / 16);
  }
  p.factor[0] = k_factor;
  p.factor[1] = v_factor;
  for (int i = 0; i < 2; ++i) p.by_six[i] = 1.f / (6.f * p.factor[i]);
  p.slots = slots;
  p.status = d.status_word;
  p.pool_rows = pool_rows;
  p.T = T;
  p.units = Hkv * (D / 8);
  p.code_bytes = fp4::code_bytes(Hkv, D);
  p.by_units = Divisor(p.units);
  p.block_rows = fp4::kThreads * fp4::kLoads / p.units;
  if (p.block_rows < 1) p.block_rows = 1;
  const unsigned blocks = static_cast<unsigned>((T + p.block_rows - 1) / p.block_rows);
  return launch_dependent(dtype == MLA_BF16 ? fp4::append_fp4_kernel<true> : fp4::append_fp4_kernel<false>, p, dim3(blocks, 2),
                          fp4::kThreads, 0, stream);
}

}  // extern "C"
