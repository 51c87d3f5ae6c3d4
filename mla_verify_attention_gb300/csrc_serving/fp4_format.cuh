// Rows of a cache held in 4 bits.  A row of Hkv heads x D values is
//   Hkv * D / 2 bytes of codes (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
//     negatives), heads in order, dimension 2 i in the low half of byte i;
//   Hkv * D / 16 bytes of steps (E4M3), one for every 16 values of a head;
//   padding up to a multiple of 16 bytes, without a meaning and never written;
// value = (E2M1 of the code) * step * the pool's own factor.  A step and a code
// have 4 and 2 significant bits, so their product is exact in fp16 (2^-10 .. 2,688).
#pragma once
#include <cstdint>

namespace mla {
namespace fp4 {

constexpr int kGroup = 16;                 // values a step

__host__ __device__ constexpr int code_bytes(int Hkv, int D) { return Hkv * (D / 2); }
__host__ __device__ constexpr int row_bytes(int Hkv, int D) {
  return (Hkv * (D / 2 + D / kGroup) + 15) / 16 * 16;
}

// Factors of a pool for which no step's product or reciprocal leaves fp32's normal range.
inline bool factor_ok(float f) { return f >= 5.421010862427522e-20f && f <= 1.8446744073709552e19f; }   // 2^-64 .. 2^64

// The nearest step at or below 448 (NaN stays one), and its value.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
// Two steps' values, fp16.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// Eight values, in steps, to codes: x[0] in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
// Eight codes to fp16 pairs.
__device__ __forceinline__ void from_e2m1x8(uint32_t codes, uint32_t* h) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

}  // namespace fp4
}  // namespace mla
