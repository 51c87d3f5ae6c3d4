// What the library's translation units share and its users do not see: the
// device's status word and the values every entry point needs.  Defined in
// csrc/mla_verify_attn.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

namespace mla {

// Bits of the per-device status word (mla_verify_attn_last_device_error).
enum : uint32_t {
  kBitSeqLen = 1u,
  kBitTimeout = 2u,
  kBitPage = 4u,
  kBitPool = 8u,
  kBitSlot = 16u,
};

struct DeviceCommon {
  int sms;
  unsigned int* status_word;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  int test_stall;             // mla_verify_attn_set_test_controls
};

// The current device's values, or a negative mla_status.
int device_common(DeviceCommon* out);

// Quotients by a number fixed for the call: exact for 0 <= n < 2^31, as one
// 64-bit product.  With 2^s >= d and m = floor(2^(31 + s) / d) + 1, m d exceeds
// 2^(31 + s) by at most 2^s, which moves n m / 2^(31 + s) by less than 1 / d.
struct Divisor {
  unsigned d, m;
  int shift;
  Divisor() = default;
  explicit Divisor(int by) : d(static_cast<unsigned>(by)), shift(31) {
    while ((1ull << (shift - 31)) < d) ++shift;
    m = static_cast<unsigned>((1ull << shift) / d + 1);
  }
  __device__ __forceinline__ int of(int n) const {
    return d == 1 ? n : static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(n)) * m >> shift);
  }
  __device__ __forceinline__ int up(int n) const { return n > 0 ? of(n - 1) + 1 : 0; }   // rounded up
};

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace mla
