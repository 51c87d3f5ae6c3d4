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

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace mla
