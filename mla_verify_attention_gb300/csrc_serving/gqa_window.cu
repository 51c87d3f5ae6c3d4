// The attention kernel with a sliding window and first tokens that stay visible.
#include "gqa_attn.cuh"
#include "gqa_host.h"

namespace mla {
namespace gqa {

AttnFn window_kernel(int D, bool bf16) {
  if (D == 128) return bf16 ? attn_kernel<128, true, kWindow> : attn_kernel<128, false, kWindow>;
  return bf16 ? attn_kernel<64, true, kWindow> : attn_kernel<64, false, kWindow>;
}

}  // namespace gqa
}  // namespace mla
