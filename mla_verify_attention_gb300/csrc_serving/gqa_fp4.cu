// The attention kernel over a cache held in 4 bits.
#include "gqa_attn.cuh"
#include "gqa_host.h"

namespace mla {
namespace gqa {

template <int D>
Fp4Fn pick_fp4(bool bf16, size_t* smem, int* threads) {
  static_assert(sizeof(Smem<D, kFp4>) <= 232448, "one CTA's shared memory");
  *smem = sizeof(Smem<D, kFp4>);
  *threads = Shape<D, kFp4>::kThreads;
  return bf16 ? attn_fp4_kernel<D, true> : attn_fp4_kernel<D, false>;
}

Fp4Fn fp4_kernel(int D, bool bf16, size_t* smem, int* threads) {
  return D == 128 ? pick_fp4<128>(bf16, smem, threads) : pick_fp4<64>(bf16, smem, threads);
}

}  // namespace gqa
}  // namespace mla
