// The attention kernel's forms that are compiled in translation units of their
// own, so that they compile side by side.
#pragma once
#include <cuda.h>

namespace mla {
namespace gqa {

struct Params;
using AttnFn = void (*)(CUtensorMap, CUtensorMap, Params);

AttnFn window_kernel(int D, bool bf16);    // gqa_window.cu

}  // namespace gqa
}  // namespace mla
