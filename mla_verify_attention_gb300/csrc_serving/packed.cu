// mla_call_packed: the serving calls with their arguments in one array.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "mla_verify_attn.h"

namespace {

// One argument from its 64-bit value; `fits` becomes false where it is too large.
template <class T>
T unpack(int64_t v, bool& fits) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(v));
  } else if constexpr (std::is_same_v<T, float>) {
    double d;
    std::memcpy(&d, &v, sizeof d);
    return static_cast<float>(d);
  } else {
    if constexpr (sizeof(T) < sizeof v) fits = fits && v >= INT_MIN && v <= INT_MAX;
    return static_cast<T>(v);
  }
}

template <class... A, size_t... I>
int call_with(int (*fn)(A...), const int64_t* a, std::index_sequence<I...>) {
  bool fits = true;
  std::tuple<A...> args{unpack<A>(a[I], fits)...};
  return fits ? std::apply(fn, args) : MLA_ERR_SHAPE;
}
template <class... A>
int call(int (*fn)(A...), const int64_t* a) {
  return call_with(fn, a, std::index_sequence_for<A...>{});
}

}  // namespace

extern "C" int mla_call_packed(int which, const int64_t* args) {
  if (!args) return MLA_ERR_NULLPTR;
  switch (which) {
    case MLA_CALL_BLOCKS_EXTEND: return call(mla_blocks_extend, args);
    case MLA_CALL_BLOCKS_TRIM: return call(mla_blocks_trim, args);
    case MLA_CALL_CACHE_APPEND: return call(mla_cache_append, args);
    case MLA_CALL_CACHE_KEEP: return call(mla_cache_keep, args);
    case MLA_CALL_GQA_VERIFY_ATTN: return call(mla_gqa_verify_attn, args);
    case MLA_CALL_GQA_VERIFY_ATTN_PAGED: return call(mla_gqa_verify_attn_paged, args);
    default: return MLA_ERR_ARG;
  }
}
