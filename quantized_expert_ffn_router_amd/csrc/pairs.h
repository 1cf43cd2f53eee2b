// pairs.h -- 16-bit values two to a word, and numbered pieces of code: what the attention,
// norm and product kernels share.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

// The two bf16 values of a word, and two values as bf16, rounded to nearest even.
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  const v2b r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// f of the numbers I .. N - 1, each as a type: where more code depends on the number than a
// loop's unrolling takes.
template <int I, int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<I + 1, N>(f);
  }
}

}  // namespace moe
