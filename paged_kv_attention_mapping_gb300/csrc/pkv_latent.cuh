// Device helpers shared by the latent-attention kernels.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b, c) in one instruction (sm_100 family); exact, like two fmaxf.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// A whole 32-byte sector (p 32-byte aligned).
__device__ __forceinline__ void st_global_32B(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Softmax weights are rounded to the cache type T for their product with the values: a
// relative half step. fp16 has no more than half a step of 2^-24 below 2^-14 though, and many
// small weights beside a large one would be lost in O but not in the row's sum. So weights and sums
// carry a factor 2^SHIFT, near fp16's range: a weight of 2^-w of the row's scale stays normal
// up to w = 14 + SHIFT. It cancels in O / l; a log sum gives it back. `most`: log2 of the
// largest weight without it (7 of 15 bits are left where a row's scale may lag by 2^8).
template <typename T>
__device__ __forceinline__ constexpr float weight_shift(float most) {
  return std::is_same<T, __nv_bfloat16>::value ? 0.f : 15.f - most;
}

// Two fp32 values rounded to the 16-bit type T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

}  // namespace pkv
