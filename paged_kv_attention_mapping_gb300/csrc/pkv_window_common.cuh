// What the window-attention kernels share: which sequence a piece of work belongs to,
// which keys its rows see, and where a key's row lies in the pages.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace window {

// Division of 0 .. 2^31 - 1 by a page size: the high word of a product, shifted.
struct PageDiv {
  uint32_t mul, shift, one;   // one: the page size is 1
};
inline PageDiv page_div(int32_t P) {
  PageDiv d{0, 0, P == 1 ? 1u : 0u};
  if (P > 1) {
    int l = 0;
    while (((int64_t)1 << l) < P) ++l;
    d.mul = (uint32_t)((((uint64_t)1 << (31 + l)) / (uint32_t)P) + 1);
    d.shift = (uint32_t)(l - 1);
  }
  return d;
}
__device__ __forceinline__ int page_of(int key, const PageDiv& d) {
  return d.one ? key : (int)(__umulhi((uint32_t)key, d.mul) >> d.shift);
}

// Work is numbered without a plan: piece `slot` of the call belongs to the last
// sequence b with first(b) <= slot, where a piece is up to `per` rows of one sequence and
// first(b) = b + cu[b] / per. Sequence b of q rows then has the numbers first(b) ..
// first(b) + ceil(q / per) - 1, all below first(b + 1), and the highest number is below
// B + T / per. With per == 1 a piece is a packed row, and first(b) = cu[b].
__device__ __forceinline__ int64_t first_piece(int b, int c, int per) {
  return per == 1 ? (int64_t)c : (int64_t)b + c / per;
}

// The sequence of a piece, found by a whole warp: 32 probes a round. `guess` is tried first
// (in a tick of single rows, packed row r is sequence r).
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int B, int64_t slot, int per, int lane) {
  int lo = 0, hi = B;   // the answer is in [lo, hi)
  if (slot < B) {
    const int g = (int)slot;
    const int c0 = __ldg(cu + g), c1 = __ldg(cu + g + 1);
    if (first_piece(g, c0, per) <= slot && slot < first_piece(g + 1, c1, per)) return g;
  }
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const bool below = b < hi && first_piece(b, __ldg(cu + b), per) <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int last = m ? 31 - __clz(m) : 0;   // (lane 0 holds when cu[0] is 0)
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The keys that rows at positions p_first .. p_last see together: [0, sinks) and
// [lo, p_last], numbered 0 .. n - 1 without the gap between them.
struct Keys {
  int lo, sinks, n;
};
__device__ __forceinline__ Keys keys_of(int p_first, int p_last, int window, int sinks) {
  Keys k;
  k.lo = max(0, p_first - window + 1);
  k.sinks = min(sinks, k.lo);
  k.n = k.sinks + (p_last + 1 - k.lo);
  return k;
}
__device__ __forceinline__ int key_at(const Keys& k, int i) { return i < k.sinks ? i : i - k.sinks + k.lo; }

__device__ __forceinline__ bool seen(int key, int p, int window, int sinks) {
  return key <= p && (key > p - window || key < sinks);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values rounded to 16 bits, the first in the low half. (Softmax weights go through it: the tensor cores multiply
// 16-bit values by 16-bit weights. Their sum is of the weights as they were; with the rounded ones' sum the outputs'
// error against 64 bits is the same to 2 %, as each rounding goes its own way.)
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Two e4m3 codes (the low 16 bits) as two f16 values: exact.
__device__ __forceinline__ uint32_t widen(uint32_t codes) {
  uint32_t out;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(out) : "h"((uint16_t)codes));
  return out;
}

// Flags a cu_seqlens_q that does not start at 0, decreases or ends beyond T. One block
// of the call looks at all of it; the others check only what they use.
__device__ __forceinline__ void check_cu(const int32_t* __restrict__ cu, int B, int T, int32_t* dev_status) {
  bool bad = threadIdx.x == 0 && __ldg(cu) != 0;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int c1 = __ldg(cu + b + 1);
    bad |= c1 < __ldg(cu + b) || c1 > T;
  }
  if (bad) atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
}

}  // namespace window
}  // namespace pkv
