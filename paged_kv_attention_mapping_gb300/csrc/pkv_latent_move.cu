// Moving rows into and out of a latent cache: the append (new tokens' latents
// and rotated keys into their slots, queries rotated) and the gather (cached
// rows of every sequence into one packed tensor).
//
// Both only move bytes, so the bound is HBM: 4 (latent_dim + 64) bytes per row
// moved, 4 * 64 more per query head that the append rotates. Rows are taken as
// 16-byte vectors, consecutive threads on consecutive vectors.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;
constexpr int ROPE = 64;          // rotary part of a row
constexpr int RV = ROPE / 2 / 8;  // rotation items of a rotary part: 8 pairs each

struct AppendP {
  int64_t c_st, kr_st, q_st, q_sh, qo_st, qo_sh, pool_slots, items;
  const int32_t* positions;
  const float4* cs;   // (cos, sin) pairs, two per vector: ROPE / 4 vectors a position
  const int64_t* slots;
  int32_t max_pos, copy_vecs, per_token, row;   // row: latent_dim + ROPE
  int32_t* dev_status;
};

// One rotation of 8 pairs: (u, w) -> (u cos - w sin, w cos + u sin), in fp32,
// rounded once to the cache type.
template <typename T>
__device__ __forceinline__ void rotate8(uint4 x1, uint4 x2, const float4* __restrict__ cs, uint4* o1, uint4* o2) {
  const T* u = reinterpret_cast<const T*>(&x1);
  const T* w = reinterpret_cast<const T*>(&x2);
  T* y1 = reinterpret_cast<T*>(o1);
  T* y2 = reinterpret_cast<T*>(o2);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float4 c = __ldg(cs + e / 2);
    const float a0 = to_f32(u[e]), b0 = to_f32(w[e]), a1 = to_f32(u[e + 1]), b1 = to_f32(w[e + 1]);
    y1[e] = from_f32<T>(a0 * c.x - b0 * c.y);
    y2[e] = from_f32<T>(b0 * c.x + a0 * c.y);
    y1[e + 1] = from_f32<T>(a1 * c.z - b1 * c.w);
    y2[e + 1] = from_f32<T>(b1 * c.z + a1 * c.w);
  }
}

// A token's items, in order: its latent part as copy_vecs vectors, the RV
// rotation items of its key part, RV for each query head. A thread takes one
// item: its data loads go out before the position and slot that decide what
// becomes of them. 8192 tokens at 16 heads (f16): 12.5 us, 4.4 TB/s, the start-up of
// a grid of this length included; 2 / 3 / 4 items a thread took 13.6 / 15.3 / 14.6.
template <typename T>
__global__ void __launch_bounds__(THREADS) latent_append_kernel(const T* __restrict__ c, const T* __restrict__ kr,
                                                                const T* q, T* q_out, T* __restrict__ cache,
                                                                AppendP p) {
  pdl_wait();
  pdl_trigger();   // what starts now waits for this grid's end before it writes, and before it relies on what it read
  const int64_t j = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  if (j >= p.items) return;
  const int64_t t = j / p.per_token;
  int r = (int)(j - t * p.per_token);
  const bool copy = r < p.copy_vecs;
  const bool key = !copy && r < p.copy_vecs + RV;
  uint4 x1, x2 = make_uint4(0, 0, 0, 0);
  T* dst = nullptr;
  int a = 0;
  if (copy) {
    x1 = *reinterpret_cast<const uint4*>(c + t * p.c_st + r * 8);
  } else {
    const int rr = r - p.copy_vecs;
    a = (rr % RV) * 8;
    const int h = rr / RV - 1;   // -1: the key
    const T* src = key ? kr + t * p.kr_st : q + t * p.q_st + h * p.q_sh;
    x1 = *reinterpret_cast<const uint4*>(src + a);
    x2 = *reinterpret_cast<const uint4*>(src + a + ROPE / 2);
    if (!key) dst = q_out + t * p.qo_st + h * p.qo_sh + a;
  }
  const int pos = __ldg(p.positions + t);
  if (pos < 0 || pos >= p.max_pos) {
    if (r == 0) atomicOr(p.dev_status, PKV_DEV_BAD_POSITION);
    return;
  }
  if (copy || key) {
    const int64_t slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= p.pool_slots) {
      if (r == 0) atomicOr(p.dev_status, PKV_DEV_BAD_SLOT);
      return;
    }
    dst = cache + slot * p.row + (copy ? r * 8 : p.copy_vecs * 8 + a);
  }
  if (copy) {
    *reinterpret_cast<uint4*>(dst) = x1;
  } else {
    uint4 o1, o2;
    rotate8<T>(x1, x2, p.cs + (int64_t)pos * (ROPE / 4) + a / 2, &o1, &o2);
    *reinterpret_cast<uint4*>(dst) = o1;
    *reinterpret_cast<uint4*>(dst + ROPE / 2) = o2;
  }
}

// A block takes R consecutive packed rows (107 k rows of 1152 bytes: 38.8 us, 6.3
// TB/s; 1 to 2 us more with 8 or 32 rows a block). Its threads first check cu_seqlens
// (every block does, so that a bad array copies nothing), then one thread per
// row finds the row's sequence and slot, then all copy.
template <int R>
__global__ void __launch_bounds__(THREADS) latent_gather_kernel(const uint4* __restrict__ cache,
                                                                const int32_t* __restrict__ tables,
                                                                const int32_t* __restrict__ cu, int32_t B,
                                                                int32_t total, int32_t max_pages, int32_t P,
                                                                int32_t num_pages, int32_t row_vecs,
                                                                uint4* __restrict__ out, int32_t* dev_status) {
  __shared__ int64_t s_src[R];
  const int tid = threadIdx.x;
  pdl_wait();
  bool bad = tid == 0 && __ldg(cu) != 0;
  for (int b = tid; b < B; b += THREADS) bad |= __ldg(cu + b + 1) < __ldg(cu + b);
  const int n = __ldg(cu + B);
  bad |= n > total;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int64_t row0 = (int64_t)blockIdx.x * R;
  if (row0 >= n) return;
  if (tid < R) {
    const int64_t t = row0 + tid;
    int64_t src = -1;
    if (t < n) {
      int lo = 0, hi = B - 1;   // the last sequence that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
      }
      const int c0 = __ldg(cu + lo);
      const int len = __ldg(cu + lo + 1) - c0;
      const int pos = (int)t - c0, page = pos / P;
      if (len > (int64_t)max_pages * P) {
        if (pos == 0) atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
      } else {
        const int id = __ldg(tables + (int64_t)lo * max_pages + page);
        if (id < 0 || id >= num_pages) atomicOr(dev_status, PKV_DEV_BAD_PAGE);
        else src = ((int64_t)id * P + (pos - page * P)) * row_vecs;
      }
    }
    s_src[tid] = src;
  }
  __syncthreads();
  const int span = R * row_vecs;
  constexpr int U = 5;   // loads in flight per thread before their stores
  for (int base = tid; base < span; base += THREADS * U) {
    uint4 x[U];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + u * THREADS;
      have[u] = false;
      if (j < span) {
        const int r = j / row_vecs;
        const int64_t src = s_src[r];
        if (src >= 0) {
          x[u] = __ldg(cache + src + (j - r * row_vecs));
          have[u] = true;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (have[u]) out[row0 * row_vecs + base + u * THREADS] = x[u];
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t s) {
  AppendP p;
  p.c_st = a.c_st;
  p.kr_st = a.kr_st;
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.qo_st = a.qo_st;
  p.qo_sh = a.qo_sh;
  p.pool_slots = a.pool_slots;
  p.positions = a.positions;
  p.cs = (const float4*)a.cos_sin;
  p.slots = a.slots;
  p.max_pos = a.max_pos;
  p.copy_vecs = a.latent_dim / 8;
  p.per_token = p.copy_vecs + RV * (1 + a.Hq);
  p.items = (int64_t)a.T * p.per_token;
  p.row = a.latent_dim + a.rope_dim;
  p.dev_status = a.dev_status;
  const int64_t blocks = (p.items + THREADS - 1) / THREADS;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  KernelTimer timer("latent_append", s);
  if (a.dtype == PKV_F16)
    return launch_after_trigger(latent_append_kernel<__half>, dim3((unsigned)blocks), dim3(THREADS), 0, s,
                                (const __half*)a.c, (const __half*)a.kr, (const __half*)a.q, (__half*)a.q_out,
                                (__half*)a.cache, p);
  return launch_after_trigger(latent_append_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(THREADS), 0, s,
                              (const __nv_bfloat16*)a.c, (const __nv_bfloat16*)a.kr, (const __nv_bfloat16*)a.q,
                              (__nv_bfloat16*)a.q_out, (__nv_bfloat16*)a.cache, p);
}

cudaError_t launch_latent_gather(const LatentGatherArgs& a, cudaStream_t s) {
  KernelTimer timer("latent_gather", s);
  constexpr int R = 16;
  const unsigned blocks = (unsigned)((a.total + (int64_t)R - 1) / R);
  return launch_after_trigger(latent_gather_kernel<R>, dim3(blocks), dim3(THREADS), 0, s, (const uint4*)a.cache,
                              a.page_tables, a.cu, a.B, a.total, a.max_pages, a.P, a.num_pages, a.row_vecs,
                              (uint4*)a.out, a.dev_status);
}

}  // namespace pkv
