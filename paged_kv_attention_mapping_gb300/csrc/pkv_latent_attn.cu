// Absorbed latent attention over the paged latent cache: for row (token i of
// sequence b, head h) with query q, and cached rows x_j = [c_j, r_j],
//   s_j = scale q . x_j,  j <= kv_len - q_len + i,
//   out = sum_j exp(s_j - m) c_j / sum_j exp(s_j - m),  lse = m + ln(sum).
// One warp per row, one pass over the keys with the running maximum and sum.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct AttnP {
  const int32_t *cu, *kv_lens, *page_tables;
  int32_t B, T, H, P, num_pages, max_pages, max_kv_len;
  float scale_log2;
  float* lse;
  int32_t* dev_status;
};

template <int LD, typename T>
__global__ void __launch_bounds__(256) latent_rows_kernel(const T* __restrict__ q, const T* __restrict__ cache,
                                                          T* __restrict__ out, AttnP p) {
  constexpr int D = LD + 64, NC = LD / 32;
  bool bad = threadIdx.x == 0 && __ldg(p.cu) != 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) bad |= __ldg(p.cu + b + 1) < __ldg(p.cu + b);
  const int n = __ldg(p.cu + p.B);
  bad |= n > p.T;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int64_t t = row / p.H;
  if (t >= n) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int c0 = __ldg(p.cu + lo), qlen = __ldg(p.cu + lo + 1) - c0, L = __ldg(p.kv_lens + lo);
  if (L < qlen || L < 1 || L > p.max_kv_len || L > (int64_t)p.max_pages * p.P) {
    if (lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int keys = L - qlen + (int)(t - c0) + 1;
  const int32_t* pt = p.page_tables + (int64_t)lo * p.max_pages;
  for (int k = 0; k * (int64_t)p.P < keys; ++k) {
    const int id = __ldg(pt + k);
    if (id < 0 || id >= p.num_pages) {
      if (lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_PAGE);
      return;
    }
  }
  float qc[NC], qr[2], o[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    qc[k] = to_f32(q[row * D + k * 32 + lane]);
    o[k] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) qr[k] = to_f32(q[row * D + LD + k * 32 + lane]);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < keys; ++j) {
    const T* x = cache + ((int64_t)__ldg(pt + j / p.P) * p.P + j % p.P) * D;
    float xc[NC], dot = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      xc[k] = to_f32(x[k * 32 + lane]);
      dot += qc[k] * xc[k];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) dot += qr[k] * to_f32(x[LD + k * 32 + lane]);
    const float sc = warp_sum(dot) * p.scale_log2;
    const float mn = fmaxf(m, sc), w = exp2f(sc - mn), f = exp2f(m - mn);
    l = l * f + w;
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = o[k] * f + w * xc[k];
    m = mn;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int k = 0; k < NC; ++k) out[row * LD + k * 32 + lane] = from_f32<T>(o[k] * inv);
  if (p.lse && lane == 0) p.lse[row] = (m + log2f(l)) * LN2;
}

template <int LD, typename T>
cudaError_t launch(const LatentAttnArgs& a, cudaStream_t s) {
  AttnP p{a.cu, a.kv_lens, a.page_tables, a.B, a.T, a.H, a.P, a.num_pages, a.max_pages, a.max_kv_len,
          a.scale * LOG2E, a.lse, a.dev.status};
  const int64_t rows = (int64_t)a.T * a.H;
  KernelTimer timer("latent_rows", s);
  latent_rows_kernel<LD, T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>((const T*)a.q, (const T*)a.cache, (T*)a.out, p);
  return cudaGetLastError();
}

}  // namespace

size_t latent_attn_workspace(int32_t, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_latent_attn(const LatentAttnArgs& a, cudaStream_t s) {
  if (a.dtype == PKV_BF16)
    return a.latent_dim == 512 ? launch<512, __nv_bfloat16>(a, s) : launch<256, __nv_bfloat16>(a, s);
  return a.latent_dim == 512 ? launch<512, __half>(a, s) : launch<256, __half>(a, s);
}

}  // namespace pkv
