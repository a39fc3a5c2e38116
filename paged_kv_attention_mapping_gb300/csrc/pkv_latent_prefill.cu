// Expanded latent attention of chunks: head h of row i of a sequence, with
// query [qn, qr], attends keys [kn_j, r_j] (r shared by the heads) and values v_j:
//   s_j = scale (qn . kn_j + qr . r_j),  j <= kv_len - q_len + i,
//   out = sum_j softmax(s)_j v_j.
// One warp per (row, head), one pass over the keys.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int NOPE = 128, ROPE = 64, DV = 128;

struct PrefillP {
  int64_t kn_st, kn_sh, v_st, v_sh, kr_st;
  const int32_t *cu_q, *cu_k;
  int32_t B, Tq, Tk, H;
  float scale_log2;
  float* lse;
  int32_t* dev_status;
};

template <typename T>
__global__ void __launch_bounds__(256) latent_prefill_rows_kernel(const T* __restrict__ q, const T* __restrict__ kn,
                                                                  const T* __restrict__ v, const T* __restrict__ kr,
                                                                  T* __restrict__ out, PrefillP p) {
  bool bad = threadIdx.x == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_k) != 0);
  for (int b = threadIdx.x; b < p.B; b += blockDim.x)
    bad |= __ldg(p.cu_q + b + 1) < __ldg(p.cu_q + b) || __ldg(p.cu_k + b + 1) < __ldg(p.cu_k + b);
  const int n = __ldg(p.cu_q + p.B);
  bad |= n > p.Tq || __ldg(p.cu_k + p.B) > p.Tk;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = row / p.H;
  const int h = (int)(row - t * p.H);
  if (t >= n) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu_q + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int c0 = __ldg(p.cu_q + lo), qlen = __ldg(p.cu_q + lo + 1) - c0;
  const int k0 = __ldg(p.cu_k + lo), L = __ldg(p.cu_k + lo + 1) - k0;
  if (L < qlen) {
    if (lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int keys = L - qlen + (int)(t - c0) + 1;
  float qn[4], qr[2], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) qn[k] = to_f32(q[row * (NOPE + ROPE) + k * 32 + lane]);
#pragma unroll
  for (int k = 0; k < 2; ++k) qr[k] = to_f32(q[row * (NOPE + ROPE) + NOPE + k * 32 + lane]);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < keys; ++j) {
    const T* x = kn + (int64_t)(k0 + j) * p.kn_st + h * p.kn_sh;
    const T* y = kr + (int64_t)(k0 + j) * p.kr_st;
    const T* z = v + (int64_t)(k0 + j) * p.v_st + h * p.v_sh;
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) dot += qn[k] * to_f32(x[k * 32 + lane]);
#pragma unroll
    for (int k = 0; k < 2; ++k) dot += qr[k] * to_f32(y[k * 32 + lane]);
    const float sc = warp_sum(dot) * p.scale_log2;
    const float mn = fmaxf(m, sc), w = exp2f(sc - mn), f = exp2f(m - mn);
    l = l * f + w;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = o[k] * f + w * to_f32(z[k * 32 + lane]);
    m = mn;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k) out[row * DV + k * 32 + lane] = from_f32<T>(o[k] * inv);
  if (p.lse && lane == 0) p.lse[row] = (m + log2f(l)) * LN2;
}

template <typename T>
cudaError_t launch(const LatentPrefillArgs& a, cudaStream_t s) {
  PrefillP p{a.kn_st, a.kn_sh, a.v_st, a.v_sh, a.kr_st, a.cu_q, a.cu_k, a.B, a.Tq, a.Tk, a.H, a.scale * LOG2E,
             a.lse, a.dev.status};
  const int64_t rows = (int64_t)a.Tq * a.H;
  KernelTimer timer("latent_prefill_rows", s);
  latent_prefill_rows_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(
      (const T*)a.q, (const T*)a.kn, (const T*)a.v, (const T*)a.kr, (T*)a.out, p);
  return cudaGetLastError();
}

}  // namespace

size_t latent_prefill_workspace(int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t s) {
  return a.dtype == PKV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace pkv
