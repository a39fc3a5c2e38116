// Pages copied between places of their pools (forks copy a sequence's partly filled
// last page, compaction moves pages to lower ids), and page tables rewritten for
// pages that have moved.
//
// A copy only moves bytes, 2 x page_size x slot_bytes a page and cache, so the bound
// is HBM. One launch serves up to MAX_CACHES caches (all layers' keys and values): their
// addresses travel as kernel arguments, so the call needs no device array of them. 112 pages of 512 KB in
// 16 caches take 270 us, 6.9 TB/s; 24 partly filled pages of 8 KB in 44 caches 3.1 us.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;                          // 16-byte loads in flight a thread
constexpr int PIECE = THREADS * UNROLL;            // 16-byte vectors a block copies
constexpr int MAX_CACHES = 256;

struct CopyP {
  uint4* cache[MAX_CACHES];
  const int32_t *src, *dst, *tokens;
  int64_t slot_vecs;   // 16-byte vectors of a slot
  int32_t num_caches, num_pages, page_size, pieces;   // pieces: blocks a page takes
  int32_t* dev_status;
};

__global__ void __launch_bounds__(THREADS) copy_pages_kernel(const __grid_constant__ CopyP p) {
  pdl_wait();
  pdl_trigger();   // what starts now waits for this grid's end before it writes, and before it relies on what it read
  const int per_copy = p.num_caches * p.pieces;
  const int i = blockIdx.x / per_copy;
  const int r = blockIdx.x - i * per_copy;
  const int c = r / p.pieces, piece = r - c * p.pieces;
  const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
  const int n = p.tokens ? __ldg(p.tokens + i) : p.page_size;
  if (from < 0 || to < 0) return;
  if (from >= p.num_pages || to >= p.num_pages || n < 0 || n > p.page_size) {
    if (r == 0 && threadIdx.x == 0)
      atomicOr(p.dev_status, n < 0 || n > p.page_size ? PKV_DEV_BAD_LENGTHS : PKV_DEV_BAD_PAGE);
    return;
  }
  if (from == to) return;
  const int64_t page = p.page_size * p.slot_vecs, end = n * p.slot_vecs;
  const uint4* a = p.cache[c] + from * page;
  uint4* b = p.cache[c] + to * page;
  const int64_t v0 = (int64_t)piece * PIECE + threadIdx.x;
  uint4 x[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k)
    if (v0 + k * THREADS < end) x[k] = a[v0 + k * THREADS];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k)
    if (v0 + k * THREADS < end) b[v0 + k * THREADS] = x[k];
}

__global__ void __launch_bounds__(THREADS) remap_pages_kernel(int32_t* tables, int64_t n,
                                                              const int32_t* __restrict__ map, int32_t num_pages,
                                                              int32_t* dev_status) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS) {
    const int32_t page = tables[i];
    if (page < 0) continue;
    const int32_t to = page < num_pages ? __ldg(map + page) : num_pages;
    if (to >= num_pages) atomicOr(dev_status, PKV_DEV_BAD_PAGE);
    else if (to != page) tables[i] = to;
  }
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesArgs& a, cudaStream_t s) {
  CopyP p;
  p.src = a.src;
  p.dst = a.dst;
  p.tokens = a.tokens;
  p.slot_vecs = a.slot_bytes / 16;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.dev_status = a.dev_status;
  const int64_t pieces = (a.page_size * p.slot_vecs + PIECE - 1) / PIECE;
  if (pieces > INT32_MAX / MAX_CACHES) return cudaErrorInvalidValue;
  p.pieces = (int32_t)pieces;
  KernelTimer timer("copy_pages", s);
  for (int32_t c0 = 0; c0 < a.num_caches; c0 += MAX_CACHES) {
    p.num_caches = a.num_caches - c0 < MAX_CACHES ? a.num_caches - c0 : MAX_CACHES;
    for (int32_t c = 0; c < p.num_caches; ++c) p.cache[c] = (uint4*)a.caches[c0 + c];
    const int64_t per_copy = pieces * p.num_caches;
    const int64_t most = INT32_MAX / per_copy;   // copies of one launch
    for (int64_t i0 = 0; i0 < a.num_copies; i0 += most) {
      const int64_t n = a.num_copies - i0 < most ? a.num_copies - i0 : most;
      p.src = a.src + i0;
      p.dst = a.dst + i0;
      p.tokens = a.tokens ? a.tokens + i0 : nullptr;
      const cudaError_t e =
          launch_after_trigger(copy_pages_kernel, dim3((unsigned)(n * per_copy)), dim3(THREADS), 0, s, p);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_remap_pages(int32_t* tables, int64_t n, const int32_t* map, int32_t num_pages,
                               const DeviceView& dev, cudaStream_t s) {
  KernelTimer timer("remap_pages", s);
  const int64_t want = (n + THREADS - 1) / THREADS, most = (int64_t)dev.num_sms * 8;
  return launch_after_trigger(remap_pages_kernel, dim3((unsigned)(want < most ? want : most)), dim3(THREADS), 0, s,
                              tables, n, map, num_pages, dev.status);
}

}  // namespace pkv
