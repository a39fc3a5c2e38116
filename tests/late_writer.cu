// Test helper: a kernel that lets the next kernel of its stream start at once and
// only some time later writes its results, as a user's own kernel may with
// programmatic launches. What follows it in the stream must see those results.
#include <cuda_runtime.h>
#include <stdint.h>

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__global__ void late_write_kernel(const uint32_t* __restrict__ src, uint32_t* __restrict__ dst, int64_t words,
                                  uint32_t delay_ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint64_t t0 = now_ns();
  for (int it = 0; it < (1 << 20) && now_ns() - t0 < delay_ns; ++it) {}
  for (int64_t i = threadIdx.x; i < words; i += blockDim.x) dst[i] = src[i];
}

// Copies `words` 32-bit words from src to dst (device memory) on `stream`, delay_us
// microseconds after its start (at most 1000). Returns the launch's cudaError_t.
extern "C" int late_write(const void* src, void* dst, int64_t words, uint32_t delay_us, void* stream) {
  if (words < 0 || delay_us > 1000) return (int)cudaErrorInvalidValue;
  late_write_kernel<<<1, 256, 0, (cudaStream_t)stream>>>((const uint32_t*)src, (uint32_t*)dst, words, delay_us * 1000u);
  return (int)cudaGetLastError();
}
