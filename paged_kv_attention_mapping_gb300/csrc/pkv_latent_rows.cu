// Absorbed latent attention for ticks with few rows a sequence (heads x new tokens
// at most 16 on average: decode with the heads of one shard). Same problem and same
// split of the tick as pkv_latent_attn.cu; here a work tile is 16 (token, head)
// rows, a step 64 keys, a worker one CTA.
//
// At 16 rows a key's 1152 bytes carry 35 kFLOP: HBM is the bound, and what counts
// is to keep its reads in flight. The tcgen05 kernel spends its shared memory on 128
// query rows, most of them absent here, and a long chain of hand-offs per step; this
// one uses warp-level mma.sync (m16n8k16) with the queries in registers, so that
// 180 KB of a CTA are key rows on their way, and every row serves the scores and the
// output from the same place. Decode of 96 sequences of 64-16384 keys at 16 heads
// (f16): 132 us for this kernel, 6.4 TB/s (174 us with the tcgen05 one).
//
//   warps 0-7  all of a step: the scores of 32 keys over a quarter of the columns
//              (partial sums joined through shared memory), the softmax of two
//              rows (weights rounded to the cache type, the other operand's: half a step of
//              each; sums stay fp32), then LD / 8 columns of O
//   warp 8     scheduler: the segments of this CTA
//   warp 9     producer (TMA): 32-key slots of a ring, 128-byte swizzled; for small boxes
//              (cp.async) several warps, slots in turn
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_latent.cuh"
#include "pkv_latent_sched.cuh"
#include "pkv_sm100.cuh"

namespace pkv {
using namespace sm100;

namespace {

constexpr int TM = 16;           // rows of a tile
constexpr int BN = 64;           // keys of a step
constexpr int HB = 32;           // keys of a ring slot
// What a tile counts beside its steps in the split. Decode of 96 sequences of 64-16384 keys at
// 16 heads with 0 / 1 / 2 / 3 / 4: 139.6 / 137.1 / 135.9 / 136.4 / 136.6 us.
constexpr int START = 2;
constexpr int MAX_CTAS = 152;    // SMs of the device; the workspace is laid out for these
constexpr int WARPS = 8;         // compute warps
// Warps that copy rows where TMA does not, slots in turn. 64 sequences of 1000-4000 keys at 16
// heads with 1 / 2 / 3 / 4: pages of 16 50.2 / 45.4 / 45.4 / 51 us, of 8 57.5 / 47.6 / 46.3 / 51.5, of
// 1 65.5 / 55.5 / 50.6 / 52.5 (by TMA, pages of 32 and more: 45.1).
constexpr int G_PRODUCERS = 3;
constexpr int producers(bool gather) { return gather ? G_PRODUCERS : 1; }
constexpr int nthreads(bool gather) { return (WARPS + 1 + producers(gather)) * 32; }
constexpr uint32_t UNIT = HB * 128;   // 32 rows x 64 columns of 16 bits
constexpr int NSEG = 4;
constexpr int S_LD = 72;         // floats between rows of the partial scores (no bank conflicts)
constexpr long long WAIT_LIMIT_CLOCKS = 4000000000ll;   // about two seconds

template <int LD>
struct Cfg {
  static constexpr int CH = LD / 64 + 1;                 // 64-column units of a row, the rotary one last
  static constexpr int KS = (LD + 64) / 16 / 4;          // 16-column steps of a quarter of the columns
  static constexpr int DW = LD / WARPS;                  // output columns of a warp
  static constexpr int NS = LD == 512 ? 5 : 9;           // ring slots
  static constexpr uint32_t SLOT = CH * UNIT;
  static constexpr uint32_t RING = NS * SLOT;
};

template <int LD, int NTHREADS>
struct State {
  uint64_t full[Cfg<LD>::NS], empty[Cfg<LD>::NS], segfull[NSEG], segempty[NSEG];
  LatentPlan<NTHREADS> plan;
  LatentSegment seg[NSEG];
  int bad[NSEG];
  int abort;
  float alpha[TM], m[TM], l[TM];
  alignas(16) float s[4][TM][S_LD];                      // scores, by quarter of the columns
  alignas(128) unsigned char p[TM * 128];                // weights in the cache type, swizzled
};

// Workspace: a record per CTA, then a bad flag, log2 sums and outputs (fp32,
// normalised) for two partial results per CTA.
struct Layout {
  static constexpr size_t rec = 0;
  static constexpr size_t bad = 4096;
  static constexpr size_t lse = 8192;
  static constexpr size_t o = lse + (size_t)2 * MAX_CTAS * TM * 4 + 128;
  static size_t total(int LD) { return o + (size_t)2 * MAX_CTAS * TM * LD * 4; }
};
static_assert(sizeof(LatentRecord) * MAX_CTAS <= 4096 && 2 * MAX_CTAS * 4 <= 4096 && Layout::o % 16 == 0, "layout");

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Barrier of the compute warps.
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The same, and whether any of their threads brought true: a warp whose wait gave
// up still comes here, and then all leave together.
__device__ __forceinline__ bool work_sync_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

template <int LD, typename T, bool GATHER>
__global__ void __launch_bounds__(nthreads(GATHER), 1)
    latent_rows_kernel(const __grid_constant__ CUtensorMap mx, const T* __restrict__ q, LatentAttnP p) {
  using C = Cfg<LD>;
  constexpr int NS = C::NS, D = LD + 64, PRODUCERS = producers(GATHER), NTHREADS = nthreads(GATHER);
  extern __shared__ __align__(1024) unsigned char sm[];
  using Sh = State<LD, NTHREADS>;
  Sh& sh = *reinterpret_cast<Sh*>(sm + C::RING);
  volatile int& s_abort = sh.abort;
  if (smem_u32(sm) & 1023u) {   // the swizzled rows need it; the array is declared so
    if (threadIdx.x == 0) atomicOr(p.dev_status, PKV_DEV_TIMEOUT);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == NTHREADS - 1) {   // a thread with no other set-up to do
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sh.full[s], GATHER ? 32 : 1);
      mbar_init(&sh.empty[s], WARPS);
    }
    for (int e = 0; e < NSEG; ++e) {
      mbar_init(&sh.segfull[e], 1);
      mbar_init(&sh.segempty[e], WARPS + PRODUCERS);
    }
    fence_mbar_init();
    sh.abort = 0;
    sh.plan.run = 0;
    sh.seg[0].valid = 0;
    sh.bad[0] = 0;
    tma_prefetch_desc(&mx);
  }
  pdl_wait();   // lengths, queries, cache rows and page tables may come from the kernel before
  latent_plan<TM, BN, START, NTHREADS>(p, blockIdx.x, gridDim.x, &sh.plan, sh.seg);
  __syncthreads();
  pdl_trigger();

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
    const long long t0 = clock64();
    for (uint32_t it = 0; !ok; ++it) {
      ok = mbar_try_wait(bar, parity);
      if (!ok && (it & 63u) == 63u) {
        if (s_abort) break;
        if (clock64() - t0 > WAIT_LIMIT_CLOCKS || it > (1u << 28)) {
          s_abort = 1;
          atomicOr(p.dev_status, PKV_DEV_TIMEOUT);
          break;
        }
      }
    }
    return __all_sync(0xffffffffu, ok);
  };

  bool ok = true;
  if (warp == WARPS) {
    // ------------------------------------------------------------- scheduler
    if (lane == 0) mbar_arrive(&sh.segfull[0]);   // the plan left the first one there
    LatentRun<TM, BN, START> run(p, sh.plan, blockIdx.x);
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t % NSEG;
      if (t >= NSEG && !(ok = wait(&sh.segempty[e], ((t / NSEG) - 1) & 1))) break;
      const LatentSegment g = run.next(p);
      if (t > 0 && lane == 0) {
        sh.seg[e] = g;
        sh.bad[e] = 0;
        mbar_arrive(&sh.segfull[e]);
      }
      __syncwarp();
      if (!g.valid) break;
    }
    if (!p.whole && lane == 0) ((LatentRecord*)(p.ws + Layout::rec))[blockIdx.x] = run.r;
  } else if (warp > WARPS) {
    // --------------------------------------------------------------- producer
    // Lane l takes box l of a slot, or finds row l for the copies. Rows behind the end and bad pages are read from
    // page 0 (masked, or discarded); a slot with no key of the tile is not read.
    constexpr int boxes = GATHER ? HB : 1;
    const uint32_t turn = warp - WARPS - 1;
    uint32_t h = 0;   // slots before the current one
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t % NSEG;
      if (!(ok = wait(&sh.segfull[e], (t / NSEG) & 1))) break;
      const LatentSegment g = sh.seg[e];
      if (!g.valid) break;
      const int32_t* pt = p.page_tables + (int64_t)g.b * p.max_pages;
      const int keys = min(g.L, g.n * BN);   // keys that the tile needs
      bool bad = false;
      auto box_row = [&](int i) {
        const int key = i * HB + lane;
        if (lane >= boxes || key >= keys) return 0;
        const int lp = key / p.P;
        const int id = __ldg(pt + lp);
        if (id >= 0 && id < p.num_pages) return id * p.P + (key - lp * p.P);
        bad = true;
        return 0;
      };
      const int i1 = g.j1 * (BN / HB);
      int row = box_row(g.j0 * (BN / HB));
      for (int i = g.j0 * (BN / HB); i < i1; ++i, ++h) {
        const int cur = row;
        if (bad) sh.bad[e] = 1;
        if (i + 1 < i1) row = box_row(i + 1);
        const uint32_t slot = h % NS;
        if (GATHER && h % PRODUCERS != turn) continue;
        if (!(ok = wait(&sh.empty[slot], ((h / NS) & 1) ^ 1))) break;
        const bool some = i * HB < keys;
        if constexpr (GATHER) {
          if (some) {
            // eight lanes copy 128 bytes of a row, four rows at a time
            const uint32_t dst = smem_u32(sm) + slot * C::SLOT;
#pragma unroll
            for (int y = 0; y < HB / 4; ++y) {
              const int r = y * 4 + (lane >> 3);
              const char* src = (const char*)p.cache + (int64_t)__shfl_sync(0xffffffffu, cur, r) * (D * 2) + (lane & 7) * 16;
              const uint32_t at = dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
#pragma unroll
              for (int u = 0; u < C::CH; ++u) cp_async_16(at + u * UNIT, src + u * 128);
            }
            cp_async_arrive(&sh.full[slot]);
          } else {
            mbar_arrive(&sh.full[slot]);
          }
          __syncwarp();
          continue;
        }
        if (lane == 0) {
          if (some) mbar_arrive_expect_tx(&sh.full[slot], C::SLOT);
          else mbar_arrive(&sh.full[slot]);
        }
        __syncwarp();
        // the slot's rows lie in one page: all of its columns at once
        if (some && lane == 0) tma_load_3d(sm + slot * C::SLOT, &mx, &sh.full[slot], 0, cur, 0);
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&sh.segempty[e]);
      __syncwarp();
    }
    if (GATHER) cp_async_wait_all();
    if (!ok && lane == 0) {
      // copies may still be on their way: give them time to land
      const uint64_t t0 = globaltimer_ns();
      for (int it = 0; it < (1 << 24) && globaltimer_ns() - t0 < 20000000ull; ++it) {}
    }
  } else {
    // ----------------------------------------------------------------- compute
    const int kg = warp & 3, kh = warp >> 2;            // scores: quarter of the columns, half of the keys
    const int srow = tid >> 4, scol = (tid & 15) * 4;   // softmax: a thread's row and four keys
    const int fr = lane >> 2, fc = (lane & 3) * 2;      // fragment row (and + 8) and column
    const uint32_t ring = smem_u32(sm), s_p = smem_u32(sh.p);
    const int d0 = warp * C::DW;                        // this warp's output columns
    const uint32_t v_unit = (d0 / 64) * UNIT, v_chunk = (d0 % 64) / 8;
    const float sc = p.scale_log2;
    constexpr float SHIFT = weight_shift<T>(0.f);       // (a row's scale is its maximum so far)
    uint32_t h = 0;   // ring slots before the current step
    for (uint32_t t = 0;; ++t) {
      const uint32_t e = t % NSEG;
      if (work_sync_or(!wait(&sh.segfull[e], (t / NSEG) & 1))) break;
      const LatentSegment g = sh.seg[e];
      if (!g.valid) break;
      // this warp's quarter of the queries (rows that are not there: zeros)
      uint32_t qa[C::KS][4];
      {
        const T* q0 = q + (int64_t)g.row0 * D + kg * C::KS * 16 + fc;
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = fr + (x & 1) * 8;
            qa[k][x] = r < g.nrows ? *reinterpret_cast<const uint32_t*>(q0 + (int64_t)r * D + k * 16 + (x >> 1) * 8) : 0u;
          }
      }
      float o[C::DW / 8][4];
#pragma unroll
      for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
      float m_run = -INFINITY, l_run = 0.f;
      const int pos = min(g.base + (g.frow0 + srow) / p.H, g.L - 1);
      for (int j = g.j0; j < g.j1; ++j, h += 2) {
        const uint32_t slot0 = h % NS, slot1 = (h + 1) % NS;
        ok = wait(&sh.full[slot0], (h / NS) & 1) && wait(&sh.full[slot1], ((h + 1) / NS) & 1);
        // ---- scores of keys [32 kh, 32 kh + 32) over this warp's quarter
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
        if (ok) {
          const uint32_t base = ring + (kh ? slot1 : slot0) * C::SLOT;
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            const int kk = kg * C::KS + k;              // 16-column step of the row
#pragma unroll
            for (int np = 0; np < 2; ++np) {
              // lanes 8i..8i+7: keys of n-tile 2 np + i / 2, columns + 8 (i & 1)
              const int key = np * 16 + (lane >> 4) * 8 + (lane & 7);
              const int chunk = (kk & 3) * 2 + ((lane >> 3) & 1);
              uint32_t b[4];
              ldsm4(b, base + (kk >> 2) * UNIT + key * 128 + ((chunk ^ (key & 7)) << 4));
              mma16816<T>(s[np * 2], qa[k], b[0], b[1]);
              mma16816<T>(s[np * 2 + 1], qa[k], b[2], b[3]);
            }
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            float* d = &sh.s[kg][fr][kh * 32 + n * 8 + fc];
            *reinterpret_cast<float2*>(d) = make_float2(s[n][0], s[n][1]);
            *reinterpret_cast<float2*>(d + 8 * S_LD) = make_float2(s[n][2], s[n][3]);
          }
        }
        if (work_sync_or(!ok)) {
          ok = false;
          break;
        }
        // ---- softmax of four keys of one row
        {
          float4 x = *reinterpret_cast<const float4*>(&sh.s[0][srow][scol]);
#pragma unroll
          for (int y = 1; y < 4; ++y) {
            const float4 z = *reinterpret_cast<const float4*>(&sh.s[y][srow][scol]);
            x.x += z.x;
            x.y += z.y;
            x.z += z.z;
            x.w += z.w;
          }
          const int lim = pos - j * BN - scol;          // this thread's keys up to lim are visible
          if (lim < 0) x.x = -INFINITY;
          if (lim < 1) x.y = -INFINITY;
          if (lim < 2) x.z = -INFINITY;
          if (lim < 3) x.w = -INFINITY;
          float mt = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
#pragma unroll
          for (int b = 1; b < 16; b <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, b));
          const float m_new = fmaxf(m_run, mt * sc);
          // a row that sees no key of this run so far has m = -inf: its weights are 0
          const float nm = m_new == -INFINITY ? 0.f : SHIFT - m_new;
          const float alpha = m_new == -INFINITY ? 1.f : ex2(m_run - m_new);
          m_run = m_new;
          const float a = ex2(fmaf(x.x, sc, nm)), b = ex2(fmaf(x.y, sc, nm)), c = ex2(fmaf(x.z, sc, nm)),
                      d = ex2(fmaf(x.w, sc, nm));
          l_run = l_run * alpha + ((a + b) + (c + d));
          *reinterpret_cast<uint2*>(sh.p + srow * 128 + (((scol >> 3) ^ (srow & 7)) << 4) + (scol & 4) * 2) =
              make_uint2(pack2<T>(a, b), pack2<T>(c, d));
          if ((tid & 15) == 0) sh.alpha[srow] = alpha;
        }
        const int end = g.L - j * BN;   // rows from here on are behind the sequence
        if (end < BN) {
          // 0 * NaN must not reach O from the slots behind the end
          for (int i = tid; i < (BN - end) * (LD / 8); i += WARPS * 32) {
            const int key = end + i / (LD / 8), c = i % (LD / 8);
            *reinterpret_cast<uint4*>(sm + (key < HB ? slot0 : slot1) * C::SLOT + (c >> 3) * UNIT + (key % HB) * 128 +
                                      (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();     // before the next copy into these slots
        }
        work_sync();
        // ---- O += P V for this warp's columns
        const float a0 = sh.alpha[fr], a1 = sh.alpha[fr + 8];
#pragma unroll
        for (int n = 0; n < C::DW / 8; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) {
          uint32_t a[4];
          {
            const int r = lane & 15, chunk = k * 2 + (lane >> 4);
            ldsm4(a, s_p + r * 128 + ((chunk ^ (r & 7)) << 4));
          }
          const int key = (k & 1) * 16 + (lane & 15);
          const uint32_t base = ring + (k < 2 ? slot0 : slot1) * C::SLOT + v_unit + key * 128;
#pragma unroll
          for (int np = 0; np < C::DW / 16; ++np) {
            const uint32_t chunk = v_chunk + np * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4t(b, base + ((chunk ^ (key & 7)) << 4));
            mma16816<T>(o[np * 2], a, b[0], b[1]);
            mma16816<T>(o[np * 2 + 1], a, b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.empty[slot0]);
          mbar_arrive(&sh.empty[slot1]);
        }
      }
      if (!ok) break;
      // ---- the rows' sums, then this warp's columns
#pragma unroll
      for (int b = 1; b < 16; b <<= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, b);
      if ((tid & 15) == 0) {
        sh.m[srow] = m_run;
        sh.l[srow] = l_run;
      }
      work_sync();
      const int bad = *(volatile int*)&sh.bad[e];
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const int slot = 2 * blockIdx.x + (g.j0 == 0 ? 1 : 0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = fr + x * 8;
        if (r >= g.nrows || (whole && bad)) continue;
        // No visible key in a partial run: zeros. A whole tile's row always sees keys; where
        // all their scores are -inf it becomes NaN, as the formula has it.
        const float inv = sh.l[r] == 0.f && !whole ? 0.f : 1.f / sh.l[r];
        const int64_t row = (int64_t)g.row0 + r;
        T* dst = (T*)p.out + row * LD + d0 + fc;
        float* part = (float*)(p.ws + Layout::o) + ((int64_t)slot * TM + r) * LD + d0 + fc;
#pragma unroll
        for (int n = 0; n < C::DW / 8; ++n) {
          const float y0 = o[n][2 * x] * inv, y1 = o[n][2 * x + 1] * inv;
          if (whole) *reinterpret_cast<uint32_t*>(dst + n * 8) = pack2<T>(y0, y1);
          else *reinterpret_cast<float2*>(part + n * 8) = make_float2(y0, y1);
        }
      }
      if (tid < TM && tid < g.nrows) {
        const float l = sh.l[tid];
        // (NaN scores: m may be -inf, l is NaN)
        const float lg = l == 0.f ? -INFINITY : sh.m[tid] + (__log2f(l) - SHIFT);
        if (!whole) ((float*)(p.ws + Layout::lse))[slot * TM + tid] = lg;
        else if (p.lse && !bad) p.lse[(int64_t)g.row0 + tid] = lg * LN2;
      }
      if (tid == 0) {
        if (!whole) ((int32_t*)(p.ws + Layout::bad))[slot] = bad;
        if (bad) atomicOr(p.dev_status, PKV_DEV_BAD_PAGE);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.segempty[e]);
    }
  }
}

// Joins the partial results of every cut tile: a row's parts weighted by
// 2^(lse_s - max). Groups of LD / 4 threads take every PG-th part, then their sums
// are added in the order of the groups. The CTAs of all workers but the last that
// share a tile divide its rows.
constexpr int CY = 4, CTHREADS = 512;
template <int LD, typename T>
__global__ void __launch_bounds__(CTHREADS) latent_rows_combine_kernel(char* ws, T* out, float* lse) {
  constexpr int NV = LD / 4, PG = CTHREADS / NV;
  __shared__ float4 s_o[PG][NV];
  __shared__ float s_t[PG];
  pdl_wait();
  const int cta = blockIdx.x;
  const LatentRecord rec = ((const LatentRecord*)(ws + Layout::rec))[cta];
  const int r0 = (int)blockIdx.y + CY * (cta - rec.owner);
  if (r0 >= rec.nrows) return;
  const float* sums = (const float*)(ws + Layout::lse);
  const int32_t* bad = (const int32_t*)(ws + Layout::bad);
  const float4* parts = (const float4*)(ws + Layout::o);
  auto slot = [&](int s) { return s == 0 ? 2 * rec.owner + 1 : 2 * (rec.owner + s); };
  const int tid = threadIdx.x, lane = tid & 31, v = tid % NV, pg = tid / NV;
  constexpr int U = 4;   // parts in flight a thread
  for (int r = r0; r < rec.nrows; r += CY * (rec.parts - 1)) {
    float w[U];
    float4 y[U];
    auto load = [&](int s0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * PG;
        w[u] = -INFINITY;
        y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < rec.parts) {
          w[u] = sums[slot(s) * TM + r];
          y[u] = parts[((int64_t)slot(s) * TM + r) * NV + v];
        }
      }
    };
    load(pg);   // under way while the maximum is found
    float m = -INFINITY;
    int any = 0;
    for (int s = lane; s < rec.parts; s += 32) {
      any |= bad[slot(s)];
      m = fmaxf(m, sums[slot(s) * TM + r]);
    }
    if (__any_sync(0xffffffffu, any)) return;   // (every warp looked at every part)
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;   // all scores -inf: weights 0, a result of NaN, a log sum of -inf
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    for (int s = pg; s < rec.parts;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = exp2f(w[u] - m);
        total += f;
        o.x += f * y[u].x;
        o.y += f * y[u].y;
        o.z += f * y[u].z;
        o.w += f * y[u].w;
      }
      if ((s += U * PG) < rec.parts) load(s);
    }
    s_o[pg][v] = o;
    if (v == 0) s_t[pg] = total;
    __syncthreads();
    if (pg == 0) {
#pragma unroll
      for (int y = 1; y < PG; ++y) {
        const float4 z = s_o[y][v];
        o.x += z.x;
        o.y += z.y;
        o.z += z.z;
        o.w += z.w;
        total += s_t[y];
      }
      const float inv = 1.f / total;
      const int64_t row = (int64_t)rec.row0 + r;
      *reinterpret_cast<uint2*>(out + row * LD + v * 4) =
          make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
      if (lse && v == 0) lse[row] = (m + log2f(total)) * LN2;
    }
    __syncthreads();
  }
}

template <int LD, typename T, bool GATHER>
cudaError_t launch(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s) {
  constexpr int smem = Cfg<LD>::RING + sizeof(State<LD, nthreads(GATHER)>);
  static_assert(smem <= 232448, "shared memory");
  static std::atomic<uint64_t> ready{0};   // devices whose kernel attribute is set
  if (!(ready.load() >> a.dev.id & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(latent_rows_kernel<LD, T, GATHER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << a.dev.id);
  }
  CUtensorMap mx;
  if (!make_map_chunks(&mx, a.cache,
                     std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     Cfg<LD>::CH, (int64_t)a.num_pages * a.P, LD + 64, HB, Cfg<LD>::CH))
    return cudaErrorInvalidValue;
  const int ctas = latent_rows_tiling(a.dev.num_sms).workers;
  cudaError_t e;
  {
    KernelTimer timer("latent_rows", s);
    e = launch_after_trigger(latent_rows_kernel<LD, T, GATHER>, dim3(ctas), dim3(nthreads(GATHER)), smem, s, mx,
                             (const T*)a.q, p);
  }
  if (e != cudaSuccess || p.whole) return e;
  KernelTimer timer("latent_combine", s);
  return launch_after_trigger(latent_rows_combine_kernel<LD, T>, dim3(ctas, CY), dim3(CTHREADS), 0, s, a.ws,
                              (T*)a.out, a.lse);
}

template <int LD, typename T>
cudaError_t launch_either(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s) {
  return p.gather ? launch<LD, T, true>(a, p, s) : launch<LD, T, false>(a, p, s);
}

}  // namespace

int latent_rows_slot() { return HB; }
LatentTiling latent_rows_tiling(int num_sms) { return LatentTiling{TM, BN, num_sms < MAX_CTAS ? num_sms : MAX_CTAS}; }
size_t latent_rows_workspace(int latent_dim) { return Layout::total(latent_dim); }

cudaError_t launch_latent_rows(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s) {
  if (a.dtype == PKV_BF16)
    return a.latent_dim == 512 ? launch_either<512, __nv_bfloat16>(a, p, s)
                               : launch_either<256, __nv_bfloat16>(a, p, s);
  return a.latent_dim == 512 ? launch_either<512, __half>(a, p, s) : launch_either<256, __half>(a, p, s);
}

}  // namespace pkv
