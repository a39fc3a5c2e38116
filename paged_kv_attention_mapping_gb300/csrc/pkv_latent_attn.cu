// Absorbed latent attention over the paged latent cache: for row (token i of
// sequence b, head h) with query q, and cached rows x_j = [c_j, r_j],
//   s_j = scale q . x_j,  j <= kv_len - q_len + i,
//   out = sum_j exp(s_j - m) c_j / sum_j exp(s_j - m),  lse = m + ln(sum).
//
// All heads of a token read the same rows, so (token, head) rows are the M side
// of a matrix product and a cached row is read once for 128 of them. A work tile
// is 128 consecutive (token, head) rows of one sequence, and a pair of CTAs
// (tcgen05 cta_group::2) computes it in steps of 128 keys:
//   S = Q X^T          M 128 (64 rows a CTA), N 128 keys, K = LD + 64
//   O += P X[:, :LD]   M 128, N = LD as one or two products of 256, K 128 keys
// O takes LD / 2 TMEM columns of each CTA, two S buffers 64 columns each. One CTA
// alone could not do it: O of 128 rows x 512 fp32 is all the TMEM that an SM has.
//
// The product S wants half of the keys in each CTA, O wants half of the latent
// columns of all keys, and one instruction names the same shared-memory offsets in
// both CTAs. Of a step's 64 loaded rows a CTA therefore keeps the columns that are
// its own for O where they are; the others, once S has read them, are overwritten
// in place with the peer's rows of its own columns (from L2). A row costs 1.44
// times its bytes in L2 traffic and nothing beyond them in shared memory; loading
// keys for S and O into buffers of their own costs 1.89 times and left room for one
// step in flight only (decode of 128 sequences at 128 heads: 198 us).
//
//   warp 0   K producer (TMA; the page table gives the rows of each box)
//   warp 1   issues S (even CTA)
//   warp 2   reload producer; zeroes the rows behind the sequence's end in the last step
//   warp 3   issues O (even CTA)
//   warps 4-11 softmax. Lane l of TMEM holds row l & 63, keys (or output columns)
//            of half l / 64; two warps share a lane quarter, each with half of its
//            columns, so four threads have a row and exchange its maximum through
//            shared memory. P goes to shared memory in the cache type (the tensor cores take
//            no fp32 operand; tf32 ones would halve their rate and double P's room): half a
//            step of each weight, the sums stay fp32. O is rescaled
//            in TMEM only when a row's maximum grows by more than 2^8.
//   warp 12  scheduler: the segments of this pair, and their Q
//   warps 13-15  where rows come by thread copies instead of TMA (page sizes that
//            share no factor of 32 with a step): more loaders beside warp 0 and warp 2,
//            taking groups in turn, since each waits for its own copies
//
// Work split: the tick's steps (all tiles, one after the other, each with START more
// for its start and end) are cut into equal runs, one per pair. A tile cut by a run's
// end leaves partial results (normalised output in fp32 and log2 sum) that
// latent_combine_kernel joins. Ticks of short contexts are split by whole tiles instead.
//
// Decode of 128 sequences of 512-8192 keys at 128 heads (bf16): 132 us, 5.1 TB/s and 1.17
// PFLOP/s; with the combine 139 us. Two step slots fit beside Q, and a slot's turn (load,
// S, softmax 1300 cycles, O, the hand-offs between them) takes two steps' time. HBM is
// busy only while loads are under way, so the next step's rows are sent for into L2
// behind each step's loads (without: 146 us; earlier by half a step 138, by one step 138 or 144, by two
// steps 144 or 156: what is sent for too early holds up the loads before it; half of the rows 146). With
// all pages in L2 it takes 115. Weights without exponentials and rows without an exchange
// of maxima: 1 % faster, so the softmax is not what bounds it. Other L2 promotions,
// rotary columns in a unit of their own: no faster.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_latent.cuh"
#include "pkv_latent_sched.cuh"
#include "pkv_sm100.cuh"

namespace pkv {
using namespace sm100;

namespace {

constexpr int BM = 128;          // (token, head) rows of a tile
constexpr int HM = 64;           // rows of one CTA
constexpr int BN = 128;          // keys of a step
// What a tile counts beside its steps in the split. 40 sequences of up to 3000 keys, 1-5
// tokens, 20 heads, latent 256 with 0 / 1 / 2 / 4 / 6: 24.4 / 22.4 / 22.4 / 22.9 / 24.0 us; decode of 128
// sequences at 128 heads: 145.8 / 145.3 / 146.8 / 148.5 / 151.
constexpr int START = 1;
constexpr int MAX_PAIRS = 76;    // 152 SMs; the workspace is laid out for these
constexpr int SM_WARPS = 8;         // softmax warps of a CTA
constexpr int SM_FIRST = 4;         // the first of them: its TMEM lanes are those of warp & 3
constexpr int SCHED = SM_FIRST + SM_WARPS;   // the scheduler's warp; K loaders 1.. and the second reloader follow
constexpr int K_LOADERS = 3, V_LOADERS = 2;  // for thread copies
// Threads of a CTA. Without thread copies there are no idle warps: with them, the
// decode of 128 sequences at 128 heads took 174 us instead of 151.
constexpr int nthreads(bool gather) { return (SCHED + 1 + (gather ? K_LOADERS + V_LOADERS - 2 : 0)) * 32; }
constexpr uint32_t UNIT = 8192;  // 64 rows x 64 columns of 16 bits: one swizzle atom wide
constexpr float RESCALE_LOG2 = 8.f;

// A step's 64 rows of one CTA lie as LD / 64 units of 64 columns, in NG groups of
// four: two units with columns of the even CTA's part of O, two of the odd CTA's;
// one product of 256 output columns reads one group. The rotary columns have
// units of their own, read by S alone.
template <int LD>
struct Cfg {
  static constexpr int CH = LD / 64 + 1;           // units of a row, the rotary one last
  static constexpr int NG = LD / 256;              // groups
  static constexpr int NST = LD == 512 ? 2 : 4;    // steps in shared memory
  static constexpr uint32_t Q_BYTES = CH * UNIT;
  static constexpr uint32_t G_BYTES = 4 * UNIT;
  static constexpr uint32_t ST_BYTES = NG * G_BYTES;
  static constexpr uint32_t X_BYTES = (1 + NST) * UNIT;   // P of keys 0-63; per step, the rotary unit, then P of keys 64-127
  static constexpr uint32_t TILES = Q_BYTES + NST * ST_BYTES + X_BYTES;
  // 64-column chunk of a row that unit u of group g holds
  static __host__ __device__ constexpr int chunk(int g, int u) { return (u < 2 ? 0 : LD / 128) + 2 * g + (u & 1); }
};

constexpr long long WAIT_LIMIT_CLOCKS = 4000000000ll;   // about two seconds
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 256;

// Workspace: a record per pair, then a bad flag, log2 sums and outputs for two partial results per pair.
struct Layout {
  static constexpr size_t rec = 0;
  static constexpr size_t bad = 2048;
  static constexpr size_t lse = 4096;
  static constexpr size_t o = lse + (size_t)2 * MAX_PAIRS * BM * 4;
  // Partial outputs lie as the epilogue's threads hold them: for a slot and a CTA,
  // four columns at a time, the 128 TMEM lanes side by side. This is the vector of
  // lane `lane` (row lane & 63 of the CTA, columns from lane / 64 * LD / 2 + 4 c).
  static __device__ int64_t vec(int LD, int slot, int rank, int c, int lane) {
    return ((int64_t)(slot * 2 + rank) * (LD / 8) + c) * BM + lane;
  }
  static size_t total(int LD) { return o + (size_t)2 * MAX_PAIRS * BM * LD * 4; }
};
static_assert(sizeof(LatentRecord) * MAX_PAIRS <= 2048 && 2 * MAX_PAIRS * 4 <= 2048 && Layout::o % 256 == 0, "layout");

__device__ __forceinline__ void row_bar_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void row_bar_arrive(int id) { asm volatile("bar.arrive %0, 128;" ::"r"(id) : "memory"); }

// A CTA's barriers and shared words, behind the tiles. k, v, q, p and sfree are
// waited on in the even CTA, where both CTAs arrive; the MMA commits signal sdone,
// odone, s and qempty in both.
constexpr int NSEG = 4;
template <int LD, int NTHREADS>
struct State {
  using C = Cfg<LD>;
  // per step slot and group: loaded for S; read by S; loaded for O; read by O (after
  // the last group: O is complete)
  uint64_t k[C::NST][C::NG], sdone[C::NST][C::NG], v[C::NST][C::NG], odone[C::NST][C::NG];
  uint64_t q, qempty;                 // Q loaded; the last S that reads it done
  uint64_t vtail[C::NG];              // the reload of a last step, before its rows are zeroed
  uint64_t s[2], sfree[2];            // S complete; read by the softmax warps
  uint64_t p;                         // P written
  uint64_t segfull[NSEG], segempty[NSEG], drain[2];
  LatentPlan<NTHREADS> plan;
  float x[2][4][HM];                  // row figures of a row's four threads, by exchange parity
  LatentSegment seg[NSEG];
  int bad[NSEG];
  int abort;
  uint32_t tmem;
};

template <int LD, typename T, bool GATHER>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(nthreads(GATHER), 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ CUtensorMap m2, LatentAttnP p) {
  using C = Cfg<LD>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int NST = C::NST, NG = C::NG, NTHREADS = nthreads(GATHER);
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* sQ = sm;
  unsigned char* sK = sQ + C::Q_BYTES;               // [step][group][unit]
  // unit 0: P, keys 0-63; unit 1 + st: rotary unit of step slot st, then P, keys 64-127
  unsigned char* sX = sK + NST * C::ST_BYTES;
  using Sh = State<LD, NTHREADS>;
  Sh& sh = *reinterpret_cast<Sh*>(sX + C::X_BYTES);
  auto& bar_k = sh.k;
  auto& bar_sdone = sh.sdone;
  auto& bar_v = sh.v;
  auto& bar_odone = sh.odone;
  auto& bar_q = sh.q;
  auto& bar_qempty = sh.qempty;
  auto& bar_vtail = sh.vtail;
  auto& bar_s = sh.s;
  auto& bar_p = sh.p;
  auto& bar_sfree = sh.sfree;
  auto& bar_seg = sh.segfull;
  auto& bar_segempty = sh.segempty;
  auto& bar_drain = sh.drain;
  auto& s_tmem = sh.tmem;
  auto& s_seg = sh.seg;
  auto& s_bad = sh.bad;
  volatile int& s_abort = sh.abort;
  auto& s_x = sh.x;
  if (smem_u32(sm) & 1023u) {   // the swizzled tiles need it; the array is declared so
    if (threadIdx.x == 0) atomicOr(p.dev_status, PKV_DEV_TIMEOUT);
    return;
  }

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == NTHREADS - 1) {   // a thread with no other set-up to do
    mbar_init(&bar_q, 2);
    mbar_init(&bar_qempty, 1);
    for (int g = 0; g < NG; ++g) {
      for (int st = 0; st < NST; ++st) {
        mbar_init(&bar_k[st][g], 2);
        mbar_init(&bar_sdone[st][g], 1);
        mbar_init(&bar_v[st][g], 2);
        mbar_init(&bar_odone[st][g], 1);
      }
      mbar_init(&bar_vtail[g], 1);
    }
    mbar_init(&bar_p, 2 * SM_WARPS);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_sfree[i], 2 * SM_WARPS);
      mbar_init(&bar_drain[i], 1);
    }
    for (int e = 0; e < NSEG; ++e) {
      mbar_init(&bar_seg[e], 1);
      // softmax, producers, MMA issuers
      mbar_init(&bar_segempty[e], SM_WARPS + (GATHER ? K_LOADERS + V_LOADERS : 2) + (rank == 0 ? 2 : 0));
    }
    fence_mbar_init();
    s_abort = 0;
    sh.plan.run = 0;
    s_seg[0].valid = 0;
    s_bad[0] = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&m2);
  }
  if (warp == 1) tmem_alloc_pair(&s_tmem, TMEM_COLS);
  __syncwarp();
  cluster_arrive();     // the peer may use this CTA's barriers once every thread of both is here
  // lengths, queries, cache rows and page tables may come from the kernel before
  pdl_wait();
  latent_plan<BM, BN, START, NTHREADS>(p, pair, pairs, &sh.plan, s_seg);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_wait();
  const uint32_t tmem = s_tmem;
  pdl_trigger();

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
    const long long t0 = clock64();   // (reading the global timer takes longer than most waits)
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
  if (warp == SCHED) {
    // ---------------------------------------------- scheduler, and producer of Q
    const uint32_t q_bar = map_to_rank(&bar_q, 0);
    auto load_q = [&](uint32_t t, int row0) -> bool {
      // Q replaces the segment before's once its last S is done
      if (t >= 1 && !wait(&bar_qempty, (t - 1) & 1)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx_cluster(q_bar, C::Q_BYTES);
        tma_load_3d_pair(sQ, &mq, q_bar, 0, row0 + (int)rank * HM, 0);
      }
      __syncwarp();
      return true;
    };
    if (lane == 0) mbar_arrive(&bar_seg[0]);   // the plan left the first segment there
    if (s_seg[0].valid) load_q(0, s_seg[0].row0);
    LatentRun<BM, BN, START> run(p, sh.plan, pair);
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t % NSEG;
      if (t >= NSEG && !(ok = wait(&bar_segempty[e], ((t / NSEG) - 1) & 1))) break;
      const LatentSegment g = run.next(p);
      if (t > 0 && lane == 0) {
        s_seg[e] = g;
        s_bad[e] = 0;
        mbar_arrive(&bar_seg[e]);
      }
      __syncwarp();
      if (!g.valid) break;
      if (t > 0) ok = load_q(t, g.row0);
    }
    // (whole tiles leave nothing to join)
    if (!p.whole && rank == 0 && lane == 0) ((LatentRecord*)(p.ws + Layout::rec))[pair] = run.r;
  } else if (warp == 0 || warp == 2 || (GATHER && warp > SCHED)) {
    // --------------------------------------------------------------- producers
    // Warp 0 loads this CTA's 64 keys of each step, warp 2 the peer's 64 keys of this
    // CTA's output columns. Lane l takes boxes l and l + 32 of the 64
    // keys. Rows behind the end and bad pages are read from page 0 (masked, or
    // discarded), so that a step's bytes are always the same. With thread copies
    // K_LOADERS and V_LOADERS warps share that, a group each in turn.
    const bool reload = warp == 2 || (GATHER && warp >= SCHED + K_LOADERS);
    const uint32_t loaders = !GATHER ? 1 : reload ? V_LOADERS : K_LOADERS;
    const uint32_t loader = warp < SM_FIRST ? 0 : reload ? warp - (SCHED + K_LOADERS) + 1 : warp - SCHED;
    const int key_half = (int)rank ^ (reload ? 1 : 0);
    const int boxes = HM / p.box;
    // 0 * NaN must not reach O from the slots behind the end: units 0 and 1 of a
    // group hold keys 0-63 of the step, 2 and 3 keys 64-127
    auto zero_rows = [&](unsigned char* group, int end) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int from = max(0, end - (u >> 1) * HM);
        uint4* base = (uint4*)(group + u * UNIT);
        for (int x = from * 8 + lane; x < HM * 8; x += 32) base[x] = make_uint4(0, 0, 0, 0);
      }
    };
    uint32_t n = 0, n_tail = 0;     // steps, and last steps with rows to zero, before the current one
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t % NSEG;
      if (!(ok = wait(&bar_seg[e], (t / NSEG) & 1))) break;
      const LatentSegment g = s_seg[e];
      if (!g.valid) break;
      const int32_t* pt = p.page_tables + (int64_t)g.b * p.max_pages;
      const int keys = min(g.L, g.n * BN);   // keys that the tile needs
      bool bad = false;
      auto box_row = [&](int j, int i) {
        const int key = j * BN + key_half * HM + i * p.box;
        if (i >= boxes || key >= keys) return 0;
        const int lp = key / p.P;
        const int id = __ldg(pt + lp);
        if (id >= 0 && id < p.num_pages) return id * p.P + (key - lp * p.P);
        bad = true;
        return 0;
      };
      int row[2] = {box_row(g.j0, lane), box_row(g.j0, lane + 32)};
      for (int j = g.j0; j < g.j1 && ok; ++j, ++n) {
        const int cur[2] = {row[0], row[1]};
        if (bad) s_bad[e] = 1;
        if (j + 1 < g.j1) {
          row[0] = box_row(j + 1, lane);
          row[1] = box_row(j + 1, lane + 32);
        }
        const uint32_t st = n % NST, par = (n / NST) & 1;
        unsigned char* stage = sK + st * C::ST_BYTES;
        const int end = g.L - j * BN;        // rows from here on are behind the sequence
        const bool tail = reload && end < BN;
        // the next step's rows go into L2 while its slot is still taken
        const bool ahead = !reload && n + 1 >= NST && j + 1 < g.j1;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          // units that this warp fills, and their columns
          const int u0 = reload ? (rank ? 0 : 2) : 0, nu = reload ? 2 : 4;
          const int c0 = reload ? (rank ? 2 : 0) : 0;
          if (GATHER && (n * NG + k) % loaders != loader) continue;
          if (!(ok = reload ? wait(&bar_sdone[st][k], par) : wait(&bar_odone[st][k], par ^ 1))) break;
          const uint32_t bar = map_to_rank(reload ? &bar_v[st][k] : &bar_k[st][k], 0);
          const bool rot = !reload && k == NG - 1;
          if constexpr (GATHER) {
            // eight lanes copy 128 bytes of a row, four rows at a time
#pragma unroll 4
            for (int y = 0; y < HM / 4; ++y) {
              const int r = y * 4 + (lane >> 3);
              const int from = __shfl_sync(0xffffffffu, y < HM / 8 ? cur[0] : cur[1], r & 31);
              const char* src = (const char*)p.cache + (int64_t)from * ((LD + 64) * 2) + (lane & 7) * 16;
              const uint32_t at = r * 128 + (((lane & 7) ^ (r & 7)) << 4);
              const uint32_t dst = smem_u32(stage) + k * C::G_BYTES + u0 * UNIT + at;
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (u < nu) cp_async_16(dst + u * UNIT, src + C::chunk(k, c0 + u) * 128);
              if (rot) cp_async_16(smem_u32(sX) + (1 + st) * UNIT + at, src + LD * 2);
            }
            if (ahead) {
              // a lane per row and chunk
              const int chunk = (lane & 2 ? C::chunk(k, 2) : C::chunk(k, 0)) + (lane & 1);
#pragma unroll
              for (int y = 0; y < HM / 8; ++y) {
                const int from = __shfl_sync(0xffffffffu, y < HM / 16 ? row[0] : row[1], (y * 8 + (lane >> 2)) & 31);
                prefetch_l2((const char*)p.cache + (int64_t)from * ((LD + 64) * 2) + chunk * 128);
              }
              if (rot) {
                prefetch_l2((const char*)p.cache + (int64_t)row[0] * ((LD + 64) * 2) + LD * 2);
                prefetch_l2((const char*)p.cache + (int64_t)row[1] * ((LD + 64) * 2) + LD * 2);
              }
            }
            cp_async_wait_all();
            __syncwarp();   // other lanes' copies too: zeros go over rows that any lane copied
            if (tail) zero_rows(stage + k * C::G_BYTES, end);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(bar);
            continue;
          }
          if (lane == 0) {
            if (tail) mbar_arrive_expect_tx(&bar_vtail[k], 2 * UNIT);
            else mbar_arrive_expect_tx_cluster(bar, (nu + (rot ? 1 : 0)) * UNIT);
          }
          __syncwarp();
          if (boxes == 1) {
            // two units at a time: an instruction costs its warp about 90 cycles
            if (lane == 0) {
#pragma unroll
              for (int u = 0; u < 4; u += 2) {
                if (u >= nu) break;
                unsigned char* dst = stage + k * C::G_BYTES + (u0 + u) * UNIT;
                if (tail) tma_load_3d(dst, &m2, &bar_vtail[k], 0, cur[0], C::chunk(k, c0 + u));
                else tma_load_3d_pair(dst, &m2, bar, 0, cur[0], C::chunk(k, c0 + u));
              }
            }
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int i = lane + w * 32;
              if (i < boxes) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  if (u >= nu) break;
                  unsigned char* dst = stage + k * C::G_BYTES + (u0 + u) * UNIT + i * p.box * 128;
                  if (tail) tma_load_3d(dst, &mx, &bar_vtail[k], 0, cur[w], C::chunk(k, c0 + u));
                  else tma_load_3d_pair(dst, &mx, bar, 0, cur[w], C::chunk(k, c0 + u));
                }
              }
            }
          }
          if (rot) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int i = lane + w * 32;
              if (i < boxes) tma_load_3d_pair(sX + (1 + st) * UNIT + i * p.box * 128, &mx, bar, 0, cur[w], LD / 64);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (!GATHER && ahead) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
            if (lane + w * 32 < boxes)
              prefetch_l2_bulk((const char*)p.cache + (int64_t)row[w] * ((LD + 64) * 2), p.box * (LD + 64) * 2);
        }
        if (!GATHER && tail) {
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            if (!(ok = wait(&bar_vtail[k], n_tail & 1))) break;
            zero_rows(stage + k * C::G_BYTES, end);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(&bar_v[st][k], 0));
          }
          ++n_tail;
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bar_segempty[e]);
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------- MMA issuers
    if (rank == 0) {
      const uint32_t id_s = idesc_f16(BM, BN, BF16, false);
      const uint32_t id_o = idesc_f16(BM, 256, BF16, true);
      const uint64_t qd = smem_desc(smem_u32(sQ), 16, 1024, LAYOUT_SW128);
      const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, LAYOUT_SW128);
      const uint64_t xd = smem_desc(smem_u32(sX), 16, 1024, LAYOUT_SW128);
      const uint64_t vd = smem_desc(smem_u32(sK), UNIT, 1024, LAYOUT_SW128);
      uint32_t n = 0;
      for (uint32_t t = 0; ok; ++t) {
        const uint32_t e = t % NSEG;
        if (!(ok = wait(&bar_seg[e], (t / NSEG) & 1))) break;
        const LatentSegment g = s_seg[e];
        if (!g.valid) break;
        const int steps = g.j1 - g.j0;
        if (warp == 1) {
          if (!(ok = wait(&bar_q, t & 1))) break;
          for (int j = 0; j < steps; ++j, ++n) {
            const uint32_t st = n % NST, par = (n / NST) & 1;
            const uint32_t d = tmem + S_COL + (n & 1) * 64;
            if (n >= 2 && !(ok = wait(&bar_sfree[n & 1], ((n >> 1) - 1) & 1))) break;
#pragma unroll
            for (int k = 0; k < NG; ++k) {
              if (!(ok = wait(&bar_k[st][k], par))) break;
              tc_fence_after();
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  mma_f16_ss_pair_warp(d, qd + (uint64_t)((C::chunk(k, u) * UNIT + x * 32) >> 4),
                                       kd + (uint64_t)((st * C::ST_BYTES + k * C::G_BYTES + u * UNIT + x * 32) >> 4),
                                       id_s, (k | u | x) ? 1u : 0u);
              mma_commit_pair_warp(&bar_sdone[st][k]);
              if (k == NG - 1) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  mma_f16_ss_pair_warp(d, qd + (uint64_t)(((C::CH - 1) * UNIT + x * 32) >> 4),
                                       xd + (uint64_t)(((1 + st) * UNIT + x * 32) >> 4), id_s, 1u);
                mma_commit_pair_warp(&bar_s[n & 1]);
              }
            }
            if (!ok) break;
          }
          if (!ok) break;
          mma_commit_pair_warp(&bar_qempty);
        } else {
          for (int j = 0; j < steps; ++j, ++n) {
            const uint32_t st = n % NST, par = (n / NST) & 1;
            // the rows are there before P as a rule: their wait is over when P comes
            if (!(ok = wait(&bar_v[st][0], par))) break;
            if (!(ok = wait(&bar_p, n & 1))) break;
#pragma unroll
            for (int k = 0; k < NG; ++k) {
              if (k > 0 && !(ok = wait(&bar_v[st][k], par))) break;
              tc_fence_after();
#pragma unroll
              for (int x = 0; x < BN / 16; ++x)
                mma_f16_ss_pair_warp(tmem + k * 128, xd + (uint64_t)(((x >> 2) * (1 + st) * UNIT + (x & 3) * 32) >> 4),
                                     vd + (uint64_t)((st * C::ST_BYTES + k * C::G_BYTES + (x >> 2) * 2 * UNIT +
                                                      (x & 3) * 2048) >>
                                                     4),
                                     id_o, (j | x) ? 1u : 0u);
              mma_commit_pair_warp(&bar_odone[st][k]);
            }
            if (!ok) break;
          }
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive(&bar_segempty[e]);
        __syncwarp();
      }
    }
  } else if (!GATHER || (warp >= SM_FIRST && warp < SCHED)) {
    // ----------------------------------------------------------------- softmax
    const int quarter = warp & 3, half = quarter >> 1;
    const int sub = (warp - SM_FIRST) >> 2;         // which half of the lane's columns
    const int who = half * 2 + sub;
    const int i = (quarter & 1) * 32 + lane;        // row of this CTA
    const uint32_t lrow = (uint32_t)(quarter * 32) << 16;
    const int bar_id = 1 + (quarter & 1);           // the four warps of the same rows
    const uint32_t p_bar = map_to_rank(&bar_p, 0), sfree_bar = map_to_rank(bar_sfree, 0);
    constexpr int OC = LD / 4;                      // output columns of a thread
    constexpr float SHIFT = weight_shift<T>(RESCALE_LOG2);
    const uint32_t o_tmem = tmem + lrow + sub * OC;
    const float sc = p.scale_log2;
    uint32_t n = 0;                                  // steps before the current one
    // Exchanges before the current one: a step's maxima, and a segment's sums, take the
    // buffers in turn, so that a warp writes one only after every sibling's barrier behind its reads of it.
    uint32_t n_x = 0;
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t % NSEG;
      if (!(ok = wait(&bar_seg[e], (t / NSEG) & 1))) break;
      const LatentSegment g = s_seg[e];
      if (!g.valid) break;
      const int r = (int)rank * HM + i;              // row of the tile
      const bool warp_rows = (int)rank * HM + (quarter & 1) * 32 < g.nrows;   // some row of this warp is there
      const int pos = min(g.base + (g.frow0 + r) / p.H, g.L - 1);
      const int j_mask = (g.base + g.frow0 / p.H + 1) / BN;   // steps before see no hidden key
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = g.j0; j < g.j1; ++j, ++n) {
        if (!(ok = wait(&bar_s[n & 1], (n >> 1) & 1))) break;
        tc_fence_after();
        uint32_t x[32];
        tmem_ld32(tmem + lrow + S_COL + (n & 1) * 64 + sub * 32, x);
        // a warp that gave up takes part in no further exchange, so nobody goes on once the flag is up
        if (!(ok = !__any_sync(0xffffffffu, s_abort))) break;
        tmem_wait_ld();
        reg_fence(x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(sfree_bar + (n & 1) * 8);
        if (j >= j_mask) {
          const int lim = pos - j * BN - half * 64 - sub * 32;  // this thread's keys up to lim are visible
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k > lim) x[k] = __float_as_uint(-INFINITY);
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        float (*sx)[HM] = s_x[n_x++ & 1];
        sx[who][i] = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        row_bar_sync(bar_id);
        const float mt = fmaxf(max3(sx[0][i], sx[1][i], sx[2][i]), sx[3][i]) * sc;
        const bool first = j == g.j0;
        const bool grow = first || mt > m_run + RESCALE_LOG2;
        const float m_new = grow ? fmaxf(mt, m_run) : m_run;
        const float alpha = grow && !first ? ex2(m_run - m_new) : 1.f;
        const bool rescale = !first && __any_sync(0xffffffffu, grow);
        // a row that sees no key of this run so far has m = -inf: its weights are 0
        const float nm = m_new == -INFINITY ? 0.f : SHIFT - m_new;
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nm, nm);
        float2 ls[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
        uint32_t w[16];
        if (warp_rows) {   // else: P of rows that nobody reads stays as it is
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 y =
              __ffma2_rn(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), sc2, nm2);
          const float a = ex2(y.x), b = ex2(y.y);
          ls[k & 3] = __fadd2_rn(ls[k & 3], make_float2(a, b));
          w[k] = pack2<T>(a, b);
        }
        }
        // m_run = m_new = -inf before the first visible key: alpha would be NaN
        const float f = m_new == -INFINITY ? 1.f : alpha;
        l_run = l_run * f + (((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y)));
        m_run = m_new;
        // the product before has read P and written O (a segment's first step
        // follows its predecessor's epilogue, which waited for that)
        if (!first) {
          if (!(ok = wait(&bar_odone[(n - 1) % NST][NG - 1], ((n - 1) / NST) & 1))) break;
          tc_fence_after();
          if (rescale) {
#pragma unroll 1
            for (int c = 0; c < OC / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_wait(o_tmem + c * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32_wait(o_tmem + c * 32, o);
            }
          }
        }
        unsigned char* p_row = sX + (half ? 1 + n % NST : 0) * UNIT + i * 128;
        if (warp_rows)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(p_row + (((sub * 4 + c) ^ (i & 7)) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_bar);
      }
      if (!ok) break;
      // epilogue: the row's sum, then this thread's OC output columns
      float (*sx)[HM] = s_x[n_x++ & 1];
      sx[who][i] = l_run;
      row_bar_sync(bar_id);
      const float l = (sx[0][i] + sx[1][i]) + (sx[2][i] + sx[3][i]);
      if (!(ok = wait(&bar_odone[(n - 1) % NST][NG - 1], ((n - 1) / NST) & 1))) break;
      tc_fence_after();
      const int bad = *(volatile int*)&s_bad[e];
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const bool store = r < g.nrows && !(whole && bad);
      const int slot = 2 * pair + (g.j0 == 0 ? 1 : 0);
      // No visible key in a partial run: zeros. A whole tile's row always sees keys; where
      // all their scores are -inf it becomes NaN, as the formula has it.
      const float inv = l == 0.f && !whole ? 0.f : 1.f / l;
      const int64_t row = (int64_t)g.row0 + r;
      T* dst = (T*)p.out + row * LD + half * (LD / 2) + sub * OC;
      float4* part = (float4*)(p.ws + Layout::o) + Layout::vec(LD, slot, rank, sub * (OC / 4), quarter * 32 + lane);
#pragma unroll 1
      for (int c = 0; c < OC / 32; ++c) {
        uint32_t o[32];
        tmem_ld32_wait(o_tmem + c * 32, o);
        if (!store) continue;
        if (whole) {
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            y[k] = pack2<T>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          if (p.out_32) {   // whole sectors, where out's alignment allows it
#pragma unroll
            for (int v = 0; v < 2; ++v) st_global_32B(dst + c * 32 + v * 16, y + v * 8);
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              *reinterpret_cast<uint4*>(dst + c * 32 + v * 8) =
                  make_uint4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
          }
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            part[(c * 8 + v) * BM] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                                 __uint_as_float(o[4 * v + 2]) * inv,
                                                 __uint_as_float(o[4 * v + 3]) * inv);
        }
      }
      if (store && who == 0) {
        const float lg = l == 0.f ? -INFINITY : m_run + (__log2f(l) - SHIFT);   // (NaN scores: m may be -inf, l is NaN)
        if (!whole) ((float*)(p.ws + Layout::lse))[slot * BM + r] = lg;
        else if (p.lse) p.lse[row] = lg * LN2;
      }
      if (r == 0 && who == 0) {
        if (!whole) ((int32_t*)(p.ws + Layout::bad))[slot] = bad;
        if (bad) atomicOr(p.dev_status, PKV_DEV_BAD_PAGE);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_segempty[e]);
    }
    if (!ok) row_bar_arrive(bar_id);   // lets the other warps of these rows leave their exchange
  }

  if (s_abort && (warp == 0 || warp == 2 || warp >= SCHED)) {
    if (GATHER) cp_async_wait_all();
    // copies of this CTA may still be on their way: give them time to land
    const uint64_t t0 = globaltimer_ns();
    for (int it = 0; it < (1 << 24) && globaltimer_ns() - t0 < 20000000ull; ++it) {}
  }
  if ((warp == 1 || warp == 3) && rank == 0) {
    // every MMA this warp issued is complete before TMEM is released
    mma_commit_pair_warp(&bar_drain[warp >> 1]);
    mbar_wait(&bar_drain[warp >> 1], 0, 500000000ull);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // no CTA leaves while the pair's MMAs or barriers need it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, TMEM_COLS);
}

// Joins the partial results of every cut tile: a row's parts weighted by
// 2^(lse_s - max), in the order of the keys. A block takes 32 column vectors of one
// half and every 8th group of 8 rows; 8 threads read the 128 bytes of 8 lanes. The
// blocks of all pairs but the last that share a tile divide its row groups, so that
// a tile of many parts has many blocks (one pair's blocks alone took more than three times
// as long for a context of 131 k keys). No shared memory: the blocks get resident beside the attention kernel's,
// which leave none, and start when the last of those ends.
constexpr int CROWS = 8, CVECS = 32, CY = 8;

// Rows r0 + rr + step * k of the tile, k < K, for this thread's column vector; U
// parts of each in flight.
template <int LD, typename T, int K, int U>
__device__ __forceinline__ void latent_join(const LatentRecord& rec, char* ws, T* out, float* lse, int r0, int step) {
  const float* sums = (const float*)(ws + Layout::lse);
  const int32_t* bad = (const int32_t*)(ws + Layout::bad);
  const float4* parts = (const float4*)(ws + Layout::o);
  auto slot = [&](int s) { return s == 0 ? 2 * rec.owner + 1 : 2 * (rec.owner + s); };
  const int rr = threadIdx.x % CROWS, q = threadIdx.x / CROWS % 4;   // a warp: 8 rows x 4 vectors
  constexpr int ZH = LD / 8 / CVECS;   // blocks along a half's columns
  const int half = blockIdx.z / ZH, c = blockIdx.z % ZH * CVECS + threadIdx.x / CROWS;
  float m[K], total[K];
  float4 o[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    m[k] = -INFINITY;
    total[k] = 0.f;
    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // the four threads of a row in a warp share the search for its maximum
  int any = 0;
  for (int s = q; s < rec.parts; s += 4) {
    any |= bad[slot(s)];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int r = r0 + step * k + rr;
      if (r < rec.nrows) m[k] = fmaxf(m[k], sums[slot(s) * BM + r]);
    }
  }
  if (__any_sync(0xffffffffu, any)) return;   // (the warp looked at every part)
#pragma unroll
  for (int k = 0; k < K; ++k) {
    m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], 8));
    m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], 16));
    if (m[k] == -INFINITY) m[k] = 0.f;   // all scores -inf: weights 0, a result of NaN, a log sum of -inf
  }
  for (int s = 0; s < rec.parts; s += U) {
    float w[U][K];
    float4 y[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int r = r0 + step * k + rr;
        w[u][k] = -INFINITY;
        y[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rec.nrows && s + u < rec.parts) {
          w[u][k] = sums[slot(s + u) * BM + r];
          y[u][k] = parts[Layout::vec(LD, slot(s + u), r / HM, c, half * HM + r % HM)];
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float f = exp2f(w[u][k] - m[k]);
        total[k] += f;
        o[k].x += f * y[u][k].x;
        o[k].y += f * y[u][k].y;
        o[k].z += f * y[u][k].z;
        o[k].w += f * y[u][k].w;
      }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int r = r0 + step * k + rr;
    if (r >= rec.nrows) continue;
    const float inv = 1.f / total[k];
    const int64_t row = (int64_t)rec.row0 + r;
    uint2 y;
    y.x = pack2<T>(o[k].x * inv, o[k].y * inv);
    y.y = pack2<T>(o[k].z * inv, o[k].w * inv);
    *reinterpret_cast<uint2*>(out + row * LD + half * (LD / 2) + c * 4) = y;
    if (lse && blockIdx.z == 0 && threadIdx.x < CROWS) lse[row] = (m[k] + log2f(total[k])) * LN2;
  }
}

template <int LD, typename T>
__global__ void __launch_bounds__(CROWS * CVECS, 4) latent_combine_kernel(char* ws, T* out, float* lse) {
  pdl_wait();
  const int pair = blockIdx.x;
  const LatentRecord rec = ((const LatentRecord*)(ws + Layout::rec))[pair];
  const int step = CY * CROWS * (rec.parts - 1);
  const int r0 = ((int)blockIdx.y + CY * (pair - rec.owner)) * CROWS;   // this block's first row
  if (r0 >= rec.nrows) return;   // no cut tile (nrows 0), or not that many rows
  constexpr int K = BM / CROWS / CY;   // row groups of a block where two pairs share the tile
  // eight parts of one row group in flight a thread, or two of each of its groups
  if (r0 + step >= rec.nrows) latent_join<LD, T, 1, 8>(rec, ws, out, lse, r0, step);
  else latent_join<LD, T, K, 8 / K / 2>(rec, ws, out, lse, r0, step);
}

int pairs_of(const LatentAttnArgs& a) { return a.dev.num_sms / 2 < MAX_PAIRS ? a.dev.num_sms / 2 : MAX_PAIRS; }

// Whether the contexts are so short that cutting tiles costs more than it gives: a cut
// shortens the longest worker's way, to the tick's average, and costs the join with
// its launch and partial results (5 steps' time, and 5 more for a tile a worker, 10 for two or
// more). Lengths are known by their bound alone; on average they are taken for 0.6 of it.
// Graph-replayed, whole tiles against cut ones, latent 512, us, at 1 / 16 / 70 / 120 sequences of kv / 8
// to kv keys: 64 heads, kv 250: 8.8 9.1 11.4 18.5 against 12.9 14.2 19.5 27.5; 500: 12.1 12.2 15.1
// 24.9 against 13.1 15.5 26.3 32.7; 1000: 16.9 18.2 22.8 36.8 against 13.8 16.9 32.4 40.8.
// 8 heads, kv 64: 4.6 4.7 4.9 5.5 against 7.4 7.9 8.1 8.1; 500: 11.8 13.5 13.7 15.4 against
// 8.7 10.3 15.0 22.0; 1000: 20.0 21.5 23.9 25.2 against 8.6 11.5 21.4 27.9. 300 at 64 heads,
// kv 250: 33 against 40, 1000: 64 against 68; 400 at 8 heads, kv 1000: 61 against 56.
bool short_contexts(const LatentAttnArgs& a, const LatentTiling& t) {
  const int64_t per_seq = ((int64_t)a.T * a.H + a.B - 1) / a.B;   // rows, on average
  const int64_t tiles = (per_seq + t.rows - 1) / t.rows * a.B;
  const float steps = (float)((a.max_kv_len + (int64_t)t.keys - 1) / t.keys), share = (float)tiles / t.workers;
  return steps * (ceilf(share) - 0.6f * share) <= 5.f + 5.f * fminf(share, 2.f);
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

template <int LD, typename T, bool GATHER>
cudaError_t launch(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s) {
  constexpr int smem = Cfg<LD>::TILES + sizeof(State<LD, nthreads(GATHER)>);
  static_assert(smem <= 232448, "shared memory");
  static std::atomic<uint64_t> ready{0};   // devices whose kernel attribute is set
  if (!(ready.load() >> a.dev.id & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(latent_attn_kernel<LD, T, GATHER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << a.dev.id);
  }
  const CUtensorMapDataType dt =
      std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int box = GATHER ? HM : p.box;
  const int64_t pool_rows = (int64_t)a.num_pages * a.P;
  CUtensorMap mq, mx, m2;
  if (!make_map_chunks(&mq, a.q, dt, Cfg<LD>::CH, (int64_t)a.T * a.H, LD + 64, HM, Cfg<LD>::CH) ||
      !make_map_chunks(&mx, a.cache, dt, Cfg<LD>::CH, pool_rows, LD + 64, box, 1) ||
      !make_map_chunks(&m2, a.cache, dt, Cfg<LD>::CH, pool_rows, LD + 64, box, 2))
    return cudaErrorInvalidValue;
  const int pairs = pairs_of(a);
  cudaError_t e;
  {
    KernelTimer timer("latent_attn", s);
    e = launch_after_trigger(latent_attn_kernel<LD, T, GATHER>, dim3(2 * pairs), dim3(nthreads(GATHER)), smem, s, mq,
                             mx, m2, p);
  }
  if (e != cudaSuccess || p.whole) return e;
  KernelTimer timer("latent_combine", s);
  return launch_after_trigger(latent_combine_kernel<LD, T>, dim3(pairs, CY, 2 * LD / 8 / CVECS),
                              dim3(CROWS * CVECS), 0, s, a.ws, (T*)a.out, a.lse);
}

template <int LD, typename T>
cudaError_t launch_either(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s) {
  return p.gather ? launch<LD, T, true>(a, p, s) : launch<LD, T, false>(a, p, s);
}

}  // namespace

// The same for every call: a workspace serves larger and smaller calls, and those of
// either kernel.
size_t latent_attn_workspace(int32_t, int32_t, int32_t, int32_t latent_dim) {
  const size_t a = Layout::total(latent_dim), b = latent_rows_workspace(latent_dim);
  return a > b ? a : b;
}

cudaError_t launch_latent_attn(const LatentAttnArgs& a, cudaStream_t s) {
  // Up to 16 rows a sequence on average go 16 to a tile on mma.sync, which HBM
  // bounds; with more of them the tensor cores' tiles of 128 rows read the keys
  // less often (rows of one sequence share a pass over its keys). Decode of 96 sequences
  // of 1000-8000 keys, latent 512, mma.sync against tcgen05: 8 heads 88 / 105 us,
  // 16 heads 94 / 106, 20 heads 153 / 107, 64 heads 292 / 115; of 4 sequences of up to
  // 500 keys: 16 heads 11.7 / 12.0, 32 heads 12.7 / 12.5.
  const bool rows = (int64_t)a.T * a.H <= (int64_t)16 * a.B;
  LatentAttnP p;
  p.cu = a.cu;
  p.kv_lens = a.kv_lens;
  p.page_tables = a.page_tables;
  p.B = a.B;
  p.T = a.T;
  p.H = a.H;
  p.P = a.P;
  // Rows of a TMA box: they lie in one page and in one slot.
  p.box = gcd(a.P, rows ? latent_rows_slot() : HM);
  // Boxes of fewer than 32 rows lose to thread copies: 64 sequences of 1000-4000 keys at 128
  // heads, TMA against copies: page size 64 58.5 / 61.8 us, 32 61.9 / 61.8, 16 67.9 / 61.6 (8 and 1,
  // in an earlier form of the kernel: 92 / 70 and 352 / 72; copies now take 63 and 65); the 16-row
  // kernel takes one box a slot.
  p.gather = p.box < 32;
  if (p.gather) p.box = 1;
  p.whole = short_contexts(a, rows ? latent_rows_tiling(a.dev.num_sms) : LatentTiling{BM, BN, pairs_of(a)});
  p.cache = a.cache;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.max_kv_len = a.max_kv_len;
  p.table_cap = a.max_pages * a.P;
  p.scale_log2 = a.scale * LOG2E;
  p.out = a.out;
  p.out_32 = ((uintptr_t)a.out & 31) == 0;
  p.lse = a.lse;
  p.ws = a.ws;
  p.dev_status = a.dev.status;
  if (rows) return launch_latent_rows(a, p, s);
  if (a.dtype == PKV_BF16)
    return a.latent_dim == 512 ? launch_either<512, __nv_bfloat16>(a, p, s)
                               : launch_either<256, __nv_bfloat16>(a, p, s);
  return a.latent_dim == 512 ? launch_either<512, __half>(a, p, s) : launch_either<256, __half>(a, p, s);
}

}  // namespace pkv
