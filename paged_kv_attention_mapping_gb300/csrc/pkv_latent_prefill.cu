// Expanded latent attention of chunks: head h of row i of a sequence, with
// query [qn, qr], attends keys [kn_j, r_j] (r shared by the heads) and values v_j:
//   s_j = scale (qn . kn_j + qr . r_j),  j <= kv_len - q_len + i,
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + ln(sum).
//
// Every head has its own keys, so the tensor cores get their work from the query
// rows. A pair of CTAs (tcgen05 cta_group::2) works on two query tiles of 256 rows
// whose products alternate, so that one tile's softmax runs under the other's MMAs;
// each CTA has 128 rows of either tile, half of the keys of a step (for S) and half
// of the value columns (for O). Per 128 keys and query tile: S = Q K^T (M 256, N 128,
// K 128 + 64) and O += P V (M 256, N 128, K 128): 2560 tensor cycles for both tiles.
// The two tiles are 512 rows of one head, which share every key tile, or, for a
// sequence's 256 rows or fewer that do not fill such a tile, the same rows of two heads.
// (One CTA with two tiles of 128 rows needs twice the shared memory for a step's
// keys: beside Q it held 1.6 steps, waited for loads, and took 499 us for 4096 tokens at
// 128 heads in bf16, this one 447: 1538 TFLOP/s.)
//
//   warp 0     TMA producer (each CTA its halves): Q of both tiles, K_j (nope part
//              and rotary part) and V_j into rings of three; V rows behind the
//              sequence's end are zeroed. The even CTA's claims the tiles.
//   warps 1, 2 MMA issuers of query tile 0, 1 (even CTA): per key tile j,
//              O_w += P_w V_{j-1}, then S_w = Q_w K_j^T over the same TMEM columns as
//              P_w (a warp's MMAs run in issue order, so the product has read P_w by
//              then). The tensor pipe queues next to nothing, and a wait or commit costs
//              its warp 100-400 cycles: the two take turns, and each does its waits and
//              commits under the other's MMAs.
//   warps 4-7, 8-11  softmax of query tile 0, 1, a thread per row; P goes back
//              over S in TMEM as the A operand of the next product, rounded to the type of
//              the values (one product's operands have one type: half a step of each weight,
//              while sums and maxima stay fp32), handed over in two halves. O is rescaled
//              only when a row's maximum grows by more than 2^8.
//
// Where the tiles are at most half as many as the pairs of CTAs (short chunks, few
// heads), each tile's keys are cut into parts, as many as there are pairs for;
// latent_prefill_combine_kernel joins their partial results.
//
// A plan kernel counts the tiles; where the call's sizes allow no more of them than pairs
// of CTAs, each pair finds its own.
//
// Tiles go head by head, each head's from its last rows (most keys) to its first:
// the CTAs that run at one time share few heads' keys, which stay in L2, and the
// last tiles to be claimed are short. Longer sequences come before shorter ones.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_latent.cuh"
#include "pkv_sm100.cuh"

namespace pkv {
using namespace sm100;

namespace {

constexpr int NOPE = 128, DV = 128;
constexpr int BM = 128;          // rows of a query tile
constexpr int BN = 128;          // keys of a step
constexpr int QM = 2 * BM;       // rows of a query tile
constexpr int ROWS = 2 * QM;     // rows of a work tile of one head
constexpr int NTHREADS = 384;
constexpr uint32_t UNIT = 16384;            // 128 rows x 64 columns of 16 bits
constexpr uint32_t Q_BYTES = 3 * UNIT;      // one CTA's rows of a query tile
constexpr int NK = 3, NV = 3;               // ring slots
constexpr uint32_t KUNIT = UNIT / 2;        // 64 keys x 64 columns
constexpr uint32_t K_BYTES = 3 * KUNIT;     // one CTA's keys of a step: nope columns, rotary columns
constexpr uint32_t V_BYTES = UNIT;          // one CTA's 64 value columns of a step's keys
constexpr uint32_t SMEM = 2 * Q_BYTES + NK * K_BYTES + NV * V_BYTES + 1024;
static_assert(SMEM <= 231424, "shared memory");
constexpr uint32_t TMEM_COLS = 512;         // S of both tiles, then O of both
constexpr float RESCALE_LOG2 = 8.f;
constexpr long long WAIT_LIMIT_CLOCKS = 4000000000ll;   // about two seconds
constexpr int PLAN_THREADS = 1024;

// Workspace: the next tile to claim, the number of tiles (parts of one count), the
// largest number of parts; the sequences in the order they are worked on, the
// tiles before each; and, used by calls that split: a record, log2 sums and outputs
// (fp32, normalised) per part.
struct Layout {
  size_t order, first, rec, lse, o, total;
};
constexpr int MAX_PAIRS = 76;      // 152 SMs
// A tile is cut into parts of MIN_STEPS or more if its longest part is at least
// MIN_SAVED steps shorter than the whole: the partial results and their join take 6-8
// us, a step 1.6. (16 heads, chunk 512 after 32768 keys: 394 -> 117 us; 128 after 8192:
// 106 -> 32; cut all the same, 256 after 700 took 29 us instead of 25.)
constexpr int MIN_STEPS = 4, MIN_SAVED = 8;
// Whether a call's tiles can be few enough to split (its padding rows aside).
bool may_split(int32_t Tq, int32_t H) { return (int64_t)Tq * H * 2 <= (int64_t)ROWS * MAX_PAIRS; }
Layout layout(int32_t B) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  // Room for parts whether this call may split or not (20 MB): a workspace for a large
  // call, which does not, serves smaller ones, which do.
  const size_t parts = MAX_PAIRS;
  Layout l;
  l.order = 256;
  l.first = l.order + al((size_t)B * 4);
  l.rec = l.first + al(((size_t)B + 1) * 4);
  l.lse = l.rec + al(parts * 128);
  l.o = l.lse + parts * ROWS * 4;
  l.total = l.o + parts * ROWS * DV * 4;
  return l;
}

struct PrefillP {
  const int32_t *cu_q, *cu_k;
  int32_t B, H, Tq, Tk;
  int32_t out_32;              // out is 32-byte aligned
  int32_t direct;              // no plan: every pair of CTAs finds its one tile itself
  int32_t kn_heads, v_heads;   // 0: every head reads head 0 (a head stride of 0)
  float scale_log2;            // > 0
  void* out;
  float* lse;
  int32_t *ctrl, *order, *first;
  char* rec;        // null: the call does not split
  float* part_lse;
  float4* part_o;
  int32_t* dev_status;
};

// A sequence's rows: tiles of ROWS rows of one head, the last of them with more than
// QM, or, where no more than QM are left over, those (its first rows) as tiles of
// one query tile of each of two heads (one head a tile: 189 us, not 170, for eight
// chunks after prefixes; no difference where pairs of CTAs are left without a tile).
__device__ __forceinline__ int narrow_rows(int q) {
  const int rest = q % ROWS;
  return rest <= QM ? rest : 0;
}
__device__ __forceinline__ int wide_tiles(int q) { return q / ROWS + (q % ROWS > QM); }
// Parts of a tile of a sequence with L keys, of which there may be `most`.
__device__ __forceinline__ int parts_of(int L, int most) {
  const int n = (L + BN - 1) / BN, parts = max(1, min(most, n / MIN_STEPS));
  return n - (n + parts - 1) / parts >= MIN_SAVED ? parts : 1;
}

// Work items of a sequence of q rows and L keys: its tiles' parts.
__device__ __forceinline__ int items_of(int q, int L, int H, int parts) {
  return (wide_tiles(q) * H + (narrow_rows(q) ? (H + 1) / 2 : 0)) * parts_of(L, parts);
}
// The tiles of a call whose lengths are not known: a tile of one head has more than QM
// rows of it, and no sequence has tiles of two heads more than once.
int64_t most_tiles(int32_t B, int32_t Tq, int32_t H) {
  return (int64_t)(Tq / (QM + 1)) * H + (int64_t)(B < Tq ? B : Tq) * ((H + 1) / 2);
}

// One CTA: checks the lengths, orders the sequences by keys (descending, up to
// PLAN_THREADS of them; more stay in their own order) and counts their tiles. The
// launch takes as many warps as there are sequences to look at: every block barrier
// here is on the way to the first tile.
__global__ void __launch_bounds__(PLAN_THREADS) latent_prefill_plan_kernel(const int32_t* __restrict__ cu_q,
                                                                          const int32_t* __restrict__ cu_k,
                                                                          int32_t B, int32_t Tq, int32_t Tk,
                                                                          int32_t H, int32_t pairs, int32_t split,
                                                                          int32_t* ctrl,
                                                                          int32_t* order, int32_t* first,
                                                                          int32_t* dev_status) {
  __shared__ int s_cost[PLAN_THREADS], s_rank[PLAN_THREADS], s_scan[32], s_carry, s_all;
  pdl_trigger();   // (whatever starts now waits for this kernel's end)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = blockDim.x;
  // The kernel before may have written the lengths, and an earlier call may still be
  // reading the workspace, until here.
  pdl_wait();
  const bool sorted = B <= nt;
  bool bad = tid == 0 && (__ldg(cu_q) != 0 || __ldg(cu_k) != 0 || __ldg(cu_q + B) > Tq || __ldg(cu_k + B) > Tk);
  for (int b = tid; b < B; b += nt)
    bad |= __ldg(cu_q + b + 1) < __ldg(cu_q + b) || __ldg(cu_k + b + 1) < __ldg(cu_k + b);
  bad = __syncthreads_or(bad);
  if (tid == 0) s_all = 0;
  int parts = 1;
  auto tiles_of = [&](int b, int* keys) {
    const int q = __ldg(cu_q + b + 1) - __ldg(cu_q + b), L = __ldg(cu_k + b + 1) - __ldg(cu_k + b);
    *keys = L;
    if (bad || q == 0) return 0;
    if (L < q) {
      atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
      return 0;
    }
    return items_of(q, L, H, parts);
  };
  if (split) {
    __syncthreads();
    int keys, mine = 0;   // (no more than pairs + 1 counts)
    for (int b = tid; b < B; b += nt) mine = min(pairs + 1, mine + min(pairs + 1, tiles_of(b, &keys)));
    if (mine > 0) atomicAdd(&s_all, mine);
    __syncthreads();
    if (s_all > 0) parts = max(1, pairs / s_all);
  }
  if (sorted) {
    int keys = 0;
    const int n = tid < B ? tiles_of(tid, &keys) : 0;
    s_cost[tid] = n > 0 ? keys : 0;
    __syncthreads();
    if (tid < B) {
      int rank = 0;
      for (int c = 0; c < B; ++c) rank += s_cost[c] > s_cost[tid] || (s_cost[c] == s_cost[tid] && c < tid);
      s_rank[rank] = tid;
    }
    __syncthreads();
  }
  if (tid == 0) s_carry = 0;
  for (int base = 0; base < B; base += nt) {
    __syncthreads();
    const int carry = s_carry;
    const int k = base + tid;
    int b = 0, keys, n = 0;
    if (k < B) {
      b = sorted ? s_rank[k] : k;
      n = tiles_of(b, &keys);
    }
    int scan = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < nt / 32; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    if (k < B) {
      order[k] = b;
      first[k] = before + scan - n;
    }
    __syncthreads();
    if (tid == 0) s_carry = all;
  }
  __syncthreads();
  if (tid == 0) {
    first[B] = s_carry;
    ctrl[0] = pairs;   // a pair's first tile has the pair's number
    ctrl[1] = s_carry;
    ctrl[2] = parts;
    if (bad) atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
  }
}

// A work tile. Query tile w: head h[w], nr[w] rows (0: none) from packed row row0[w],
// the first at position pos[w], reading n[w] key tiles. split: the two tiles
// are of two heads, with keys of their own.
// The work is steps [j0, j1) of the n[] key tiles: part number part of parts,
// the tile's first part being item number item0.
struct Tile {
  int valid, split, k0, L;
  int j0, j1, part, parts, item0;
  int h[2], row0[2], nr[2], pos[2], n[2];
};
static_assert(sizeof(Tile) <= 128, "record");
// First step of a part of n steps (fewer than 2^24 steps and 2^7 parts).
__device__ __forceinline__ int part_begin(int n, int part, int parts) { return n * part / parts; }

// By a warp: what the plan kernel finds out, for calls of no more items than pairs of CTAs
// (no more sequences either): the number of items, the largest number of parts, and the
// sequence of item `item` with the number of items before it.
struct Found {
  int items, parts, b, before;
};
__device__ __forceinline__ Found find_item(const PrefillP& p, int item, int pairs) {
  const int lane = threadIdx.x & 31;
  bool bad = lane == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_k) != 0 || __ldg(p.cu_q + p.B) > p.Tq ||
                           __ldg(p.cu_k + p.B) > p.Tk);
  for (int b = lane; b < p.B; b += 32)
    bad |= __ldg(p.cu_q + b + 1) < __ldg(p.cu_q + b) || __ldg(p.cu_k + b + 1) < __ldg(p.cu_k + b);
  bad = __any_sync(0xffffffffu, bad);
  Found f{0, 1, 0, 0};
  auto items = [&](int b) {
    if (bad || b >= p.B) return 0;
    const int q = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b), L = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
    if (q > 0 && L < q && item == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return q == 0 || L < q ? 0 : items_of(q, L, p.H, f.parts);
  };
  if (bad && item == 0 && lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
  if (p.rec) {
    int all = 0;
    for (int b = lane; b < p.B; b += 32) all += items(b);
    all = __reduce_add_sync(0xffffffffu, all);
    if (all > 0) f.parts = max(1, pairs / all);
  }
  for (int base = 0; base < p.B; base += 32) {
    const int n = items(base + lane);
    int scan = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    const int before = f.items + scan - n;
    const unsigned here = __ballot_sync(0xffffffffu, before <= item && item < before + n);
    if (here) {
      f.b = base + __ffs(here) - 1;
      f.before = __shfl_sync(0xffffffffu, before, __ffs(here) - 1);
    }
    f.items += __shfl_sync(0xffffffffu, scan, 31);
  }
  return f;
}

// Partial outputs: for a part and 128 rows (a CTA's of a query tile), four columns
// at a time, the rows side by side. The vector of row r (of ROWS) and columns 4 c ..
__device__ __forceinline__ int64_t part_vec(int item, int r, int c) {
  return (((int64_t)item * (ROWS / BM) + r / BM) * (DV / 4) + c) * BM + r % BM;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mr,
                          PrefillP p) {
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = sm;                         // [query tile][3 units]
  unsigned char* sK = sQ + 2 * Q_BYTES;           // [slot][nope, nope, rotary]
  unsigned char* sV = sK + NK * K_BYTES;          // [slot]

  // q, k, v and p are waited on in the even CTA, where both CTAs arrive; the MMA
  // commits signal kempty, vempty, qempty, s and o in both
  __shared__ __align__(8) uint64_t bar_q, bar_qempty, bar_k[NK], bar_kempty[NK], bar_v[NV], bar_vempty[NV], bar_vtail,
      bar_s[2], bar_p[2][2], bar_o[2], bar_tfull[2], bar_tempty[2], bar_turn[2], bar_drain[2];
  __shared__ uint32_t s_tmem;
  __shared__ Tile s_tile[2];
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    mbar_init(&bar_q, 2);
    mbar_init(&bar_qempty, 2);             // both issuers
    for (int s = 0; s < NK; ++s) {
      mbar_init(&bar_k[s], 2);
      mbar_init(&bar_kempty[s], 2);        // both issuers, or one of them twice
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&bar_v[s], 2);
      mbar_init(&bar_vempty[s], 2);
    }
    mbar_init(&bar_vtail, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      for (int hf = 0; hf < 2; ++hf) mbar_init(&bar_p[w][hf], 8);   // four softmax warps of either CTA
      mbar_init(&bar_o[w], 1);
      mbar_init(&bar_tfull[w], 1);
      mbar_init(&bar_tempty[w], 2 + 8 + 8 + 1);   // issuers, softmax warps of both CTAs, the odd CTA's producer
      mbar_init(&bar_turn[w], 1);
      mbar_init(&bar_drain[w], 1);
    }
    fence_mbar_init();
    mbar_arrive(&bar_turn[0]);   // query tile 0 has the first turn
    s_abort = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mr);
  }
  if (warp == 1) tmem_alloc_pair(&s_tmem, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();   // the peer's barriers are ready too
  const uint32_t tmem = s_tmem;
  pdl_wait();   // the plan, and whatever wrote the inputs, the lengths among them

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
  // the tile of entry e, once it is there
  auto wait_tile = [&](uint32_t t) -> bool {
    const bool there = wait(&bar_tfull[t & 1], (t >> 1) & 1);
    if (rank) fence_cluster();   // the even CTA wrote it
    return there;
  };
  const uint32_t tempty = map_to_rank(bar_tempty, 0);
  bool ok = true;

  if (warp == 0) {
    // --------------------------------------------------------------- producer
    Found found{0, 1, 0, 0};
    if (p.direct) found = find_item(p, blockIdx.x >> 1, gridDim.x >> 1);
    const int n_tiles = p.direct ? found.items : *(volatile const int32_t*)&p.ctrl[1];
    const int most_parts = p.direct ? found.parts : *(volatile const int32_t*)&p.ctrl[2];
    if (p.direct && p.rec && blockIdx.x == 0 && lane == 0) {   // for the join
      p.ctrl[1] = n_tiles;
      p.ctrl[2] = most_parts;
    }
    const uint32_t q_bar = map_to_rank(&bar_q, 0);
    uint32_t n_claims = 0;
    // Up to 32 sequences: a lane keeps one, in the plan's order, so that a claim waits for
    // nothing but its number (16 chunks of 30-128 rows after 2000 keys at 32 heads 154.3 -> 150.2 us).
    const bool kept = !p.direct && p.B <= 32;
    int my_b = 0, my_first = INT32_MAX, my_q0 = 0, my_q = 0, my_k0 = 0, my_L = 0;
    if (rank == 0 && kept && lane < p.B) {
      my_b = p.order[lane];
      my_first = p.first[lane];
      my_q0 = __ldg(p.cu_q + my_b);
      my_q = __ldg(p.cu_q + my_b + 1) - my_q0;
      my_k0 = __ldg(p.cu_k + my_b);
      my_L = __ldg(p.cu_k + my_b + 1) - my_k0;
    }
    uint32_t n_k = 0, n_v = 0, n_tail = 0;    // K, V loads and last tiles with rows to zero so far
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      if (rank == 0 || p.direct) {   // (without a plan both CTAs find the tile)
        // entry e is free again once every consumer is done with tile t - 2
        if (t >= 2 && !(ok = wait(&bar_tempty[e], ((t >> 1) - 1) & 1))) break;
        Tile ti{};
        for (bool skip = true; skip;) {
          int tt = n_claims++ == 0 ? (int)(blockIdx.x >> 1) : p.direct ? n_tiles : lane == 0 ? atomicAdd(&p.ctrl[0], 1) : 0;
          tt = __shfl_sync(0xffffffffu, tt, 0);
          if (__any_sync(0xffffffffu, s_abort)) tt = n_tiles;
          int lo = 0;   // the last sequence that starts at or before tile tt, searched 32 ways
          for (int m = p.direct || kept || tt >= n_tiles ? 0 : p.B; m > 1;) {
            const int step = (m + 31) / 32, at = lo + lane * step;
            const bool before = lane * step < m && p.first[at] <= tt;
            lo += (__popc(__ballot_sync(0xffffffffu, before)) - 1) * step;
            m = min(step, p.B - lo);
          }
          skip = false;
          if (tt < n_tiles) {
            int before, q_lo, q;
            if (kept) {
              lo = 31 - __clz(__ballot_sync(0xffffffffu, my_first <= tt));
              before = __shfl_sync(0xffffffffu, my_first, lo);
              q_lo = __shfl_sync(0xffffffffu, my_q0, lo);
              q = __shfl_sync(0xffffffffu, my_q, lo);
              ti.k0 = __shfl_sync(0xffffffffu, my_k0, lo);
              ti.L = __shfl_sync(0xffffffffu, my_L, lo);
            } else {
              const int b = p.direct ? found.b : p.order[lo];
              before = p.direct ? found.before : p.first[lo];
              q_lo = __ldg(p.cu_q + b);
              q = __ldg(p.cu_q + b + 1) - q_lo;
              ti.k0 = __ldg(p.cu_k + b);
              ti.L = __ldg(p.cu_k + b + 1) - ti.k0;
            }
            const int wide = wide_tiles(q), rest = narrow_rows(q);
            int at = tt - before;
            ti.parts = 1;
            ti.part = 0;
            if (most_parts > 1) {
              ti.parts = parts_of(ti.L, most_parts);
              ti.part = at % ti.parts;
              at /= ti.parts;
            }
            ti.item0 = tt - ti.part;
            ti.split = at >= wide * p.H;
            const int h = ti.split ? (at - wide * p.H) * 2 : at / wide;
            const int q0 = ti.split ? 0 : rest + (wide - 1 - (at - h * wide)) * ROWS;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int q_w = ti.split ? 0 : q0 + w * QM;
              ti.h[w] = h + (ti.split ? w : 0);
              ti.row0[w] = q_lo + q_w;
              ti.nr[w] = ti.split ? (ti.h[w] < p.H ? rest : 0) : max(0, min(QM, q - q_w));
              ti.pos[w] = ti.L - q + q_w;
              ti.n[w] = ti.nr[w] ? (ti.pos[w] + ti.nr[w] + BN - 1) / BN : 0;
            }
            const int n = max(ti.n[0], ti.n[1]);
            ti.parts = min(ti.parts, n);   // (a tile's own steps may be fewer than its sequence's)
            skip = ti.part >= ti.parts;
            ti.j0 = 0;
            ti.j1 = n;
            if (ti.parts > 1 && !skip) {
              ti.j0 = part_begin(n, ti.part, ti.parts);
              ti.j1 = part_begin(n, ti.part + 1, ti.parts);
            }
            ti.valid = 1;
            if (most_parts > 1 && rank == 0 && lane == 0) *reinterpret_cast<Tile*>(p.rec + (size_t)tt * 128) = ti;
          } else {
            ti.valid = 0;
          }
        }
        if (lane == 0) {
          s_tile[e] = ti;
          if (!p.direct) {
            const uint32_t peer = map_to_rank(&s_tile[e], 1);
            const uint32_t* words = reinterpret_cast<const uint32_t*>(&ti);
#pragma unroll
            for (int i = 0; i < (int)(sizeof(Tile) / 4); ++i) st_cluster_u32(peer + 4 * i, words[i]);
            fence_cluster();
            mbar_arrive_cluster(map_to_rank(&bar_tfull[e], 1));
          }
          mbar_arrive(&bar_tfull[e]);
        }
        __syncwarp();
      }
      if (!(ok = wait_tile(t))) break;
      const Tile ti = s_tile[e];
      if (!ti.valid) break;
      const int streams = ti.split && ti.nr[1] ? 2 : 1;
      // Q of this tile replaces the one before once its last S is done
      if (t >= 1 && !(ok = wait(&bar_qempty, (t - 1) & 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx_cluster(q_bar, (ti.nr[1] ? 2 : 1) * Q_BYTES);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (ti.nr[w])
              tma_load_3d_pair(sQ + w * Q_BYTES + c * UNIT, &mq, q_bar, c * 64, ti.h[w], ti.row0[w] + (int)rank * BM);
      }
      __syncwarp();
      for (int j = ti.j0; j < ti.j1 && ok; ++j) {
        for (int w = 0; w < streams; ++w, ++n_k) {
          const uint32_t slot = n_k % NK;
          if (!(ok = wait(&bar_kempty[slot], ((n_k / NK) & 1) ^ 1))) break;
          if (lane == 0) {
            const uint32_t bar = map_to_rank(&bar_k[slot], 0);
            unsigned char* dst = sK + slot * K_BYTES;
            const int row = ti.k0 + j * BN + (int)rank * (BN / 2), h = ti.h[w] * p.kn_heads;
            mbar_arrive_expect_tx_cluster(bar, K_BYTES);
            tma_load_3d_pair(dst, &mk, bar, 0, h, row);
            tma_load_3d_pair(dst + KUNIT, &mk, bar, 64, h, row);
            tma_load_2d_pair(dst + 2 * KUNIT, &mr, bar, 0, row);
          }
          __syncwarp();
        }
        if (!ok) break;
        for (int w = 0; w < streams; ++w, ++n_v) {
          const uint32_t slot = n_v % NV;
          if (!(ok = wait(&bar_vempty[slot], ((n_v / NV) & 1) ^ 1))) break;
          const uint32_t bar = map_to_rank(&bar_v[slot], 0);
          unsigned char* dst = sV + slot * V_BYTES;
          const int end = ti.L - j * BN;   // rows from here on are behind the sequence
          if (lane == 0) {
            const int col = (int)rank * (DV / 2), h = ti.h[w] * p.v_heads, row = ti.k0 + j * BN;
            if (end < BN) {
              mbar_arrive_expect_tx(&bar_vtail, V_BYTES);
              tma_load_3d(dst, &mv, &bar_vtail, col, h, row);
            } else {
              mbar_arrive_expect_tx_cluster(bar, V_BYTES);
              tma_load_3d_pair(dst, &mv, bar, col, h, row);
            }
          }
          __syncwarp();
          if (end < BN) {
            // 0 * NaN must not reach O from the rows behind the sequence's end
            if (!(ok = wait(&bar_vtail, n_tail++ & 1))) break;
            uint4* base = (uint4*)dst;
            for (int x = end * 8 + lane; x < BN * 8; x += 32) base[x] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(bar);
          }
        }
      }
      if (rank && ok && lane == 0) mbar_arrive_cluster(tempty + e * 8);
      __syncwarp();
    }
    if (!ok && lane == 0) {
      // let every copy this warp issued land before the CTA may exit
      const uint64_t t0 = globaltimer_ns();
      for (int it = 0; it < (1 << 24) && globaltimer_ns() - t0 < 20000000ull; ++it) {}
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers
    if (rank == 0) {
      const int w = warp - 1;
      const uint32_t id_s = idesc_f16(QM, BN, BF16, false);
      const uint32_t id_o = idesc_f16(QM, DV, BF16, true);
      const uint64_t qd = smem_desc(smem_u32(sQ) + w * Q_BYTES, 16, 1024, LAYOUT_SW128);
      const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, LAYOUT_SW128);
      const uint64_t vd = smem_desc(smem_u32(sV), UNIT, 1024, LAYOUT_SW128);
      const uint32_t s_tm = tmem + w * 128, o_tm = tmem + 256 + w * 128;
      uint32_t base = 0;                  // K (and V) loads before the current tile
      uint32_t n_p = 0, turns = 0;
      for (uint32_t t = 0; ok; ++t) {
        const uint32_t e = t & 1;
        if (!(ok = wait_tile(t))) break;
        if (!s_tile[e].valid) break;
        const int n = s_tile[e].j1 - s_tile[e].j0;               // steps, and those of this query tile
        const int mine = max(0, min(n, s_tile[e].n[w] - s_tile[e].j0));
        const bool both = s_tile[e].nr[1] != 0, split = s_tile[e].split && both;
        const bool active = mine > 0;
        // a slot that one tile alone reads is released by two commits of its issuer
        const bool twice = split || !both;
        if (!(ok = wait(&bar_q, t & 1))) break;
        // turn j: O_w (+)= P_w V_{j-1}, then S_w = Q_w K_j^T. The first product of a
        // tile overwrites O_w: its P comes after the softmax threads read the
        // tile before out of TMEM. A query tile that is done, or absent, takes its
        // turns, and releases what it shares, like the other.
        for (int j = 0; j <= n; ++j) {
          const uint32_t kl = base + (split ? 2 * j + w : j), vl = base + (split ? 2 * (j - 1) + w : j - 1);
          const uint32_t ks = kl % NK, vs = vl % NV;
          const bool o = j > 0 && j - 1 < mine, sj = j < mine;
          const bool has_v = j > 0 && (active || !twice), has_k = j < n && (active || !twice);
          if (has_v && !(ok = wait(&bar_v[vs], (vl / NV) & 1))) break;
          if (has_k && !(ok = wait(&bar_k[ks], (kl / NK) & 1))) break;
          // the turn before P: P comes last in the steady state, and the product follows it at once
          if (!(ok = wait(&bar_turn[w], turns++ & 1))) break;
          if (o) {
            const uint64_t v = vd + (uint64_t)((vs * V_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k) {
              if ((k & 3) == 0) {
                if (!(ok = wait(&bar_p[w][k >> 2], n_p & 1))) break;
                tc_fence_after();
              }
              mma_f16_ta_pair_warp(o_tm, s_tm + k * 8, v + (uint64_t)((k * 2048) >> 4), id_o,
                                   (j > 1 || k > 0) ? 1u : 0u);
            }
            if (!ok) break;
            ++n_p;
          }
          if (has_v) {
            mma_commit_pair_warp(&bar_vempty[vs]);
            if (twice) mma_commit_pair_warp(&bar_vempty[vs]);
          }
          if (sj) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 12; ++k) {
              // the other tile's first MMAs may follow the last two of this turn at once
              if (k == 10 && lane == 0) mbar_arrive(&bar_turn[w ^ 1]);
              mma_f16_ss_pair_warp(s_tm, qd + (uint64_t)(((k >> 2) * UNIT + (k & 3) * 32) >> 4),
                                   kd + (uint64_t)((ks * K_BYTES + (k >> 2) * KUNIT + (k & 3) * 32) >> 4), id_s,
                                   k ? 1u : 0u);
            }
            mma_commit_pair_warp(&bar_s[w]);
          } else if (lane == 0) {
            mbar_arrive(&bar_turn[w ^ 1]);
          }
          __syncwarp();
          if (o && j == mine) mma_commit_pair_warp(&bar_o[w]);
          if (has_k) {
            mma_commit_pair_warp(&bar_kempty[ks]);
            if (twice) mma_commit_pair_warp(&bar_kempty[ks]);
          }
          if (j == n - 1) mma_commit_pair_warp(&bar_qempty);
        }
        base += split ? 2 * n : n;
        if (ok && lane == 0) mbar_arrive_cluster(tempty + e * 8);
        __syncwarp();
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax
    const int w = (warp - 4) >> 2;                // query tile
    const int quarter = warp & 3;                 // TMEM lanes of this warp
    const int i = (int)rank * BM + quarter * 32 + lane;   // row of the query tile
    const uint32_t lrow = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = w * 128, o_col = 256 + w * 128;
    const uint32_t p_bar = map_to_rank(bar_p[w], 0);
    const float sc = p.scale_log2;
    constexpr float SHIFT = weight_shift<T>(RESCALE_LOG2);
    uint32_t n_s = 0, n_o = 0;                    // S and O hand-offs taken
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      if (!(ok = wait_tile(t))) break;
      const Tile& ti = s_tile[e];
      if (!ti.valid) break;
      const int j0 = ti.j0, j1 = min(ti.j1, ti.n[w]);
      if (j0 < j1) {
        const int pos = min(ti.pos[w] + i, ti.L - 1);
        const int j_mask = (ti.pos[w] + (int)rank * BM + 1) / BN;   // key tiles before have no hidden key
        float m_run = -INFINITY, l_run = 0.f;
        for (int j = j0; j < j1; ++j) {
          // S complete also means that the product that read P is
          if (!(ok = wait(&bar_s[w], n_s & 1))) break;
          ++n_s;
          tc_fence_after();
          uint32_t r[2][2][32];   // two halves of 64 keys
          auto load = [&](int hf, uint32_t (&x)[2][32]) {
            tmem_ld32(tmem + lrow + s_col + hf * 64, x[0]);
            tmem_ld32(tmem + lrow + s_col + hf * 64 + 32, x[1]);
          };
          const bool masked = j >= j_mask;
          auto arrived = [&](int hf, uint32_t (&x)[2][32]) {
            reg_fence(x[0]);
            reg_fence(x[1]);
            if (masked) {
              const int lim = pos - j * BN - hf * 64;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (c * 32 + k > lim) x[c][k] = __float_as_uint(-INFINITY);
            }
          };
          load(0, r[0]);
          load(1, r[1]);
          tmem_wait_ld();
          arrived(0, r[0]);
          arrived(1, r[1]);
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              mx[(k >> 1) & 7] = max3(mx[(k >> 1) & 7], __uint_as_float(r[c >> 1][c & 1][k]),
                                      __uint_as_float(r[c >> 1][c & 1][k + 1]));
          const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
          const bool first = j == j0;
          const bool grow = first || mt > m_run + RESCALE_LOG2;
          const float m_new = grow ? fmaxf(mt, m_run) : m_run;
          if (!first && __any_sync(0xffffffffu, grow)) {
            // (m_new is finite: it grew)
            const float alpha = grow ? ex2(m_run - m_new) : 1.f;
            l_run *= alpha;
#pragma unroll 1
            for (int c = 0; c < DV / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_wait(tmem + lrow + o_col + c * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st32_wait(tmem + lrow + o_col + c * 32, o);
            }
          }
          m_run = m_new;
          // a row that sees no key of this part so far has m = -inf: its weights are 0
          const float nm = m_run == -INFINITY ? 0.f : SHIFT - m_run;
          const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nm, nm);
          float2 ls[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if (hf == 1) {   // read again: held through the first half's exponentials it spills (475 us, not 450)
              load(1, r[0]);
              tmem_wait_ld();
              arrived(1, r[0]);
            }
            uint32_t pw[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int k0 = 2 * k;
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[0][k0 >> 5][k0 & 31]),
                                                      __uint_as_float(r[0][k0 >> 5][(k0 & 31) + 1])), sc2, nm2);
              const float2 y = make_float2(ex2(x.x), ex2(x.y));
              ls[k & 3] = __fadd2_rn(ls[k & 3], y);
              pw[k] = pack2<T>(y.x, y.y);
            }
            tmem_st32(tmem + lrow + s_col + hf * 32, pw);
            tmem_wait_st();
            reg_fence(pw);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(p_bar + hf * 8);
          }
          l_run += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
        }
        if (!ok) break;
        if (!(ok = wait(&bar_o[w], n_o & 1))) break;
        ++n_o;
        tc_fence_after();
        const bool store = i < ti.nr[w];
        const bool whole = ti.parts == 1;
        // No visible key in a part: zeros. A whole tile's row always sees keys; where all
        // their scores are -inf it becomes NaN, as the formula has it.
        const float inv = l_run == 0.f && !whole ? 0.f : 1.f / l_run;
        const int64_t row = (int64_t)(ti.row0[w] + i) * p.H + ti.h[w];
        const int prow = (ti.item0 + ti.part) * ROWS + w * QM + i;
        float4* part = p.part_o + part_vec(ti.item0 + ti.part, w * QM + i, 0);
        T* dst = (T*)p.out + row * DV;
#pragma unroll 1
        for (int c = 0; c < DV / 32; ++c) {
          uint32_t o[32];
          tmem_ld32_wait(tmem + lrow + o_col + c * 32, o);
          if (!store) continue;
          if (!whole) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              part[(c * 8 + v) * BM] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                                   __uint_as_float(o[4 * v + 2]) * inv,
                                                   __uint_as_float(o[4 * v + 3]) * inv);
            continue;
          }
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            y[k] = pack2<T>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          if (p.out_32) {
#pragma unroll
            for (int v = 0; v < 2; ++v) st_global_32B(dst + c * 32 + v * 16, y + v * 8);
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              *reinterpret_cast<uint4*>(dst + c * 32 + v * 8) =
                  make_uint4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
          }
        }
        // (NaN scores: m may be -inf, l_run is NaN)
        const float lg = l_run == 0.f ? -INFINITY : m_run + (__log2f(l_run) - SHIFT);
        if (store && !whole) p.part_lse[prow] = lg;
        else if (store && p.lse) p.lse[row] = lg * LN2;
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty + e * 8);
    }
  }

  if ((warp == 1 || warp == 2) && rank == 0) {
    // every MMA this warp issued is complete before TMEM is released
    mma_commit_pair_warp(&bar_drain[warp - 1]);
    mbar_wait(&bar_drain[warp - 1], 0, 500000000ull);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // no CTA leaves while the pair's MMAs or barriers need it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, TMEM_COLS);
}

// Joins a tile's parts: a row's parts weighted by 2^(lse_s - max), in the order of
// the keys. The blocks of all its parts share the tile's groups of 8 rows; 8 threads
// read the 128 bytes of 8 rows.
constexpr int CROWS = 8, CY = 8;
template <typename T>
__global__ void __launch_bounds__(CROWS * DV / 4) latent_prefill_combine_kernel(PrefillP p) {
  pdl_wait();
  const int item = blockIdx.x;
  if (p.ctrl[2] == 1 || item >= p.ctrl[1]) return;
  const Tile ti = *reinterpret_cast<const Tile*>(p.rec + (size_t)item * 128);
  if (ti.parts == 1 || ti.part >= ti.parts) return;
  const int n = max(ti.n[0], ti.n[1]);
  const int c = threadIdx.x / CROWS;
  for (int g = blockIdx.y + CY * ti.part; g < ROWS / CROWS; g += CY * ti.parts) {
    const int r = g * CROWS + threadIdx.x % CROWS, w = r / QM;
    if (r % QM >= ti.nr[w]) continue;
    // parts that begin behind the query tile's last key have nothing for it
    int parts = ti.parts;
    while (part_begin(n, parts - 1, ti.parts) >= ti.n[w]) --parts;
    float m = -INFINITY;
    for (int s = 0; s < parts; ++s) m = fmaxf(m, p.part_lse[(ti.item0 + s) * ROWS + r]);
    if (m == -INFINITY) m = 0.f;   // all scores -inf: weights 0, a result of NaN, a log sum of -inf
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float f = exp2f(p.part_lse[(ti.item0 + s) * ROWS + r] - m);
      const float4 y = p.part_o[part_vec(ti.item0 + s, r, c)];
      total += f;
      o.x += f * y.x;
      o.y += f * y.y;
      o.z += f * y.z;
      o.w += f * y.w;
    }
    const float inv = 1.f / total;
    const int64_t row = (int64_t)(ti.row0[w] + r % QM) * p.H + ti.h[w];
    *reinterpret_cast<uint2*>((T*)p.out + row * DV + c * 4) =
        make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
    if (p.lse && c == 0) p.lse[row] = (m + log2f(total)) * LN2;
  }
}

template <typename T>
cudaError_t launch(const LatentPrefillArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};   // devices whose kernel attribute is set
  if (!(ready.load() >> a.dev.id & 1)) {
    const cudaError_t e =
        cudaFuncSetAttribute(latent_prefill_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << a.dev.id);
  }
  const CUtensorMapDataType dt =
      std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const Layout lay = layout(a.B);
  const int pairs = a.dev.num_sms / 2 < MAX_PAIRS ? a.dev.num_sms / 2 : MAX_PAIRS;
  // (a tile of fewer steps than the two add up to is never cut)
  const bool split = may_split(a.Tq, a.H) && a.Tk > (MIN_SAVED + MIN_STEPS - 1) * BN;
  PrefillP p;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.B = a.B;
  p.H = a.H;
  p.Tq = a.Tq;
  p.Tk = a.Tk;
  // (3 prompts of 20-300 tokens at 16 heads: 13.8 us, with the plan kernel 15.2)
  p.direct = a.B <= pairs && most_tiles(a.B, a.Tq, a.H) <= pairs;
  // a stride that no index uses (one head, one row) or 0 (one head for all) is not a
  // stride for the tensor map: such a dimension has one entry there
  p.kn_heads = a.H > 1 && a.kn_sh > 0;
  p.v_heads = a.H > 1 && a.v_sh > 0;
  p.scale_log2 = a.scale * LOG2E;
  p.out = a.out;
  p.out_32 = ((uintptr_t)a.out & 31) == 0;
  p.lse = a.lse;
  p.ctrl = (int32_t*)a.ws;
  p.order = (int32_t*)(a.ws + lay.order);
  p.first = (int32_t*)(a.ws + lay.first);
  p.rec = split ? a.ws + lay.rec : nullptr;
  p.part_lse = (float*)(a.ws + lay.lse);
  p.part_o = (float4*)(a.ws + lay.o);
  p.dev_status = a.dev.status;
  auto row_stride = [&](int64_t st) { return a.Tk > 1 ? st : (int64_t)NOPE; };
  CUtensorMap mq, mk, mv, mr;
  if (!make_map_boxed(&mq, a.q, dt, 2, NOPE + 64, a.H, a.Tq, 64, BM) ||
      !make_map_strided(&mk, a.kn, dt, NOPE, p.kn_heads ? a.H : 1, a.Tk, p.kn_heads ? a.kn_sh : NOPE,
                        row_stride(a.kn_st), BN / 2) ||
      !make_map_strided(&mv, a.v, dt, DV, p.v_heads ? a.H : 1, a.Tk, p.v_heads ? a.v_sh : DV, row_stride(a.v_st),
                        BN) ||
      !make_map_rows(&mr, a.kr, dt, 64, a.Tk, row_stride(a.kr_st), BN / 2))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (!p.direct) {
    KernelTimer timer("latent_prefill_plan", s);
    e = launch_after_trigger(latent_prefill_plan_kernel, dim3(1),
                             dim3(a.B < PLAN_THREADS ? (a.B + 31) / 32 * 32 : PLAN_THREADS), 0, s, a.cu_q, a.cu_k, a.B, a.Tq,
                             a.Tk, a.H, pairs, split ? 1 : 0, p.ctrl, p.order, p.first, a.dev.status);
  }
  if (e != cudaSuccess) return e;
  {
    KernelTimer timer("latent_prefill", s);
    e = launch_after_trigger(latent_prefill_kernel<T>, dim3(2 * pairs), dim3(NTHREADS), SMEM, s, mq, mk, mv, mr, p);
  }
  if (e != cudaSuccess || !split) return e;
  KernelTimer timer("latent_combine", s);
  return launch_after_trigger(latent_prefill_combine_kernel<T>, dim3(pairs, CY), dim3(CROWS * DV / 4), 0, s, p);
}

}  // namespace

size_t latent_prefill_workspace(int32_t B, int32_t, int32_t) { return layout(B).total; }

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t s) {
  return a.dtype == PKV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace pkv
