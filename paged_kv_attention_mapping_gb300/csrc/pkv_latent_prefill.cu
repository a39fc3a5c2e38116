// Expanded latent attention of chunks: head h of row i of a sequence, with
// query [qn, qr], attends keys [kn_j, r_j] (r shared by the heads) and values v_j:
//   s_j = scale (qn . kn_j + qr . r_j),  j <= kv_len - q_len + i,
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + ln(sum).
//
// Every head has its own keys, so the tensor cores get their work from the query
// rows: a work tile is 256 rows of one head, as two query tiles of 128 whose
// products alternate, so that one tile's softmax runs under the other's MMAs.
// Per 128 keys and query tile: S = Q K^T (M 128, N 128, K 128 + 64) and O += P V
// (M 128, N 128, K 128): 2560 tensor cycles for both tiles, the bound.
//
//   warp 0   TMA producer: Q of both tiles, then K_j (nope part and rotary part)
//            and V_j into a ring of three 32 KB slots (nope keys or values) and two
//            rotary units; V rows behind the sequence's end are zeroed
//   warp 1   TMEM owner and MMA issuer: per key tile j and query tile w,
//            O_w += P_w V_{j-1}, then S_w = Q_w K_j^T over the same TMEM columns as
//            P_w (MMAs run in issue order, so the product has read P_w by then)
//   warps 2-5, 6-9  softmax of query tile 0, 1, a thread per row; P goes back
//            over S in TMEM as the A operand of the next product. O is rescaled
//            only when a row's maximum grows by more than 2^8.
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
constexpr int ROWS = 2 * BM;     // rows of a work tile
constexpr int NTHREADS = 320;
constexpr uint32_t UNIT = 16384;            // 128 rows x 64 columns of 16 bits
constexpr uint32_t Q_BYTES = 3 * UNIT;      // one query tile
constexpr int NSLOT = 3;
constexpr uint32_t SLOT_BYTES = 2 * UNIT;
constexpr uint32_t SMEM = 2 * Q_BYTES + NSLOT * SLOT_BYTES + 2 * UNIT + 1024;
static_assert(SMEM <= 231424, "shared memory");
constexpr uint32_t TMEM_COLS = 512;         // S of both tiles, then O of both
constexpr float RESCALE_LOG2 = 8.f;
constexpr int PLAN_THREADS = 1024;

// Workspace: the next tile to claim, the number of tiles, then the sequences in
// the order they are worked on and the tiles before each.
struct Layout {
  size_t order, first, total;
};
Layout layout(int32_t B) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  Layout l;
  l.order = 256;
  l.first = l.order + al((size_t)B * 4);
  l.total = l.first + al(((size_t)B + 1) * 4);
  return l;
}

struct PrefillP {
  const int32_t *cu_q, *cu_k;
  int32_t B, H;
  int32_t kn_heads, v_heads;   // 0: every head reads head 0 (a head stride of 0)
  float scale_log2;            // > 0
  void* out;
  float* lse;
  int32_t *ctrl, *order, *first;
  int32_t* dev_status;
};

// One CTA: checks the lengths, orders the sequences by keys (descending, up to
// PLAN_THREADS of them; more stay in their own order) and counts their tiles.
__global__ void __launch_bounds__(PLAN_THREADS) latent_prefill_plan_kernel(const int32_t* __restrict__ cu_q,
                                                                          const int32_t* __restrict__ cu_k,
                                                                          int32_t B, int32_t Tq, int32_t Tk,
                                                                          int32_t H, int32_t* ctrl, int32_t* order,
                                                                          int32_t* first, int32_t* dev_status) {
  __shared__ int s_cost[PLAN_THREADS], s_rank[PLAN_THREADS], s_scan[32], s_carry;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool sorted = B <= PLAN_THREADS;
  bool bad = tid == 0 && (__ldg(cu_q) != 0 || __ldg(cu_k) != 0 || __ldg(cu_q + B) > Tq || __ldg(cu_k + B) > Tk);
  for (int b = tid; b < B; b += PLAN_THREADS)
    bad |= __ldg(cu_q + b + 1) < __ldg(cu_q + b) || __ldg(cu_k + b + 1) < __ldg(cu_k + b);
  bad = __syncthreads_or(bad);
  auto tiles_of = [&](int b, int* keys) {
    const int q = __ldg(cu_q + b + 1) - __ldg(cu_q + b), L = __ldg(cu_k + b + 1) - __ldg(cu_k + b);
    *keys = L;
    if (bad || q == 0) return 0;
    if (L < q) {
      atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
      return 0;
    }
    return (q + ROWS - 1) / ROWS;
  };
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
  pdl_wait();   // an earlier call may still be reading the workspace until here
  for (int base = 0; base < B; base += PLAN_THREADS) {
    __syncthreads();
    const int carry = s_carry;
    const int k = base + tid;
    int b = 0, keys, n = 0;
    if (k < B) {
      b = sorted ? s_rank[k] : k;
      n = tiles_of(b, &keys) * H;
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
    for (int w = 0; w < 32; ++w) {
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
    ctrl[0] = 0;
    ctrl[1] = s_carry;
    if (bad) atomicOr(dev_status, PKV_DEV_BAD_LENGTHS);
  }
}

// A work tile. Query tile w has rows row0 + 128 w .. (nr[w] of them, 0: none),
// its first at position pos[w], and reads n[w] key tiles.
struct Tile {
  int valid, h, k0, L, row0;
  int nr[2], pos[2], n[2];
};

template <typename T>
__global__ void __launch_bounds__(NTHREADS, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mr,
                          PrefillP p) {
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = sm;                                  // [query tile][3 units]
  unsigned char* sRing = sQ + 2 * Q_BYTES;                 // [slot][2 units]
  unsigned char* sRope = sRing + NSLOT * SLOT_BYTES;       // [2]

  __shared__ __align__(8) uint64_t bar_q, bar_qempty, bar_full[NSLOT], bar_empty[NSLOT], bar_sfull[2], bar_pfull[2],
      bar_odone[2], bar_tfull[2], bar_tempty[2], bar_vfix[2], bar_drain;
  __shared__ uint32_t s_tmem;
  __shared__ Tile s_tile[2];
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&bar_q, 1);
    mbar_init(&bar_qempty, 1);
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_sfull[w], 1);
      mbar_init(&bar_pfull[w], BM);
      mbar_init(&bar_odone[w], 1);
      mbar_init(&bar_tfull[w], 1);
      mbar_init(&bar_tempty[w], 1 + 8);   // the MMA warp and every softmax warp
      mbar_init(&bar_vfix[w], 1);
    }
    mbar_init(&bar_drain, 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mr);
  }
  if (warp == 1) tmem_alloc(&s_tmem, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();   // the plan, and whatever wrote the inputs

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait_or_abort(bar, parity, &s_abort, p.dev_status, p.dev_status);
  };
  const int n_tiles = *(volatile const int32_t*)&p.ctrl[1];
  bool ok = true;

  if (warp == 0) {
    // --------------------------------------------------------------- producer
    uint32_t ring = 0, ropes = 0;    // loads and steps before the current one
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      // entry e is free again once every consumer is done with tile t - 2
      if (t >= 2 && !(ok = wait(&bar_tempty[e], ((t >> 1) - 1) & 1))) break;
      if (lane == 0) {
        Tile ti{};
        const int tt = s_abort ? n_tiles : atomicAdd(&p.ctrl[0], 1);
        if (tt < n_tiles) {
          int lo = 0, hi = p.B - 1;   // the last sequence that starts at or before tile tt
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.first[mid] <= tt) lo = mid; else hi = mid - 1;
          }
          const int b = p.order[lo];
          const int q_lo = __ldg(p.cu_q + b), q = __ldg(p.cu_q + b + 1) - q_lo;
          ti.k0 = __ldg(p.cu_k + b);
          ti.L = __ldg(p.cu_k + b + 1) - ti.k0;
          const int per = (q + ROWS - 1) / ROWS, at = tt - p.first[lo];
          ti.h = at / per;
          const int q0 = (per - 1 - (at - ti.h * per)) * ROWS;
          ti.row0 = q_lo + q0;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            ti.nr[w] = max(0, min(BM, q - q0 - w * BM));
            ti.pos[w] = ti.L - q + q0 + w * BM;
            ti.n[w] = ti.nr[w] ? (ti.pos[w] + ti.nr[w] + BN - 1) / BN : 0;
          }
          ti.valid = 1;
        }
        s_tile[e] = ti;
        mbar_arrive(&bar_tfull[e]);
      }
      __syncwarp();
      const Tile ti = s_tile[e];
      if (!ti.valid) break;
      const int W = ti.nr[1] ? 2 : 1, n = max(ti.n[0], ti.n[1]);
      // Q of this tile replaces the one before once its last S is done
      if (t >= 1 && !(ok = wait(&bar_qempty, (t - 1) & 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar_q, W * Q_BYTES);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (w < W) tma_load_3d(sQ + w * Q_BYTES + c * UNIT, &mq, &bar_q, c * 64, ti.h, ti.row0 + w * BM);
      }
      __syncwarp();
      for (int j = 0; j < n && ok; ++j, ++ropes) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++ring) {
          const uint32_t slot = ring % NSLOT, round = ring / NSLOT;
          if (!(ok = wait(&bar_empty[slot], (round & 1) ^ 1))) break;
          unsigned char* dst = sRing + slot * SLOT_BYTES;
          const int row = ti.k0 + j * BN;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar_full[slot], (kv ? 2 : 3) * UNIT);
            const int h = ti.h * (kv ? p.v_heads : p.kn_heads);
            tma_load_3d(dst, kv ? &mv : &mk, &bar_full[slot], 0, h, row);
            tma_load_3d(dst + UNIT, kv ? &mv : &mk, &bar_full[slot], 64, h, row);
            // the rotary unit of two steps ago: its S is done, or the slot would not be free
            if (!kv) tma_load_2d(sRope + (ropes & 1) * UNIT, &mr, &bar_full[slot], 0, row);
          }
          __syncwarp();
          if (kv && j == n - 1) {
            // 0 * NaN must not reach O from the rows behind the sequence's end
            const int end = ti.L - j * BN;
            if (end < BN) {
              if (!(ok = wait(&bar_full[slot], round & 1))) break;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint4* base = (uint4*)(dst + c * UNIT);
                for (int x = end * 8 + lane; x < BN * 8; x += 32) base[x] = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(&bar_vfix[e]);
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // let every copy this warp issued land before the CTA may exit
      const uint64_t t0 = globaltimer_ns();
      for (int it = 0; it < (1 << 24) && globaltimer_ns() - t0 < 20000000ull; ++it) {}
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    // The tensor pipe holds a few MMAs ahead of the issue and a wait costs on the
    // order of 100 cycles, so the waits for the next operands sit behind MMAs
    // already queued.
    const uint32_t id_s = idesc_f16(BM, BN, BF16, false);
    const uint32_t id_o = idesc_f16(BM, DV, BF16, true);
    const uint64_t qd = smem_desc(smem_u32(sQ), 16, 1024, LAYOUT_SW128);
    const uint64_t kd = smem_desc(smem_u32(sRing), 16, 1024, LAYOUT_SW128);
    const uint64_t rd = smem_desc(smem_u32(sRope), 16, 1024, LAYOUT_SW128);
    const uint64_t vd = smem_desc(smem_u32(sRing), UNIT, 1024, LAYOUT_SW128);
    uint32_t ring = 0, ropes = 0, p_use[2] = {0, 0};
    auto issue_s = [&](int w, uint32_t slot, uint32_t rope) {
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        const uint32_t off = (k >> 2) * UNIT + (k & 3) * 32;
        mma_f16_ss_warp(tmem + w * 128, qd + (uint64_t)((w * Q_BYTES + off) >> 4),
                        k < 8 ? kd + (uint64_t)((slot * SLOT_BYTES + off) >> 4)
                              : rd + (uint64_t)((rope * UNIT + (k & 3) * 32) >> 4),
                        id_s, k ? 1u : 0u);
      }
      mma_commit_warp(&bar_sfull[w]);
    };
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      if (!(ok = wait(&bar_tfull[e], (t >> 1) & 1))) break;
      const Tile ti = s_tile[e];
      if (!ti.valid) break;
      const int W = ti.nr[1] ? 2 : 1, n = max(ti.n[0], ti.n[1]);
      // K_j is the tile's load 2j, V_j load 2j + 1
      uint32_t ks = ring % NSLOT, kph = (ring / NSLOT) & 1;
      uint32_t vs = (ring + 1) % NSLOT, vph = ((ring + 1) / NSLOT) & 1;
      ring += 2 * n;
      auto advance = [](uint32_t& s, uint32_t& ph) {
        s += 2;
        if (s >= (uint32_t)NSLOT) {
          s -= NSLOT;
          ph ^= 1;
        }
      };
      if (!(ok = wait(&bar_q, t & 1))) break;
      if (!(ok = wait(&bar_full[ks], kph))) break;
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (w < W) issue_s(w, ks, ropes & 1);
      mma_commit_warp(&bar_empty[ks]);
      if (n == 1) mma_commit_warp(&bar_qempty);
      advance(ks, kph);
      if (!(ok = wait(&bar_full[vs], vph))) break;
      // step j: O_w (+)= P_w V_{j-1}, then S_w = Q_w K_j^T. The first product of a
      // tile overwrites O_w: its P comes after the softmax threads read the
      // tile before out of TMEM.
      for (int j = 1; j <= n; ++j) {
        if (j == n && !(ok = wait(&bar_vfix[e], (t >> 1) & 1))) break;
        const uint64_t v = vd + (uint64_t)((vs * SLOT_BYTES) >> 4);
        bool have_k = false;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w >= W) break;
          if (j - 1 < ti.n[w]) {
            if (!(ok = wait(&bar_pfull[w], p_use[w] & 1))) break;
            ++p_use[w];
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_f16_ta_warp(tmem + 256 + w * 128, tmem + w * 128 + k * 8, v + (uint64_t)((k * 2048) >> 4), id_o,
                              (j > 1 || k > 0) ? 1u : 0u);
            if (j == ti.n[w]) mma_commit_warp(&bar_odone[w]);
          }
          if (w == W - 1) {   // V_{j-1} has no reader left
            mma_commit_warp(&bar_empty[vs]);
            advance(vs, vph);
          }
          if (j < ti.n[w]) {
            if (!have_k && !(ok = wait(&bar_full[ks], kph))) break;
            have_k = true;
            if (w == W - 1 && !(ok = wait(&bar_full[vs], vph))) break;
            issue_s(w, ks, (ropes + j) & 1);
          }
        }
        if (!ok) break;
        if (j < n) {
          mma_commit_warp(&bar_empty[ks]);
          if (j == n - 1) mma_commit_warp(&bar_qempty);
          advance(ks, kph);
        }
      }
      ropes += n;
      if (ok && lane == 0) mbar_arrive(&bar_tempty[e]);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int w = (warp - 2) >> 2;                // query tile
    const int quarter = warp & 3;                 // TMEM lanes of this warp
    const int i = quarter * 32 + lane;            // row of the query tile
    const uint32_t lrow = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = w * 128, o_col = 256 + w * 128;
    const float sc = p.scale_log2;
    uint32_t n_s = 0, n_o = 0;                    // S and O hand-offs taken
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      if (!(ok = wait(&bar_tfull[e], (t >> 1) & 1))) break;
      const Tile& ti = s_tile[e];
      if (!ti.valid) break;
      const int n = ti.n[w];
      if (n > 0) {
        const int pos = min(ti.pos[w] + i, ti.L - 1);
        const int j_mask = (ti.pos[w] + 1) / BN;   // key tiles before have no hidden key
        float m_run = -INFINITY, l_run = 0.f;
        for (int j = 0; j < n; ++j) {
          // S complete also means that the product that read P is
          if (!(ok = wait(&bar_sfull[w], n_s & 1))) break;
          ++n_s;
          tc_fence_after();
          uint32_t r[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lrow + s_col + c * 32, r[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_fence(r[c]);
          if (j >= j_mask) {
            const int lim = pos - j * BN;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (c * 32 + k > lim) r[c][k] = __float_as_uint(-INFINITY);
          }
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              mx[(k >> 1) & 7] = max3(mx[(k >> 1) & 7], __uint_as_float(r[c][k]), __uint_as_float(r[c][k + 1]));
          const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
          const bool first = j == 0;
          const bool grow = first || mt > m_run + RESCALE_LOG2;
          const float m_new = grow ? fmaxf(mt, m_run) : m_run;
          if (!first && __any_sync(0xffffffffu, grow)) {
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
          const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m_run, -m_run);
          float2 ls[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t pw[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int k0 = hf * 64 + 2 * k;
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(r[k0 >> 5][k0 & 31]), __uint_as_float(r[k0 >> 5][(k0 & 31) + 1])), sc2,
                  nm2);
              const float a = ex2(x.x), b = ex2(x.y);
              ls[k & 3] = __fadd2_rn(ls[k & 3], make_float2(a, b));
              pw[k] = pack2<T>(a, b);
            }
            tmem_st32(tmem + lrow + s_col + hf * 32, pw);
            tmem_wait_st();
            reg_fence(pw);
          }
          l_run += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
          tc_fence_before();
          mbar_arrive(&bar_pfull[w]);
        }
        if (!ok) break;
        if (!(ok = wait(&bar_odone[w], n_o & 1))) break;
        ++n_o;
        tc_fence_after();
        const bool store = i < ti.nr[w];
        const float inv = 1.f / l_run;
        const int64_t row = (int64_t)(ti.row0 + w * BM + i) * p.H + ti.h;
        T* dst = (T*)p.out + row * DV;
#pragma unroll 1
        for (int c = 0; c < DV / 32; ++c) {
          uint32_t o[32];
          tmem_ld32_wait(tmem + lrow + o_col + c * 32, o);
          if (!store) continue;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = pack2<T>(__uint_as_float(o[v * 8 + 2 * k]) * inv, __uint_as_float(o[v * 8 + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + c * 32 + v * 8) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        if (store && p.lse) p.lse[row] = (m_run + __log2f(l_run)) * LN2;
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_tempty[e]);
    }
  }

  if (warp == 1) {
    // every MMA this warp issued is complete before TMEM is released
    mma_commit_warp(&bar_drain);
    mbar_wait(&bar_drain, 0, 500000000ull);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
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
  PrefillP p;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.B = a.B;
  p.H = a.H;
  // a stride that no index uses (one head, one row) or 0 (one head for all) is not a
  // stride for the tensor map: such a dimension has one entry there
  p.kn_heads = a.H > 1 && a.kn_sh > 0;
  p.v_heads = a.H > 1 && a.v_sh > 0;
  p.scale_log2 = a.scale * LOG2E;
  p.out = a.out;
  p.lse = a.lse;
  p.ctrl = (int32_t*)a.ws;
  p.order = (int32_t*)(a.ws + lay.order);
  p.first = (int32_t*)(a.ws + lay.first);
  p.dev_status = a.dev.status;
  auto row_stride = [&](int64_t st) { return a.Tk > 1 ? st : (int64_t)NOPE; };
  CUtensorMap mq, mk, mv, mr;
  if (!make_map_boxed(&mq, a.q, dt, 2, NOPE + 64, a.H, a.Tq, 64, BM) ||
      !make_map_strided(&mk, a.kn, dt, NOPE, p.kn_heads ? a.H : 1, a.Tk, p.kn_heads ? a.kn_sh : NOPE,
                        row_stride(a.kn_st), BN) ||
      !make_map_strided(&mv, a.v, dt, DV, p.v_heads ? a.H : 1, a.Tk, p.v_heads ? a.v_sh : DV, row_stride(a.v_st),
                        BN) ||
      !make_map_rows(&mr, a.kr, dt, 64, a.Tk, row_stride(a.kr_st), BN))
    return cudaErrorInvalidValue;
  cudaError_t e;
  {
    KernelTimer timer("latent_prefill_plan", s);
    e = launch_after_trigger(latent_prefill_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, s, a.cu_q, a.cu_k, a.B, a.Tq,
                             a.Tk, a.H, p.ctrl, p.order, p.first, a.dev.status);
  }
  if (e != cudaSuccess) return e;
  KernelTimer timer("latent_prefill", s);
  return launch_after_trigger(latent_prefill_kernel<T>, dim3(a.dev.num_sms), dim3(NTHREADS), SMEM, s, mq, mk, mv, mr,
                              p);
}

}  // namespace

size_t latent_prefill_workspace(int32_t B, int32_t, int32_t) { return layout(B).total; }

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t s) {
  return a.dtype == PKV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace pkv
