// Window attention for chunks of rows, on the tensor cores (tcgen05, TMEM).
//
// A query tile is 128 rows of the MMA: PP consecutive positions of one sequence times the
// G query heads of one KV head (PP = 128 / G), so that a tile's positions, and with them the
// keys that some row sees beside each row's own window, are few: window + PP - 1 keys and
// the sinks, against window + 127 for a tile of one head. A work tile is two query tiles
// (2 PP positions) over the keys that either sees; they share each key and value tile.
//
//   warp 0      producer: finds the work tiles, loads Q, then K_j and V_j of each step (128
//               keys) into a ring of shared-memory slots by TMA
//   warp 1      TMEM owner and MMA issuer: O_w += P_w V_{j-1} (P_w read from TMEM), S_w =
//               Q_w K_j^T into the same columns; the pipe runs in issue order
//   warps 2-5   softmax of query tile 0, one thread a row; warps 6-9 of query tile 1
//   warp 10     zeroes the rows of a value tile that no row of the work tile sees (the keys
//               before the first window and after the last row): 0 * NaN must not reach O.
//               Over an e4m3 cache warps 10 and 11 instead widen every key and value tile to
//               f16 in its slot, with those rows as zeros.
// Steps are 128 keys each: from key 0 on while there are sinks, then from the first window's first
// key (rounded down to 32) to the last row's. Each step has a range of 32-key pieces that a query tile
// sees at all; loads, products and the softmax take that range only, and a query tile without
// one skips the step.
// The softmax keeps a running maximum and sum; O is rescaled in TMEM only when a row's
// maximum grows by more than 2^8. A row can start with pieces that it does not see: its
// maximum is then -inf, and its weights 0.
// What bounds it: the one warp that issues all products, in order. Cycles of a step of both query tiles, by time stamps
// in it and in a softmax warp of each (which cost 14 %):
//   16384 tokens, window 2048: 3970, of which the products are 2048. The MMA warp waits 790 for weights (460 for the
//     first half, 330 for the second; nothing of the other query tile's is issued meanwhile) and 280 for K and V; the
//     other 850 are its issue and hand-offs, and the stamps. A softmax warp has a step's weights 1310 after its scores
//     and then waits 1810 for the next ones, so its own work is not the bound (without it the calls take 12 % less).
//   seven prompts at window 512: 5040, of which 1480 are waits for weights; a work tile is four steps (20990 of
//     its 22830 cycles), its first scores and last output with nothing beside them, its output's store 2090.
//   16384 tokens, window 128: two steps of 6530 a work tile, 2320 of each waits for weights.
// 16384 tokens, 32 / 8 heads of 128, no sinks: window 2048 436 us, 1182 TFLOP/s (62 % of the measured burst
// rate); 512 174 us; 128 104 us; with 64 sinks at 2048 455; over e4m3 with bf16 queries 659, 339 and 250. Seven
// prompts of 300 to 2500 tokens at window 512, 28 / 4 heads: 95 us.
// Steps taken (16384 tokens at window 2048): ranges in place of whole tiles at the ends, whole steps with their
// scores in registers and others read twice (610 -> 497 us), ranges as words for the MMA warp, which is short of
// issue slots (465), weights handed over in halves and 32-byte stores (456; with work tiles numbered without
// gaps, a bad page's flag a query tile's own: 452, 456).
// Without gain: two threads a row (526; the exponentials share a unit), an MMA warp for each query
// tile (479), both forms of a step over registers (2261, spills), masked steps over registers (498) or two
// pieces at a time (509), partial steps as a function (702), boxes of 128 rows, a ring of four slots,
// looking the next tile up early.
// Every mbarrier wait is bounded (PKV_DEV_TIMEOUT); TMEM accesses are warp-uniform.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pkv_sm100.cuh"
#include "pkv_window_common.cuh"

namespace pkv {
using namespace sm100;
using namespace window;

namespace {

constexpr int BM = 128, BN = 128;
constexpr int NQ = 2;                    // query tiles of a work tile
constexpr int PIECE = 32;                // keys of a piece
constexpr int SOFTMAX_WARPS = 4 * NQ;
constexpr int HELPER = 2 + SOFTMAX_WARPS;   // first helper warp
constexpr uint32_t TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.f;
// f16 weights carry this power of two, so that small ones are not lost to f16's smallest
// exponents; a weight is at most 2^8 (above), 2^15 with it
constexpr float F16_SHIFT = 7.f;

struct TilesP {
  const int32_t *cu, *kv_lens, *tables;
  int32_t B, T, Hq, Hkv, G, PP, P, num_pages, max_pages, window, sinks, min_q;
  int32_t box, wide, beside;   // rows of a page block; out is 32-byte aligned; a row kernel follows in this call
  PageDiv div;
  float scale_log2;
  const float *ks, *vs;
  void* out;
  float* lse;
  int32_t* dev_status;
};

struct Tile {
  int valid, b, kvh, row0, np, p_first;
  int lo, sinks;          // keys of the work tile: [0, sinks) and [lo, p_first + np)
  int js, ws, steps;      // steps 0 .. js - 1 begin at key 128 step, later ones at ws + 128 (step - js)
  int bad;                // a bit a query tile: one of its pages is outside the pool
};

// Rows [0, a) and [b, e) of a key tile are seen, in the pieces [c0, c1); c0 == c1: none is.
struct Range {
  int a, b, e, c0, c1;
};
__device__ __forceinline__ Range range_of(int k0, int sinks, int lo, int end) {
  Range r;
  r.a = min(max(sinks - k0, 0), BN);
  r.b = min(max(lo - k0, 0), BN);
  r.e = min(max(end - k0, 0), BN);
  if (r.e <= r.b) r.b = r.e = r.a;   // nothing of the window here
  const int first = r.a > 0 ? 0 : r.b, last = max(r.a, r.e);
  r.c0 = first / PIECE;
  r.c1 = last > first ? (last + PIECE - 1) / PIECE : r.c0;
  return r;
}
__device__ __forceinline__ int step_key(const Tile& t, int i) { return i < t.js ? i * BN : t.ws + (i - t.js) * BN; }
__device__ __forceinline__ Range union_range(const Tile& t, int k0) {
  return range_of(k0, t.sinks, t.lo, t.p_first + t.np);
}
// What query tile w sees.
__device__ __forceinline__ Range tile_range(const Tile& t, int w, int PP, int window, int sinks, int k0) {
  const int pa = t.p_first + w * PP, pe = t.p_first + min((w + 1) * PP, t.np);
  const int lo = max(0, pa - window + 1);
  return range_of(k0, min(sinks, lo), lo, pe);
}
// What the MMA warp has to know of a step, a word that the producer works out (a warp that issues
// products back to back has no time for it): for query tile w, in byte w, the first piece and (3 bits on) the
// number of pieces it sees, and (bit 7) whether this is its last step.
constexpr uint32_t WHOLE_STEP = (uint32_t)(BN / PIECE) << 3;   // of one query tile
__device__ __forceinline__ uint32_t step_word(const Tile& t, int nq, int PP, int window, int sinks, int k0) {
  uint32_t word = 0;
  for (int w = 0; w < nq; ++w) {
    const Range r = tile_range(t, w, PP, window, sinks, k0);
    const int last_key = t.p_first + min((w + 1) * PP, t.np) - 1;
    const uint32_t last = last_key >= k0 && last_key < k0 + BN;
    word |= ((uint32_t)r.c0 | (uint32_t)(r.c1 - r.c0) << 3 | last << 7) << (8 * w);
  }
  return word;
}

// Rows of the pieces that no row of the work tile sees.
__device__ __forceinline__ bool has_gaps(const Range& r) { return r.b > r.a || r.e < r.c1 * PIECE; }

// What the widening warps need of one load (e4m3 caches).
struct LoadDesc {
  Range r;
  int zero, q_first, q_par, entry, nq, stop;
};

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int NS = D == 128 ? 5 : 8;
  static constexpr uint32_t Q_BYTES = BM * D * 2;
  static constexpr uint32_t SLOT = BN * D * 2;
  static constexpr uint32_t SMEM = NQ * Q_BYTES + NS * SLOT + 1024;
  static_assert(SMEM <= 232448 - 2048, "shared memory");
};

__device__ __forceinline__ void mma_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]));
}

// 16 values of an output row: one 32-byte store where out is aligned to it (half the store
// instructions, whole sectors), else two.
template <typename T>
__device__ __forceinline__ void store16(T* dst, const uint32_t (&x)[8], int wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// max(a, b, c) in one instruction; a NaN is passed over, as by fmaxf.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// e4m3 tiles: codes lie in the upper half of the slot, 128 a row, 128-byte swizzled; the
// f16 tile is what a 16-bit load would have made of it (two 64-column halves). A lane reads a
// row's codes before it writes the row, and row r's codes are overwritten by row r alone.
__device__ __forceinline__ void widen_rows(unsigned char* slot, const LoadDesc& d, int warp, int lane) {
  const unsigned char* stg = slot + BN * 128;
  for (int r = d.r.c0 * PIECE + warp * 32 + lane; r < d.r.c1 * PIECE; r += 64) {
    const int sw = r & 7;
    uint4 c[8];
    if (d.zero && !(r < d.r.a || (r >= d.r.b && r < d.r.e))) {
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = *reinterpret_cast<const uint4*>(stg + r * 128 + ((k ^ sw) << 4));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
      uint32_t h[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[2 * q] = widen(w[q]);
        h[2 * q + 1] = widen(w[q] >> 16);
      }
      unsigned char* row = slot + (k >> 2) * BN * 128 + r * 128;
      const int ch = (k & 3) * 2;
      *reinterpret_cast<uint4*>(row + ((ch ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(row + (((ch + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
}

// bf16 queries over an e4m3 cache: f16 in place, each row times the power of two that brings its
// largest value to 2^8 .. 2^9 (bf16 has exponents that f16 lacks); its inverse's exponent goes to `back`.
__device__ __forceinline__ void narrow_q(unsigned char* q, uint8_t* back, int lane) {
  for (int r = lane; r < BM; r += 32) {
    float top = 0.f;
    for (int c = 0; c < 16; ++c) {
      const uint4 x = *reinterpret_cast<const uint4*>(q + (c >> 3) * BM * 128 + r * 128 + ((c & 7) << 4));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
    }
    const int eb = (int)(__float_as_uint(top) >> 23);
    const int fe = eb == 0 || eb == 255 ? 127 : min(max(262 - eb, 2), 252);
    const float f = __uint_as_float((uint32_t)fe << 23);
    back[r] = (uint8_t)(254 - fe);
    for (int c = 0; c < 16; ++c) {
      uint4* at = reinterpret_cast<uint4*>(q + (c >> 3) * BM * 128 + r * 128 + ((c & 7) << 4));
      uint4 x = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack2<__half>(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
      *at = x;
    }
  }
}

// What a row sees of a step: the columns <= hi that are > lo or < se.
struct RowStep {
  int hi, lo, se;
};

// Which of a piece's 32 columns are seen: a few shifts a piece, then a select a column.
__device__ __forceinline__ uint32_t seen_bits(const RowStep& st, int c) {
  const int h = st.hi - c * PIECE, l = st.lo - c * PIECE, s = st.se - c * PIECE;
  const uint32_t mh = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
  const uint32_t ml = l < 0 ? ~0u : l >= 31 ? 0u : ~((2u << l) - 1u);
  const uint32_t ms = s <= 0 ? 0u : s >= 32 ? ~0u : (1u << s) - 1u;
  return mh & (ml | ms);
}
__device__ __forceinline__ void hide(uint32_t (&r)[PIECE], uint32_t seen) {
#pragma unroll
  for (int x = 0; x < PIECE; ++x)
    if (!(seen >> x & 1)) r[x] = __float_as_uint(-INFINITY);
}
__device__ __forceinline__ void max_of(const uint32_t (&r)[PIECE], float (&mx)[8]) {
#pragma unroll
  for (int x = 0; x < PIECE; x += 2)
    mx[(x >> 1) & 7] = max3(mx[(x >> 1) & 7], __uint_as_float(r[x]), __uint_as_float(r[x + 1]));
}

// The running maximum after a step (log2 units); O and the sum follow it where it grows by more
// than 2^8.
template <int D>
__device__ __forceinline__ void new_maximum(float mt, uint32_t to, bool first, float& m_run, float& l_run) {
  const bool grow = mt > m_run + RESCALE_LOG2;   // (from -inf: any maximum but -inf)
  const float m_new = grow ? mt : m_run;
  if (!first && __any_sync(0xffffffffu, grow)) {
    const float alpha = grow ? ex2(m_run - m_new) : 1.f;
    l_run *= alpha;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {   // (16 columns at a time: a whole step's scores stay in registers)
      uint32_t o[16];
      tmem_ld16(to + c * 16, o);
      tmem_wait_ld();
      reg_fence16(o);
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
      tmem_st16(to + c * 16, o);
    }
    tmem_wait_st();
  }
  m_run = m_new;
}

// Weights of a piece, their sums by pairs of columns, and where they go (16-bit pairs: the layout
// of an A operand).
template <typename MT>
__device__ __forceinline__ void weigh(const uint32_t (&r)[PIECE], float sc, float nm, float2 (&ls)[4], uint32_t to) {
  const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nm, nm);
  uint32_t pw[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), sc2, nm2);
    const float a = ex2(y.x), b = ex2(y.y);
    ls[x & 3] = __fadd2_rn(ls[x & 3], make_float2(a, b));
    pw[x] = pack2<MT>(a, b);
  }
  tmem_st16(to, pw);
}

// TQ: type of q and out. KV8: e4m3 caches (head_dim 128), products in f16.
template <int D, typename TQ, bool KV8>
__global__ void __launch_bounds__((HELPER + (KV8 ? 2 : 1)) * 32, 1)
    window_tiles_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, const __grid_constant__ TilesP p) {
  using C = Cfg<D>;
  using MT = typename std::conditional<KV8, __half, TQ>::type;
  constexpr bool BF16 = std::is_same<MT, __nv_bfloat16>::value;
  constexpr bool QCONV = KV8 && std::is_same<TQ, __nv_bfloat16>::value;
  constexpr float SHIFT = BF16 ? 0.f : F16_SHIFT;
  constexpr int NS = C::NS;
  static_assert(!KV8 || D == 128, "e4m3 tiles are one 128-code row wide");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = sm;
  unsigned char* sRing = sQ + NQ * C::Q_BYTES;

  // Work tiles pass through two entries (tile t in entry t & 1): the producer fills the next
  // one and loads its Q while tile t finishes.
  __shared__ __align__(8) uint64_t bar_q, bar_qempty, bar_full[NS], bar_empty[NS], bar_sfull[NQ],
      bar_pfull[NQ][2], bar_odone[NQ], bar_tfull[2], bar_tempty[2], bar_drain;
  // loads that a helper warp works on before the MMA may read them land here: the value tiles
  // with rows to zero; over an e4m3 cache every tile, and bf16 queries
  __shared__ __align__(8) uint64_t bar_land[NS], bar_qland;
  __shared__ LoadDesc s_ld[KV8 ? NS : 1];
  __shared__ uint8_t s_back[2][QCONV ? NQ * BM : 1];   // (by entry: a slow softmax may still read the last tile's)
  __shared__ Tile s_tile[2];
  __shared__ uint32_t s_step[8];
  __shared__ uint32_t s_tmem;
  __shared__ int32_t s_err;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // The row kernel of the same call may start beside this one. Nothing else: CTAs of the next call that
  // get their SMs one by one as this one's end lose the order in which neighbours share keys in L2
  // (calls of 7 prompts back to back: 126 us each with the trigger, 96 without).
  if (p.beside) pdl_trigger();
  if (blockIdx.x == 0) check_cu(p.cu, p.B, p.T, p.dev_status);
  if (tid == 0) {
    mbar_init(&bar_q, QCONV ? 2 : 1);
    // free for the next Q: its products are done and, with QCONV, every softmax warp has seen this one's phase of
    // bar_q (only then may the next phase complete: a warp that came late would wait for one that is over)
    mbar_init(&bar_qempty, QCONV ? 1 + SOFTMAX_WARPS : 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bar_full[s], KV8 ? 2 : 1);
      mbar_init(&bar_empty[s], 1);
      mbar_init(&bar_land[s], 1);
    }
    mbar_init(&bar_qland, 1);
    for (int w = 0; w < NQ; ++w) {
      mbar_init(&bar_sfull[w], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&bar_pfull[w][h], SOFTMAX_WARPS / NQ);
      mbar_init(&bar_odone[w], 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(&bar_tfull[e], 1);
      mbar_init(&bar_tempty[e], 1 + SOFTMAX_WARPS + (KV8 ? 0 : 1));   // MMA, softmax and zeroing warps
    }
    mbar_init(&bar_drain, 1);
    fence_mbar_init();
    s_abort = 0;
    s_err = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == 1) tmem_alloc(&s_tmem, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait_or_abort(bar, parity, &s_abort, &s_err, p.dev_status);
  };

  if (warp == 0) {
    // --------------------------------------------------------------- producer
    // a bit a slot: parity of its loads, of those that land for a helper, and whether the last did
    uint32_t ring = 0, loads = 0, landing = 0, last_land = 0, used = 0, q_loads = 0;
    bool ok = true;
    // Work tiles are numbered without gaps, sequence by sequence, so that the CTAs' shares differ by one tile at
    // most: with the row kernel's numbers, which need no counting, 16 sequences of 32 rows (window 4096, 32 / 8
    // heads of 128) took 105 us for 60, 12 of 50 rows 130 for 73, 16 of 64 (window 512; no gaps) 24.9 for 25.4.
    // Lane l counts the tiles of `share` sequences and keeps the number behind them. (A cu_seqlens_q that breaks
    // its rules may count more than `most`, which its rows could make; counts stop there, so that 32 bits hold
    // them, and no more are worked on.)
    const int per = NQ * p.PP, share = (p.B + 31) / 32;
    const uint32_t most = (uint32_t)p.B + (uint32_t)(p.T / per);
    auto count = [&](int b, int& c0, int& c1) {
      c0 = __ldg(p.cu + b);
      c1 = __ldg(p.cu + b + 1);
      return c0 >= 0 && c1 > c0 && c1 <= p.T && c1 - c0 >= p.min_q ? (uint32_t)((c1 - c0 - 1) / per + 1) : 0u;
    };
    auto running = [&](uint32_t n) {   // sum over the lanes up to this one
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n = min(n + x, most);
      }
      return n;
    };
    uint32_t behind = 0;
    for (int i = 0; i < share; ++i) {
      int c0, c1;
      if (lane * share + i < p.B) behind = min(behind + count(lane * share + i, c0, c1), most);
    }
    behind = running(behind);
    const uint32_t units = __shfl_sync(0xffffffffu, behind, 31) * (uint32_t)p.Hkv;
    uint32_t u = blockIdx.x;
    for (uint32_t t = 0; ok; ++t) {
      // the next work tile of this CTA
      Tile ti;
      ti.valid = 0;
      ti.bad = 0;
      for (; u < units && !ti.valid; u += gridDim.x) {
        const uint32_t k = u / (uint32_t)p.Hkv;
        ti.kvh = (int)(u - k * (uint32_t)p.Hkv);
        const int l = __ffs(__ballot_sync(0xffffffffu, behind > k)) - 1;   // the lane that counted it
        const uint32_t before = __shfl_sync(0xffffffffu, behind, max(l - 1, 0));
        uint32_t rest = k - (l > 0 ? before : 0u);
        int b = -1, c0 = 0, c1 = 0, q0 = 0;
        if (share == 1) {   // (the lane counted one sequence: this one)
          b = l;
          c0 = __ldg(p.cu + b);
          c1 = __ldg(p.cu + b + 1);
          q0 = (int)rest * per;
        } else {
          const int end = min((l + 1) * share, p.B);
          for (int s0 = l * share; s0 < end; s0 += 32) {
            int m0 = 0, m1 = 0;
            const uint32_t tiles = s0 + lane < end ? count(s0 + lane, m0, m1) : 0u, to = running(tiles);
            const unsigned found = __ballot_sync(0xffffffffu, to > rest);
            if (found) {
              const int j = __ffs(found) - 1;
              b = s0 + j;
              c0 = __shfl_sync(0xffffffffu, m0, j);
              c1 = __shfl_sync(0xffffffffu, m1, j);
              const uint32_t left = __shfl_sync(0xffffffffu, to, max(j - 1, 0));
              q0 = (int)(rest - (j > 0 ? left : 0u)) * per;
              break;
            }
            rest -= __shfl_sync(0xffffffffu, to, 31);
          }
        }
        if (b < 0) continue;
        const int n = c1 - c0, L = __ldg(p.kv_lens + b);
        if (L < n || L > (int64_t)p.max_pages * p.P) {
          if (q0 == 0 && ti.kvh == 0 && lane == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
          continue;
        }
        ti.b = b;
        ti.row0 = c0 + q0;
        ti.np = min(per, n - q0);
        ti.p_first = L - n + q0;
        const int p_last = ti.p_first + ti.np - 1;
        ti.lo = max(0, ti.p_first - p.window + 1);
        ti.sinks = min(p.sinks, ti.lo);
        ti.js = (ti.sinks + BN - 1) / BN;
        ti.ws = max(ti.js * BN, ti.lo / PIECE * PIECE);
        ti.steps = ti.js + (p_last >= ti.ws ? (p_last - ti.ws) / BN + 1 : 0);
        ti.valid = 1;
      }
      const uint32_t e = t & 1;
      // entry e is free again once every consumer is done with tile t - 2
      if (t >= 2 && !wait(&bar_tempty[e], ((t >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        s_tile[e] = ti;
        mbar_arrive(&bar_tfull[e]);   // releases the entry's fields to its waiters
      }
      __syncwarp();
      if (!ti.valid) break;
      const int nq = ti.np > p.PP ? 2 : 1;
      if (t >= 1 && !wait(&bar_qempty, (t - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        uint64_t* bar = QCONV ? &bar_qland : &bar_q;
        mbar_arrive_expect_tx(bar, nq * C::HALVES * (uint32_t)(p.G * p.PP * 128));
        for (int w = 0; w < nq; ++w)
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(sQ + w * C::Q_BYTES + h * BM * 128, &mq, bar, h * 64, ti.kvh * p.G, ti.row0 + w * p.PP);
      }
      ++q_loads;
      const int32_t* pt = p.tables + (int64_t)ti.b * p.max_pages;
      for (int i = 0; i < ti.steps && ok; ++i) {
        const int k0 = step_key(ti, i);
        const Range r = union_range(ti, k0);
        // lane (block, half): box rows of one page, 64 channels (e4m3: all 128); the rows of
        // blocks without a key that is seen are left as they are
        constexpr int LH = KV8 ? 1 : C::HALVES;
        const int row = (lane / LH) * p.box, half = lane % LH;
        const bool in = row < r.c1 * PIECE && row + p.box > r.c0 * PIECE && row < BN &&
                        (row < r.a || (row < r.e && row + p.box > r.b));
        int at = 0;
        bool bad = false;
        if (in) {
          const int pg = page_of(k0 + row, p.div);
          const int id = __ldg(pt + pg);
          bad = id < 0 || id >= p.num_pages;
          at = id * p.P + (k0 + row - pg * p.P);
        }
        const bool load = in && !bad;
        const uint32_t word = step_word(ti, nq, p.PP, p.window, p.sinks, k0);
        if (__any_sync(0xffffffffu, bad)) {
          // the query tiles with a block of the bad page among this step's operands (nothing is loaded there). A tile
          // reads its own bit after its last product, so all of its steps have been looked at by then, and the
          // same rows are left out in every run
          for (int w = 0; w < NQ; ++w) {
            const int c0 = word >> (8 * w) & 7, c1 = c0 + (word >> (8 * w + 3) & 7);
            if (__any_sync(0xffffffffu, bad && row < c1 * PIECE && row + p.box > c0 * PIECE) && lane == 0)
              atomicOr(&s_tile[e].bad, 1 << w);
          }
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * (uint32_t)(p.box * 128);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t slot = ring % NS, round = ring / NS;
          ++ring;
          if (!wait(&bar_empty[slot], (round & 1) ^ 1)) {
            ok = false;
            break;
          }
          unsigned char* dst = sRing + slot * C::SLOT + (KV8 ? BN * 128 : 0);
          // (the word of step n is read with K_n; with the slot of K_{n + 8} free, K_{n + 4} at least is used up)
          if (kv == 0 && lane == 0) s_step[(ring - 1) / 2 % 8] = word;
          const bool land = KV8 || (kv == 1 && has_gaps(r));
          uint64_t* bar = land ? &bar_land[slot] : &bar_full[slot];
          const uint32_t bit = 1u << slot;
          used |= bit;
          loads ^= bit;
          if (land) landing ^= bit;
          last_land = land ? last_land | bit : last_land & ~bit;
          if constexpr (KV8) {
            if (lane == 0) {
              LoadDesc d;
              d.r = r;
              d.zero = kv;
              d.q_first = QCONV && i == 0 && kv == 0;
              d.q_par = t & 1;
              d.entry = (int)e;
              d.nq = nq;
              d.stop = 0;
              s_ld[slot] = d;
            }
          }
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (load) tma_load_3d(dst + half * BN * 128 + row * 128, kv ? &mv : &mk, bar, half * 64, ti.kvh, at);
        }
      }
    }
    if constexpr (KV8) {
      // no more loads: let the widening warps leave
      const uint32_t slot = ring % NS, round = ring / NS;
      if (ok && wait(&bar_empty[slot], (round & 1) ^ 1) && lane == 0) {
        s_ld[slot].stop = 1;
        mbar_arrive(&bar_land[slot]);
      }
    }
    if (!ok && lane == 0) {
      // let every copy this warp issued land before the CTA may exit (a slot's loads before its last were
      // consumed; parity 1 after the first load: phase 0)
      if (q_loads > 0) mbar_wait(QCONV ? &bar_qland : &bar_q, (q_loads - 1) & 1, 500000000ull);
      for (int s = 0; s < NS; ++s)
        if (used >> s & 1) {
          const bool land = last_land >> s & 1;
          mbar_wait(land ? &bar_land[s] : &bar_full[s], (((land ? landing : loads) >> s) & 1) ^ 1, 500000000ull);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    // The whole warp runs this loop and elect.sync picks the lane that issues. The tensor pipe holds
    // only a few products ahead of the issue, so every instruction between them counts: ring
    // positions advance step by step, ranges come as words, and a whole step's products are unrolled.
    const uint32_t id_pv = idesc_f16(BM, D, BF16, true), id_qk = idesc_f16(BM, 0, BF16, false);
    const uint32_t ring_u32 = smem_u32(sRing);
    const uint64_t qd = smem_desc(smem_u32(sQ), 16, 1024, LAYOUT_SW128);
    uint32_t p_use = 0;                           // parity of each query tile's hand-offs, a bit a tile
    uint32_t ks = 0, kph = 0, n = 0;              // slot and phase of the next K; steps so far
    auto issue_qk = [&](int w, uint32_t slot, uint32_t b) {
      const uint64_t kd = smem_desc(ring_u32 + slot * C::SLOT, 16, 1024, LAYOUT_SW128);
      const uint32_t c0 = b & 7, nc = b >> 3 & 7;
      const uint32_t idesc = id_qk | (nc * (PIECE >> 3)) << 17;
      const uint32_t dt = tmem + w * 128 + c0 * PIECE;
      const uint64_t kc = kd + (uint64_t)(c0 * (PIECE * 128 >> 4)), qw = qd + (uint64_t)(w * (C::Q_BYTES >> 4));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * BM * 128 + (kk % 4) * 32, offk = (kk / 4) * BN * 128 + (kk % 4) * 32;
        mma_f16_ss_warp(dt, qw + (uint64_t)(off >> 4), kc + (uint64_t)(offk >> 4), idesc, kk > 0 ? 1u : 0u);
      }
      mma_commit_warp(&bar_sfull[w]);
    };
    // O_w (+)= P_w V, the weights handed over in two halves of the step's pieces
    auto issue_pv = [&](int w, uint64_t vd, uint32_t b, uint32_t acc, uint32_t par) {
      const uint32_t dt = tmem + 256 + w * 128, at = tmem + w * 128;
      if (!wait(&bar_pfull[w][0], par)) return false;
      tc_fence_after();
      if ((b & 63) == WHOLE_STEP) {
#pragma unroll
        for (int kk = 0; kk < BN / 32; ++kk)
          mma_ts_warp(dt, at + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), id_pv, kk > 0 ? 1u : acc);
        if (!wait(&bar_pfull[w][1], par)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = BN / 32; kk < BN / 16; ++kk)
          mma_ts_warp(dt, at + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), id_pv, 1u);
      } else {
        const uint32_t c0 = b & 7, c1 = c0 + (b >> 3 & 7), mid = (c0 + c1 + 1) >> 1;
        for (uint32_t c = c0; c < c1; ++c) {
          if (c == mid) {
            if (!wait(&bar_pfull[w][1], par)) return false;
            tc_fence_after();
          }
#pragma unroll
          for (uint32_t h = 0; h < PIECE / 16; ++h) {
            const uint32_t kk = c * (PIECE / 16) + h;
            mma_ts_warp(dt, at + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), id_pv, acc);
            acc = 1;
          }
        }
        if (mid == c1 && !wait(&bar_pfull[w][1], par)) return false;   // (one piece: an empty second half)
      }
      return true;
    };
    bool ok = true;
    for (uint32_t t = 0; ok; ++t) {
      const uint32_t e = t & 1;
      if (!wait(&bar_tfull[e], (t >> 1) & 1)) break;
      if (!s_tile[e].valid) break;
      const int nq = s_tile[e].np > p.PP ? 2 : 1, steps = s_tile[e].steps;
      ok = wait(&bar_q, t & 1);
      tc_fence_after();
      uint32_t vs = ks, prev = 0, acc = 0;   // V_{j-1}; the last step's word; a bit a query tile begun
      // step j: O_w (+)= P_w V_{j-1}, then S_w = Q_w K_j^T, for each query tile w that sees it. The
      // waits for K_j and V_j stand behind products already queued.
      for (int j = 0; j <= steps && ok; ++j) {
        const bool qk = j < steps;
        uint32_t now = 0;
        const uint64_t vd = smem_desc(ring_u32 + vs * C::SLOT, BN * 128, 1024, LAYOUT_SW128);
        const uint32_t kslot = ks, kphase = kph;
        uint32_t nvs = ks + 1, nvph = kph;   // V_j
        if (nvs == (uint32_t)NS) {
          nvs = 0;
          nvph ^= 1;
        }
#pragma unroll
        for (int w = 0; w < NQ; ++w) {
          if (w >= nq) break;
          const uint32_t pb = prev >> (8 * w);
          if (pb & 56) {
            ok = issue_pv(w, vd, pb, acc >> w & 1, p_use >> w & 1);
            if (!ok) break;
            p_use ^= 1u << w;
            acc |= 1u << w;
            if (pb & 128) mma_commit_warp(&bar_odone[w]);
          }
          if (w == nq - 1 && j > 0) mma_commit_warp(&bar_empty[vs]);
          if (qk) {
            if (w == 0) {
              ok = wait(&bar_full[kslot], kphase);
              now = s_step[n % 8];
            }
            if (w == nq - 1 && j > 0 && ok) ok = wait(&bar_full[nvs], nvph);
            if (!ok) break;
            const uint32_t nb = now >> (8 * w);
            if (nb & 56) issue_qk(w, kslot, nb);
          }
        }
        if (!ok) break;
        if (qk) {
          mma_commit_warp(&bar_empty[kslot]);
          if (j == steps - 1) mma_commit_warp(&bar_qempty);
          if (j == 0) ok = wait(&bar_full[nvs], nvph);
          vs = nvs;
          ks = nvs + 1;
          kph = nvph;
          if (ks == (uint32_t)NS) {
            ks = 0;
            kph ^= 1;
          }
          ++n;
        }
        prev = now;
      }
      if (ok && lane == 0) mbar_arrive(&bar_tempty[e]);
      __syncwarp();
    }
  } else if (warp >= HELPER) {
    if constexpr (KV8) {
      // ------------------------------------------------------ e4m3: widening
      const int cw = warp - HELPER;
      for (uint32_t n = 0;; ++n) {
        const uint32_t slot = n % NS;
        if (!wait(&bar_land[slot], (n / NS) & 1)) break;
        // (written before the load's barrier completed)
        const LoadDesc d = s_ld[slot];
        if (d.stop) break;
        if (QCONV && d.q_first) {
          if (!wait(&bar_qland, d.q_par)) break;
          if (cw < d.nq) narrow_q(sQ + cw * C::Q_BYTES, &s_back[d.entry][cw * BM], lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_q);
        }
        widen_rows(sRing + slot * C::SLOT, d, cw, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_full[slot]);
      }
    } else {
      // -------------------------------------- zeros for values that nobody sees
      uint32_t ring = 0, landed = 0;   // landed: parity of each slot's loads of this kind, a bit a slot
      bool ok = true;
      for (uint32_t t = 0; ok; ++t) {
        const uint32_t e = t & 1;
        if (!wait(&bar_tfull[e], (t >> 1) & 1)) break;
        const Tile ti = s_tile[e];
        if (!ti.valid) break;
        for (int i = 0; i < ti.steps; ++i) {
          const Range r = union_range(ti, step_key(ti, i));
          const uint32_t slot = (ring + 2 * i + 1) % NS;
          if (!has_gaps(r)) continue;
          if (!wait(&bar_land[slot], (landed >> slot) & 1)) {
            ok = false;
            break;
          }
          landed ^= 1u << slot;
          for (int h = 0; h < C::HALVES; ++h) {
            uint4* base = reinterpret_cast<uint4*>(sRing + slot * C::SLOT + h * BN * 128);
            for (int q = max(r.a, r.c0 * PIECE) * 8 + lane; q < r.b * 8; q += 32) base[q] = make_uint4(0, 0, 0, 0);
            for (int q = r.e * 8 + lane; q < r.c1 * PIECE * 8; q += 32) base[q] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();   // the MMA (async proxy) reads what these threads wrote
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_full[slot]);
        }
        ring += 2 * ti.steps;
        if (ok && lane == 0) mbar_arrive(&bar_tempty[e]);
        __syncwarp();
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // The softmax threads share their sub-partitions with the MMA warp, whose issue slots dense work
    // here takes away: three-input maxima, fp32x2 multiply-adds and sums. A whole step (all four
    // pieces, every column seen) keeps its scores in registers; another reads them twice, a piece
    // at a time (with both forms over registers the kernel spills: 16384 tokens at window 2048 took
    // 2261 us against 588). The weights go to the MMA warp in two halves of the step's pieces: the first
    // half's products run during the second half's exponentials.
    const int w = (warp - 2) >> 2;
    const int i = (warp & 3) * 32 + lane;         // row within the tile; warp & 3: its TMEM lane quarter
    const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + w * 128, to = ts + 256;
    const int pi = i / p.G;
    uint32_t my_s = 0, my_o = 0;
    // (a barrier for each half: the MMA warp may come to either after both are handed over)
    auto hand = [&](int h) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_pfull[w][h]);
    };
    for (uint32_t t = 0;; ++t) {
      const uint32_t e = t & 1;
      if (!wait(&bar_tfull[e], (t >> 1) & 1)) break;
      const Tile* tile = &s_tile[e];
      if (!tile->valid) break;
      bool ok = true;
      // (each tile's: a phase that is not waited for would be mistaken for the next)
      if constexpr (QCONV) {
        if (!wait(&bar_q, t & 1)) break;
        if (lane == 0) mbar_arrive(&bar_qempty);
      }
      const int npw = min(tile->np - w * p.PP, p.PP);   // positions of this query tile
      if (npw > 0) {
        const int pa = tile->p_first + w * p.PP, pb = pa + npw - 1;
        const int p_i = min(pa + pi, pb);
        float sc = p.scale_log2;
        if constexpr (KV8) sc *= __ldg(p.ks + tile->kvh);
        if constexpr (QCONV) sc *= __uint_as_float((uint32_t)s_back[e][w * BM + i] << 23);
        float m_run = -INFINITY, l_run = 0.f;
        bool first = true;
        // keys that every row of the tile sees: [0, all_sinks) and (all_lo, pa]
        const int steps = tile->steps, js = tile->js, ws = tile->ws - js * BN;
        const int first_key = max(0, pa - p.window + 1), all_lo = max(pb - p.window, -1);
        const int my_sinks = min(p.sinks, first_key);
        for (int j = 0; j < steps; ++j) {
          const int k0 = j * BN + (j < js ? 0 : ws);
          if (!(k0 < my_sinks || (k0 + BN > first_key && k0 <= pb))) continue;
          const bool whole = (k0 > all_lo && k0 + BN - 1 <= pa) || k0 + BN <= my_sinks;
          // S_w complete also means every earlier MMA (the PV that read P_w) is done
          if (!wait(&bar_sfull[w], my_s & 1)) {
            ok = false;
            break;
          }
          ++my_s;
          tc_fence_after();
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
          float2 ls[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
          auto top = [&]() {
            return max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
          };
          auto minus = [&]() { return SHIFT - (m_run == -INFINITY ? 0.f : m_run); };
          if (whole) {
            uint32_t r[BN / PIECE][PIECE];
#pragma unroll
            for (int c = 0; c < BN / PIECE; ++c) tmem_ld32(ts + c * PIECE, r[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < BN / PIECE; ++c) reg_fence(r[c]);
#pragma unroll
            for (int c = 0; c < BN / PIECE; ++c) max_of(r[c], mx);
            new_maximum<D>(top(), to, first, m_run, l_run);
            const float nm = minus();
#pragma unroll
            for (int c = 0; c < BN / PIECE; ++c) {
              weigh<MT>(r[c], sc, nm, ls, ts + c * 16);
              if (c == BN / PIECE / 2 - 1) hand(0);
            }
          } else {
            const Range rg = range_of(k0, my_sinks, first_key, pb + 1);
            const RowStep st{p_i - k0, max(p_i - p.window, -1) - k0, p.sinks - k0};
#pragma unroll 1
            for (int c = rg.c0; c < rg.c1; ++c) {
              uint32_t r[PIECE];
              tmem_ld32_wait(ts + c * PIECE, r);
              hide(r, seen_bits(st, c));
              max_of(r, mx);
            }
            new_maximum<D>(top(), to, first, m_run, l_run);
            const float nm = minus();
            const int mid = (rg.c0 + rg.c1 + 1) >> 1;
            // (the weights of piece c go over scores of pieces up to c / 2)
#pragma unroll 1
            for (int c = rg.c0; c < rg.c1; ++c) {
              uint32_t r[PIECE];
              tmem_ld32_wait(ts + c * PIECE, r);
              hide(r, seen_bits(st, c));
              weigh<MT>(r, sc, nm, ls, ts + c * 16);
              if (c == mid - 1) hand(0);
            }
          }
          hand(1);
          first = false;
          l_run += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
        }
        if (ok) ok = wait(&bar_odone[w], my_o & 1);
        ++my_o;
        tc_fence_after();
        if (ok) {
          const int bad = *(volatile const int*)&s_tile[e].bad >> w & 1;
          const bool store = pi < npw && !bad;
          const float inv = (KV8 ? __ldg(p.vs + tile->kvh) : 1.f) / l_run;
          const int64_t at = (int64_t)(tile->row0 + w * p.PP + pi) * p.Hq + tile->kvh * p.G + (i - pi * p.G);
          TQ* dst = (TQ*)p.out + at * D;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_wait(to + c * 32, o);
            if (!store) continue;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                x[k] = pack2<TQ>(__uint_as_float(o[v * 16 + 2 * k]) * inv, __uint_as_float(o[v * 16 + 2 * k + 1]) * inv);
              store16(dst + c * 32 + v * 16, x, p.wide);
            }
          }
          if (store && p.lse) p.lse[at] = (m_run + __log2f(l_run) - SHIFT) * LN2;
          if (bad && i == 0) atomicOr(p.dev_status, PKV_DEV_BAD_PAGE);
        }
        tc_fence_before();
      }
      if (!ok) break;
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

template <int D, typename TQ, bool KV8>
cudaError_t launch(const WindowArgs& a, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<uint64_t> ready{0};   // devices whose kernel attribute is set
  const uint64_t bit = (uint64_t)1 << (a.dev.id & 63);
  if (!(ready.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(window_tiles_kernel<D, TQ, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  TilesP p;
  p.cu = a.cu;
  p.kv_lens = a.kv_lens;
  p.tables = a.page_tables;
  p.B = a.B;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.PP = BM / p.G;
  p.P = a.P;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.window = a.window;
  p.sinks = a.sinks;
  p.min_q = a.tile_min_q;
  p.box = a.P < PIECE ? a.P : PIECE;
  p.beside = a.tile_min_q > 1;
  p.wide = ((uintptr_t)a.out & 31) == 0;
  p.div = page_div(a.P);
  p.scale_log2 = a.scale * LOG2E;
  p.ks = a.k_scale;
  p.vs = a.v_scale;
  p.out = a.out;
  p.lse = a.lse;
  p.dev_status = a.dev.status;
  const CUtensorMapDataType dt =
      std::is_same<TQ, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapDataType kdt = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : dt;
  const int kelt = KV8 ? 1 : 2;
  const int64_t rows = (int64_t)a.num_pages * a.P;
  CUtensorMap mq, mk, mv;
  if (!make_map_heads(&mq, a.q, dt, D, a.Hq, a.T, p.G, p.PP) ||
      !make_map_boxed(&mk, a.k_cache, kdt, kelt, D, a.Hkv, rows, 128 / kelt, p.box) ||
      !make_map_boxed(&mv, a.v_cache, kdt, kelt, D, a.Hkv, rows, 128 / kelt, p.box))
    return cudaErrorInvalidValue;
  const int64_t most = ((int64_t)a.B + a.T / (NQ * p.PP)) * a.Hkv;   // work tiles
  if (most > INT32_MAX - 65535) return cudaErrorInvalidValue;         // (their numbers are 32 bits)
  const int64_t grid = most < a.dev.num_sms ? most : a.dev.num_sms;
  KernelTimer timer("window_tiles", s);
  return launch_after_trigger(window_tiles_kernel<D, TQ, KV8>, dim3((unsigned)grid),
                              dim3((HELPER + (KV8 ? 2 : 1)) * 32), C::SMEM, s, mq, mk, mv, p);
}

}  // namespace

// 16-bit caches at head_dim 64 and 128, e4m3 caches at 128, pages that 128-key tiles divide or that
// divide them (blocks of at least 8 rows: one swizzle pattern).
bool window_tiles_supported(int kv_dtype, int D, int P) {
  if (kv_dtype == PKV_F32 || D == 256 || (kv_dtype == PKV_FP8_E4M3 && D != 128)) return false;
  return P % BN == 0 || (P >= 8 && BN % P == 0);
}

cudaError_t launch_window_tiles(const WindowArgs& a, cudaStream_t s) {
  if (a.kv_dtype == PKV_FP8_E4M3)
    return a.dtype == PKV_BF16 ? launch<128, __nv_bfloat16, true>(a, s) : launch<128, __half, true>(a, s);
  if (a.dtype == PKV_BF16) return a.D == 64 ? launch<64, __nv_bfloat16, false>(a, s) : launch<128, __nv_bfloat16, false>(a, s);
  return a.D == 64 ? launch<64, __half, false>(a, s) : launch<128, __half, false>(a, s);
}

}  // namespace pkv
