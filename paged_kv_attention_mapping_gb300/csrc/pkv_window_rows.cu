// Window attention for few rows of a sequence (decode rows, drafted tokens, any shape
// that the tile kernel does not take).
//
// A row at position p sees the keys j <= p with j > p - window or j < sinks: at most
// window + sinks of them, whatever the context's length. A piece of work is up to 8 NT
// columns (rows x query heads of one KV head, that is) of one sequence over the keys that
// some of them sees. The bound is HBM: a key and a value are read once for all columns.
//
// A warp copies 16 keys and values a step, whole rows an instruction, asynchronously into a ring of
// its own in shared memory, two or three steps ahead: many more bytes are in flight than registers
// would hold, no warp waits for another, and any page size does. Scores are S^T = K Q^T with 16
// keys as the rows of m16n8k16; the channels of a product are permuted, alike in K and Q, so that 16
// bytes of a key are a lane's own operand. The output is O^T += V^T P^T with 16 channels as the rows; a
// lane takes 16 bytes of each of four keys and pairs them with byte permutes, and P^T is S^T transposed
// in registers. A warp has a running maximum and sum of its own; warps are merged at the end in shared
// memory, and the CTAs that share a piece's keys (a cluster) through distributed shared memory: no
// workspace and one launch.
//
// 128 rows of up to 4096 keys, 32 / 8 heads of 128, bf16: 249 us, 6.4 TB/s, 96 % of the measured copy; 64
// rows of 132 keys, heads of 64: 5.9 us, four dependent reads and the join. Steps taken (the first case):
// operands straight from global memory into registers 308 us; copied asynchronously by the lane that
// consumes them, 64 bytes of eight rows an instruction, 311; whole rows an instruction 252; keys in one
// page without a look-up a row 244. Ring depths: two steps of 8 KB 243, but 113 us against 100 for 38 rows.
#include <cuda_runtime.h>

#include <atomic>

#include "pkv_sm100.cuh"
#include "pkv_window_common.cuh"

namespace pkv {
using namespace sm100;
using namespace window;

namespace {

constexpr int NW = 4;              // warps of a CTA
constexpr int THREADS = NW * 32;
constexpr int MAX_SPLIT = 8;       // CTAs of a cluster (portable)
// f16 softmax weights carry this power of two, so that small ones are not lost to f16's
// smallest exponents; a weight is at most 1, so the largest is 2^15 < 65504.
constexpr float F16_SHIFT = 15.f;

struct RowsP {
  const void *q, *kc, *vc;
  const int32_t *cu, *kv_lens, *tables;
  int32_t B, T, Hq, Hkv, G, per, P, num_pages, max_pages, window, sinks, tile_min_q, parts, heads;
  int32_t numbered;  // rows for each number of first_piece: per, or 1
  int32_t per_seq;   // pieces numbered for each sequence (0: as first_piece has it)
  int32_t beside;    // launched beside the tile kernel, which is the one before it
  PageDiv div;
  float scale_log2;
  const float *ks, *vs;
  void* out;
  float* lse;
  int32_t* dev_status;
};

// One piece of work of this CTA (all CTAs of a cluster have the same).
struct Piece {
  int row0, np, p_first, kvh, part, b;   // first packed row, rows, position of the first
  Keys keys;
  int split, splits;
};

// False: nothing to do (for every CTA of the cluster).
__device__ __forceinline__ bool find_piece(const RowsP& p, Piece* w) {
  const int lane = threadIdx.x & 31;
  // The tile kernel lets this one start once the kernel before it is done, so nothing is left to wait
  // for but its end, which the last block sees to: this grid is not over before it.
  if (!p.beside) {
    pdl_wait();
    pdl_trigger();
  } else {
    __threadfence();   // (no line that an earlier kernel left in this SM's L1 is read)
  }
  if (blockIdx.x == 0 && !p.beside) check_cu(p.cu, p.B, p.T, p.dev_status);
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(w->splits));
  w->split = (int)cluster_rank();
  int64_t u = blockIdx.x / w->splits;
  w->part = (int)(u % p.parts);
  u /= p.parts;
  w->kvh = (int)(u % p.Hkv);
  const int64_t slot = u / p.Hkv;
  const int b = p.per_seq ? (int)(slot / p.per_seq) : find_seq(p.cu, p.B, slot, p.numbered, lane);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), L = __ldg(p.kv_lens + b);
  const int64_t first = p.per_seq ? (int64_t)b * p.per_seq : first_piece(b, c0, p.numbered);
  const int64_t q0 = (slot - first) * p.per;
  if (c0 < 0 || c1 < c0 || c1 > p.T) return false;   // (before the difference, which could wrap to a small count)
  const int n = c1 - c0;
  if (q0 < 0 || q0 >= n || n >= p.tile_min_q) return false;
  if (L < n || L > (int64_t)p.max_pages * p.P) {
    if (q0 == 0 && w->kvh == 0 && w->part == 0 && w->split == 0 && threadIdx.x == 0)
      atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    return false;
  }
  w->b = b;
  w->row0 = c0 + (int)q0;
  w->np = min(p.per, n - (int)q0);
  w->p_first = L - n + (int)q0;
  w->keys = keys_of(w->p_first, w->p_first + w->np - 1, p.window, p.sinks);
  return true;
}

__device__ __forceinline__ void end(const RowsP& p) {
  if (p.beside && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// Slot of key number i in the pool: -1 past the last key, -2 where its page is outside it.
__device__ __forceinline__ int slot_of(const RowsP& p, const Piece& w, int i) {
  if (i >= w.keys.n) return -1;
  const int key = key_at(w.keys, i);
  const int pg = page_of(key, p.div);
  const int id = __ldg(p.tables + (int64_t)w.b * p.max_pages + pg);
  return id < 0 || id >= p.num_pages ? -2 : id * p.P + (key - pg * p.P);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float ld_cluster_f(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// 16 bytes from global to shared memory, zeros where `from` is null.
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, const void* any) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from ? from : any), "r"(from ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The warps' results, then the cluster's: maximum (log2 units), sum and unnormalised
// output of every column.
template <int COLS, int D>
struct Merge {
  static constexpr int LD = D + 4;
  float m[NW][COLS], l[NW][COLS];
  float cm[COLS], cl[COLS];   // this CTA's
  alignas(16) float o[NW][COLS][LD];
};

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 r;
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(dst) = r;
  }
}

// Column c of the piece is query head kvh * G + part * heads + c % heads of row c / heads. (The
// last part of a group that HB does not divide has columns without a head.)
template <typename TQ, int COLS, int D>
__device__ __forceinline__ void finish(const RowsP& p, const Piece& w, Merge<COLS, D>& s, int& s_bad, float shift) {
  const int tid = threadIdx.x, heads = p.heads;
  const int cols = w.np * heads;
  __syncthreads();
  if (w.splits > 1) {
    // this CTA's warps into one: each thread the 4 values that it alone reads and writes
    for (int u = tid; u < COLS * (D / 4); u += THREADS) {
      const int c = u / (D / 4), d = (u - c * (D / 4)) * 4;
      float top = s.m[0][c];
#pragma unroll
      for (int k = 1; k < NW; ++k) top = fmaxf(top, s.m[k][c]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float f = s.m[k][c] == -INFINITY ? 0.f : ex2(s.m[k][c] - top);
        // (a warp without a key, or with none but -inf scores: its sum is 0, or NaN, and its weight 1)
        const float g = s.m[k][c] == -INFINITY ? 1.f : f;
        const float4 x = *reinterpret_cast<const float4*>(&s.o[k][c][d]);
        a.x = fmaf(x.x, g, a.x);
        a.y = fmaf(x.y, g, a.y);
        a.z = fmaf(x.z, g, a.z);
        a.w = fmaf(x.w, g, a.w);
        l = fmaf(s.l[k][c], g, l);
      }
      *reinterpret_cast<float4*>(&s.o[0][c][d]) = a;
      if (d == 0) {
        s.cm[c] = top;
        s.cl[c] = l;
      }
    }
    fence_cluster();
    cluster_sync_all();
  }
  const int parts = w.splits > 1 ? w.splits : NW;
  bool any_bad = s_bad != 0;
  if (w.splits > 1) {
    any_bad = false;
    for (int k = 0; k < parts; ++k) any_bad |= __float_as_int(ld_cluster_f(map_to_rank(&s_bad, k))) != 0;
  }
  if (any_bad && tid == 0 && w.split == 0) atomicOr(p.dev_status, PKV_DEV_BAD_PAGE);
  for (int u = tid * w.splits + w.split; u < cols * (D / 8) && !any_bad; u += THREADS * w.splits) {
    const int c = u / (D / 8), d = (u - c * (D / 8)) * 8;
    float top = -INFINITY, l = 0.f, x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (w.splits > 1) {
      for (int k = 0; k < parts; ++k) top = fmaxf(top, ld_cluster_f(map_to_rank(&s.cm[c], k)));
      for (int k = 0; k < parts; ++k) {
        const float m = ld_cluster_f(map_to_rank(&s.cm[c], k));
        const float f = m == -INFINITY ? 1.f : ex2(m - top);
        const uint32_t at = map_to_rank(&s.o[0][c][d], k);
        const float4 a = ld_cluster_f4(at), b = ld_cluster_f4(at + 16);
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        l = fmaf(ld_cluster_f(map_to_rank(&s.cl[c], k)), f, l);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], f, x[e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NW; ++k) top = fmaxf(top, s.m[k][c]);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float f = s.m[k][c] == -INFINITY ? 1.f : ex2(s.m[k][c] - top);
        l = fmaf(s.l[k][c], f, l);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(s.o[k][c][d + e], f, x[e]);
      }
    }
    const int row = w.row0 + c / heads, head = w.kvh * p.G + w.part * heads + c % heads;
    if (w.part * heads + c % heads >= p.G) continue;
    const float inv = (p.vs ? __ldg(p.vs + w.kvh) : 1.f) / l;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= inv;
    const int64_t at = (int64_t)row * p.Hq + head;
    store8((TQ*)p.out + at * D + d, x);
    if (d == 0 && p.lse) p.lse[at] = (top + __log2f(l) - shift) * LN2;
  }
  if (w.splits > 1) cluster_sync_all();   // peers have read this CTA's shared memory
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's step of 16 keys in shared memory: their rows, then their values' rows, each row's 16-byte
// chunks permuted within 128 bytes (by `turn`), so that the operand loads meet no bank twice: a
// quarter of a warp takes chunks t + 4 j of keys g and g + 1, or chunks g and g + 1 of values 2t (or 2t + 1).
template <bool KV8, int D>
struct Share {
  static constexpr int RB = D * (KV8 ? 1 : 2);           // bytes of a key's row
  static constexpr int CH = RB / 16;                     // its chunks
  static constexpr int KJ = RB / 64;                     // a lane's chunks of a key: t + 4 j
  static constexpr int SEGS = RB >= 128 ? RB / 128 : 1;  // a lane's pieces of a value: at segment * 128 + g * VB
  static constexpr int VB = RB >= 128 ? 16 : 8;
  static constexpr int BYTES = 2 * 16 * RB;              // of a warp's step
  // steps of a ring, all but one of them in flight: four of 2 KB, three of more (of 8 KB two CTAs of 96 KB an SM, of 16
  // KB, head_dim 256 in 16 bits, one of 192)
  static constexpr int STAGES = BYTES >= 4096 ? 3 : 4;
  static __device__ __forceinline__ int turn(int r) { return ((r & 6) ^ (r & 1) << 2) & (RB >= 128 ? 7 : 3); }
};

// TQ: type of q and out. KV8: the caches hold e4m3 codes (products in f16), else TQ.
template <typename TQ, bool KV8, int D, int NT>
__global__ void __launch_bounds__(THREADS) window_rows_kernel(const __grid_constant__ RowsP p) {
  using MT = typename std::conditional<KV8, __half, TQ>::type;
  using H = Share<KV8, D>;
  constexpr bool F16 = std::is_same<MT, __half>::value;
  constexpr float SHIFT = F16 ? F16_SHIFT : 0.f;
  constexpr int COLS = 8 * NT, RB = H::RB, KJ = H::KJ, SEGS = H::SEGS, VB = H::VB, VR = VB / 4, ST = H::STAGES;
  constexpr int CPR = KV8 ? 4 : 2;                // channels a 32-bit register holds
  constexpr int MT_SEG = VR * CPR / 2;            // 16-channel output tiles of a segment
  extern __shared__ __align__(128) unsigned char dyn[];
  Merge<COLS, D>& sm = *reinterpret_cast<Merge<COLS, D>*>(dyn);   // (once the copies are used up)
  __shared__ int s_bad;
  Piece w;
  if (!find_piece(p, &w)) return end(p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) s_bad = 0;

  // 16 keys of this warp a step; lane i % 16 looks up key i
  const int step = w.splits * NW * 16, base0 = (w.split * NW + warp) * 16;
  unsigned char* const mine = dyn + warp * ST * H::BYTES;
  const int64_t row = (int64_t)p.Hkv * RB;
  const char* const kb = (const char*)p.kc + w.kvh * RB + lane % H::CH * 16;
  const int64_t k_to_v = (const char*)p.vc - (const char*)p.kc;
  bool bad = false;
  auto fetch = [&](int slot, int stage) {
    bad |= slot == -2;
    // a copy instruction takes whole rows: 32 / CH of them. Keys that follow one another in one page
    // (most steps) need no look-up a row
    const uint32_t to = smem_u32(mine + stage * H::BYTES);
    const int s0 = __shfl_sync(0xffffffffu, slot, 0);
    if (__all_sync(0xffffffffu, slot >= 0 && slot == s0 + (lane & 15))) {
      const char* src = kb + (s0 + lane / H::CH) * row;
#pragma unroll
      for (int i = 0; i < H::CH / 2; ++i) {
        const int r = i * (32 / H::CH) + lane / H::CH;
        const uint32_t at = to + r * RB + ((lane % H::CH) ^ H::turn(r)) * 16;
        cp_async_16(at, src);
        cp_async_16(at + 16 * RB, src + k_to_v);
        src += 32 / H::CH * row;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < H::CH / 2; ++i) {
      const int r = i * (32 / H::CH) + lane / H::CH;
      const int s = __shfl_sync(0xffffffffu, slot, r);
      const char* src = s >= 0 ? kb + s * row : nullptr;
      const uint32_t at = to + r * RB + ((lane % H::CH) ^ H::turn(r)) * 16;
      copy_async(at, src, p.kc);
      copy_async(at + 16 * RB, src ? src + k_to_v : nullptr, p.kc);
    }
  };
  int slots[ST];
#pragma unroll
  for (int i = 0; i < ST; ++i) slots[i] = slot_of(p, w, base0 + i * step + (lane & 15));
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    if (base0 + i * step < w.keys.n) fetch(slots[i], i);
    copy_commit();
  }
  int next = slots[ST - 1];

  // queries: column g of each 8, its channels in the order in which the lane's pieces of a
  // key come
  uint32_t qf[NT][D / 16][2];
  float cs[NT][2];   // what turns a score of columns 2t, 2t + 1 into log2 units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = nt * 8 + g;
    const bool have = c < w.np * p.heads;
    const int64_t at = (int64_t)(w.row0 + c / p.heads) * p.Hq + w.kvh * p.G + w.part * p.heads + c % p.heads;
    const TQ* src = (const TQ*)p.q + at * D;
    float back = 1.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int e = KV8 ? (t + 4 * (ks / 4)) * 16 + 4 * (ks % 4) : (t + 4 * (ks / 2)) * 8 + 4 * (ks % 2);
      const uint2 x = have ? *reinterpret_cast<const uint2*>(src + e) : make_uint2(0, 0);
      qf[nt][ks][0] = x.x;
      qf[nt][ks][1] = x.y;
    }
    if constexpr (KV8 && std::is_same<TQ, __nv_bfloat16>::value) {
      // bf16 has exponents that f16 lacks: a row goes to f16 times the power of two that
      // brings its largest value to 2^8 .. 2^9, and the scores are scaled back
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[nt][ks][k] << 16)),
                                 fabsf(__uint_as_float(qf[nt][ks][k] & 0xffff0000u))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int eb = (int)(__float_as_uint(top) >> 23);
      const int fe = eb == 0 || eb == 255 ? 127 : min(max(262 - eb, 2), 252);
      const float f = __uint_as_float((uint32_t)fe << 23);
      back = __uint_as_float((uint32_t)(254 - fe) << 23);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = qf[nt][ks][k];
          qf[nt][ks][k] = pack2<__half>(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
        }
    }
    const float f = p.scale_log2 * (KV8 ? __ldg(p.ks + w.kvh) : 1.f) * back;
    cs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
    cs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
  }

  int pos[NT][2];   // positions of columns 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) pos[nt][k] = w.p_first + (nt * 8 + 2 * t + k) / p.heads;
  float m[NT][2], l[NT][2], o[NT][SEGS * MT_SEG][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[nt][k] = -INFINITY;
      l[nt][k] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < SEGS * MT_SEG; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
  }

  // TT: tiles of columns that have any (a count known when compiled lets them overlap)
  int stage = 0;
  auto work = [&](auto tt) {
    constexpr int TT = decltype(tt)::value;
    for (int base = base0; base < w.keys.n; base += step) {
      __syncwarp();   // every lane has read the last step
      // the step ST - 1 ahead goes where that was, and the page ids of the one behind it are looked up
      const int ahead = base + (ST - 1) * step;
      if (ahead < w.keys.n) {
        fetch(next, stage == 0 ? ST - 1 : stage - 1);
        next = slot_of(p, w, ahead + step + (lane & 15));
      }
      copy_commit();
      copy_wait<ST - 1>();
      __syncwarp();   // every lane's copies have landed
      const unsigned char* const ks = mine + stage * H::BYTES;
      const unsigned char* const vs = ks + 16 * RB;
      stage = stage + 1 == ST ? 0 : stage + 1;
      float c[TT][4];
#pragma unroll
      for (int nt = 0; nt < TT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) c[nt][k] = 0.f;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int at = g * RB + ((t + 4 * j) ^ H::turn(g)) * 16;   // (keys g and g + 8 turn alike)
        const uint4 k0 = *reinterpret_cast<const uint4*>(ks + at);
        const uint4 k1 = *reinterpret_cast<const uint4*>(ks + at + 8 * RB);
        const uint32_t a[4] = {k0.x, k0.y, k0.z, k0.w};
        const uint32_t b[4] = {k1.x, k1.y, k1.z, k1.w};
        if constexpr (KV8) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t a0 = widen(a[r]), a1 = widen(b[r]), a2 = widen(a[r] >> 16), a3 = widen(b[r] >> 16);
#pragma unroll
            for (int nt = 0; nt < TT; ++nt) mma<MT>(c[nt], a0, a1, a2, a3, qf[nt][4 * j + r][0], qf[nt][4 * j + r][1]);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int nt = 0; nt < TT; ++nt)
              mma<MT>(c[nt], a[2 * r], b[2 * r], a[2 * r + 1], b[2 * r + 1], qf[nt][2 * j + r][0], qf[nt][2 * j + r][1]);
        }
      }

      // scores of keys g, g + 8 for columns 2t, 2t + 1, in log2 units. Most steps have 16 keys that
      // every row sees
      uint32_t pb[TT][2];
      const int ka = key_at(w.keys, base), kz = key_at(w.keys, base + 15);
      const bool all = base + 16 <= w.keys.n &&
                       (w.np == 1 || (kz <= w.p_first && (ka > w.p_first + w.np - 1 - p.window || kz < p.sinks)));
      const int i0 = base + g, i1 = i0 + 8;
      const int k0 = key_at(w.keys, i0), k1 = key_at(w.keys, i1);
#pragma unroll
      for (int nt = 0; nt < TT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float a = c[nt][k] * cs[nt][k], b = c[nt][2 + k] * cs[nt][k];
          if (!all) {
            const bool va = i0 < w.keys.n && (w.np == 1 || seen(k0, pos[nt][k], p.window, p.sinks));
            const bool vb2 = i1 < w.keys.n && (w.np == 1 || seen(k1, pos[nt][k], p.window, p.sinks));
            a = va ? a : -INFINITY;
            b = vb2 ? b : -INFINITY;
          }
          float top = fmaxf(a, b);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float mn = fmaxf(m[nt][k], top);
          const float use = mn == -INFINITY ? 0.f : mn;
          const float alpha = ex2(m[nt][k] - use);
          m[nt][k] = mn;
          a = ex2(a - use + SHIFT);
          b = ex2(b - use + SHIFT);
          l[nt][k] = fmaf(l[nt][k], alpha, a + b);
          c[nt][k] = a;
          c[nt][2 + k] = b;
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int i = 0; i < SEGS * MT_SEG; ++i) {
              o[nt][i][k] *= alpha;
              o[nt][i][2 + k] *= alpha;
            }
          }
        }
        pb[nt][0] = transpose8(pack2<MT>(c[nt][0], c[nt][1]));
        pb[nt][1] = transpose8(pack2<MT>(c[nt][2], c[nt][3]));
      }

      // O^T += V^T P^T: output tile i of segment j holds channels 2i, 2i + 1 of each lane's piece
#pragma unroll
      for (int j = 0; j < SEGS; ++j) {
        uint32_t vr[4][VR];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int r = 2 * t + (h & 1) + 8 * (h >> 1);
          const unsigned char* at = vs + r * RB + (VB == 16 ? (g + 8 * j) ^ H::turn(r) : (g >> 1) ^ H::turn(r)) * 16 +
                                    (VB == 16 ? 0 : (g & 1) * 8);
          if constexpr (VR == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            vr[h][0] = x.x;
            vr[h][1] = x.y;
            vr[h][2] = x.z;
            vr[h][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            vr[h][0] = x.x;
            vr[h][1] = x.y;
          }
        }
#pragma unroll
        for (int r = 0; r < VR; ++r) {
          const uint32_t v0 = vr[0][r], v1 = vr[1][r], v2 = vr[2][r], v3 = vr[3][r];
          if constexpr (KV8) {
            const uint32_t x0 = __byte_perm(v0, v1, 0x5140), x1 = __byte_perm(v2, v3, 0x5140);
            const uint32_t y0 = __byte_perm(v0, v1, 0x7362), y1 = __byte_perm(v2, v3, 0x7362);
            const uint32_t a0 = widen(x0), a1 = widen(x0 >> 16), a2 = widen(x1), a3 = widen(x1 >> 16);
            const uint32_t b0 = widen(y0), b1 = widen(y0 >> 16), b2 = widen(y1), b3 = widen(y1 >> 16);
#pragma unroll
            for (int nt = 0; nt < TT; ++nt) {
              mma<MT>(o[nt][j * MT_SEG + 2 * r], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
              mma<MT>(o[nt][j * MT_SEG + 2 * r + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
            }
          } else {
            const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
            const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
            for (int nt = 0; nt < TT; ++nt) mma<MT>(o[nt][j * MT_SEG + r], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          }
        }
      }
    }
  };
  if (NT == 1 || w.np * p.heads <= 8) work(std::integral_constant<int, 1>());
  else work(std::integral_constant<int, NT>());
  copy_wait<0>();
  __syncthreads();   // every warp's copies are used up (and s_bad is cleared)
  if (bad) s_bad = 1;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = nt * 8 + 2 * t + k;
      float s = l[nt][k];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (g == 0) {
        sm.m[warp][c] = m[nt][k];
        sm.l[warp][c] = s;
      }
#pragma unroll
      for (int j = 0; j < SEGS; ++j)
#pragma unroll
        for (int i = 0; i < MT_SEG; ++i)
          *reinterpret_cast<float2*>(&sm.o[warp][c][j * (D / SEGS) + g * (MT_SEG * 2) + 2 * i]) =
              make_float2(o[nt][j * MT_SEG + i][k], o[nt][j * MT_SEG + i][2 + k]);
    }
  finish<TQ, COLS, D>(p, w, sm, s_bad, SHIFT);
  end(p);
}

// fp32 caches, on the fused multiply-adds (tensor cores have no fp32 products): a piece is
// one row and HB of its query heads of a KV head. Eight lanes hold a key's channels (16-byte
// pieces e + 8 j), so a warp takes four keys at a time; q and the output stay in registers.
template <int D, int HB>
__global__ void __launch_bounds__(THREADS) window_rows_f32_kernel(const RowsP p) {
  constexpr int J = D / 32;   // a lane's pieces
  __shared__ Merge<HB, D> sm;
  __shared__ int s_bad;
  Piece w;
  if (!find_piece(p, &w)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = lane & 7, sub = lane >> 3;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  float4 q[HB][J], o[HB][J];
  float m[HB], l[HB];
#pragma unroll
  for (int h = 0; h < HB; ++h) {
    const int hh = w.part * HB + h;
    const float* src = (const float*)p.q + ((int64_t)w.row0 * p.Hq + w.kvh * p.G + hh) * D + e * 4;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      q[h][j] = hh < p.G ? *reinterpret_cast<const float4*>(src + j * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
      o[h][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    m[h] = -INFINITY;
    l[h] = 0.f;
  }
  bool bad = false;
  const int step = w.splits * NW * 4;
  int i = (w.split * NW + warp) * 4 + sub;
  int next = slot_of(p, w, i);
  for (; i - sub < w.keys.n; i += step) {
    const int slot = next;
    bad |= slot == -2;
    const int64_t at = ((int64_t)slot * p.Hkv + w.kvh) * D + e * 4;
    float4 k[J], v[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
      k[j] = slot >= 0 ? __ldg(reinterpret_cast<const float4*>((const float*)p.kc + at + j * 32))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < J; ++j)
      v[j] = slot >= 0 ? __ldg(reinterpret_cast<const float4*>((const float*)p.vc + at + j * 32))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    next = slot_of(p, w, i + step);
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        s = fmaf(q[h][j].x, k[j].x, fmaf(q[h][j].y, k[j].y, fmaf(q[h][j].z, k[j].z, fmaf(q[h][j].w, k[j].w, s))));
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s = i < w.keys.n ? s * p.scale_log2 : -INFINITY;
      // (each group of eight lanes has a running maximum of its own; a row of one position
      // sees every key of its piece)
      const float mn = fmaxf(m[h], s);
      const float use = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m[h] - use), a = exp2f(s - use);
      m[h] = mn;
      l[h] = fmaf(l[h], alpha, a);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        o[h][j].x = fmaf(o[h][j].x, alpha, a * v[j].x);
        o[h][j].y = fmaf(o[h][j].y, alpha, a * v[j].y);
        o[h][j].z = fmaf(o[h][j].z, alpha, a * v[j].z);
        o[h][j].w = fmaf(o[h][j].w, alpha, a * v[j].w);
      }
    }
  }
  if (bad) s_bad = 1;
#pragma unroll
  for (int h = 0; h < HB; ++h) {
    // the warp's four groups of lanes into one
#pragma unroll
    for (int x = 8; x < 32; x <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[h], x), lo = __shfl_xor_sync(0xffffffffu, l[h], x);
      const float top = fmaxf(m[h], mo);
      const float f = m[h] == -INFINITY ? 1.f : exp2f(m[h] - top), fo = mo == -INFINITY ? 1.f : exp2f(mo - top);
      m[h] = top;
      l[h] = l[h] * f + lo * fo;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        o[h][j].x = o[h][j].x * f + __shfl_xor_sync(0xffffffffu, o[h][j].x, x) * fo;
        o[h][j].y = o[h][j].y * f + __shfl_xor_sync(0xffffffffu, o[h][j].y, x) * fo;
        o[h][j].z = o[h][j].z * f + __shfl_xor_sync(0xffffffffu, o[h][j].z, x) * fo;
        o[h][j].w = o[h][j].w * f + __shfl_xor_sync(0xffffffffu, o[h][j].w, x) * fo;
      }
    }
    if (sub == 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) *reinterpret_cast<float4*>(&sm.o[warp][h][j * 32 + e * 4]) = o[h][j];
      if (e == 0) {
        sm.m[warp][h] = m[h];
        sm.l[warp][h] = l[h];
      }
    }
  }
  finish<float, HB, D>(p, w, sm, s_bad, 0.f);
}

struct Call {
  int64_t pieces, busy, keys;   // pieces of the grid, those of them with rows, keys of the longest
};

// CTAs that share a piece's keys: as many as have a place at once (`occupancy` an SM, an eighth of them
// left for sequences that have more pieces than the estimate), while each has two rounds of its warps.
// A second wave costs more than the wider split gains: bf16, D 128, 4096 keys: 8 pieces by 1 / 2 / 4 / 8
// CTAs take 54 / 31 / 19 / 13 us, 64 pieces 56 / 34 / 27 / 33; 64 of 516 keys 10.6 / 9.3 / 8.6 / 14.1; 256 of
// 260 keys 10 / 17 / 27 / 49; 72 pieces of 8000 e4m3 keys by 4 / 5 / 6 / 7: 59 / 51 / 46 / 68.
int splits_of(const Call& c, int occupancy, int num_sms) {
  int64_t s = (int64_t)occupancy * num_sms * 7 / 8 / c.busy;
  if (s > MAX_SPLIT) s = MAX_SPLIT;
  if (s > c.keys / (2 * NW * 16)) s = c.keys / (2 * NW * 16);
  return s < 1 ? 1 : (int)s;
}

template <typename K>
cudaError_t launch_kernel(K kernel, const WindowArgs& a, const Call& c, int smem, std::atomic<int>* occupancy,
                          cudaStream_t s, const RowsP& p) {
  int occ = occupancy[a.dev.id & 63].load();   // (the same for every call of this kernel on the device)
  if (occ == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, THREADS, smem);
    if (e != cudaSuccess) return e;
    if (occ < 1) return cudaErrorInvalidConfiguration;
    occupancy[a.dev.id & 63].store(occ);
  }
  const int splits = splits_of(c, occ, a.dev.num_sms);
  if (c.pieces * splits > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.pieces * splits));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename TQ, bool KV8, int D, int NT>
cudaError_t launch16(const WindowArgs& a, const Call& c, cudaStream_t s, const RowsP& p) {
  using H = Share<KV8, D>;
  constexpr int ring = NW * H::STAGES * H::BYTES, merge = sizeof(Merge<8 * NT, D>);
  constexpr int smem = ring > merge ? ring : merge;
  static_assert(smem <= 232448 - 256, "shared memory");
  static std::atomic<int> occupancy[64];
  return launch_kernel(window_rows_kernel<TQ, KV8, D, NT>, a, c, smem, occupancy, s, p);
}

template <typename TQ, bool KV8>
cudaError_t by_shape(const WindowArgs& a, int nt, const Call& c, cudaStream_t s, const RowsP& p) {
  if (nt == 2) return a.D == 64 ? launch16<TQ, KV8, 64, 2>(a, c, s, p) : launch16<TQ, KV8, 128, 2>(a, c, s, p);
  if (a.D == 64) return launch16<TQ, KV8, 64, 1>(a, c, s, p);
  if (a.D == 128) return launch16<TQ, KV8, 128, 1>(a, c, s, p);
  return launch16<TQ, KV8, 256, 1>(a, c, s, p);
}

template <int D, int HB>
cudaError_t launch32(const WindowArgs& a, const Call& c, cudaStream_t s, const RowsP& p) {
  static std::atomic<int> occupancy[64];
  return launch_kernel(window_rows_f32_kernel<D, HB>, a, c, 0, occupancy, s, p);
}

}  // namespace

cudaError_t launch_window_rows(const WindowArgs& a, cudaStream_t s) {
  RowsP p;
  p.q = a.q;
  p.kc = a.k_cache;
  p.vc = a.v_cache;
  p.cu = a.cu;
  p.kv_lens = a.kv_lens;
  p.tables = a.page_tables;
  p.B = a.B;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.P = a.P;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.window = a.window;
  p.sinks = a.sinks;
  p.tile_min_q = a.tile_min_q;
  p.div = page_div(a.P);
  p.scale_log2 = a.scale * LOG2E;
  p.ks = a.k_scale;
  p.vs = a.v_scale;
  p.out = a.out;
  p.lse = a.lse;
  p.dev_status = a.dev.status;
  const bool f32 = a.kv_dtype == PKV_F32;
  // 16 heads of a KV head are 16 columns, but at head_dim 256 two parts of 8 (registers). Calls
  // with more rows than sequences take 16 columns too, so that more rows of a sequence share its
  // keys (a piece of 8 columns or fewer leaves the second tile's products out)
  const int nt = (p.G > 8 || a.T > a.B) && a.D <= 128 && !f32 ? 2 : 1;
  p.heads = f32 ? (a.D == 256 ? 2 : 4) : p.G < 8 * nt ? p.G : 8 * nt;
  p.parts = (p.G + p.heads - 1) / p.heads;
  p.per = f32 ? 1 : 8 * nt / p.heads;
  p.numbered = p.per;
  p.per_seq = 0;
  int64_t slots;
  if (a.tile_min_q != INT32_MAX) {   // every sequence of this kernel has fewer rows than that
    p.per_seq = (a.tile_min_q - 1 + p.per - 1) / p.per;
    slots = (int64_t)a.B * p.per_seq;
  } else {
    // a call of no more rows than sequences is one of single rows: a number for each row. Where it has a chunk
    // and idle sequences all the same, the chunk's first numbers take `per` rows each and the others none. 400 rows at
    // window 1024 in a call of 512 places, 8 KV heads of 128 with 1 / 2 / 4 heads: 39 / 61 / 110 us, 193 with a row a
    // number. (Pieces of 16 columns there, for 5 to 8 heads: 107 to 159 us in place of 194, but 128 decode rows of
    // 4096 keys 249 -> 250.5, 64 over e4m3 98 -> 131.)
    if (a.T <= a.B) p.numbered = 1;
    slots = p.numbered == 1 ? a.T : (int64_t)a.B + a.T / p.per;
  }
  const int64_t pieces = slots * a.Hkv * p.parts;
  // pieces that have rows: all, or (with the tile kernel) as many as the rows of even sequences make
  int64_t busy = slots;
  if (p.per_seq) {
    const int64_t even = ((int64_t)a.T + (int64_t)a.B * (p.per - 1) / 2) / p.per;
    if (even < busy) busy = even < 1 ? 1 : even;
  }
  Call call{pieces, busy * a.Hkv * p.parts, 0};
  const int64_t cap = (int64_t)a.max_pages * a.P;
  call.keys = (int64_t)a.window + a.sinks < cap ? (int64_t)a.window + a.sinks : cap;
  p.beside = a.tile_min_q != INT32_MAX;
  KernelTimer timer("window_rows", s);
  if (f32) {
    if (a.D == 64) return launch32<64, 4>(a, call, s, p);
    if (a.D == 128) return launch32<128, 4>(a, call, s, p);
    return launch32<256, 2>(a, call, s, p);
  }
  if (a.kv_dtype == PKV_FP8_E4M3)
    return a.dtype == PKV_BF16 ? by_shape<__nv_bfloat16, true>(a, nt, call, s, p) : by_shape<__half, true>(a, nt, call, s, p);
  return a.dtype == PKV_BF16 ? by_shape<__nv_bfloat16, false>(a, nt, call, s, p) : by_shape<__half, false>(a, nt, call, s, p);
}

}  // namespace pkv
