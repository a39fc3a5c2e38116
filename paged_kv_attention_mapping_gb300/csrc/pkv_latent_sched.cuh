// The absorbed latent-attention kernels' common ground: the call's arguments, the
// tiles of a tick, and their split into equal runs of steps, one per worker (a
// pair of CTAs, or a CTA).
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

// gather: rows come by 16-byte copies of threads (box is 1), not by TMA boxes. A
// TMA instruction costs its warp about 90 cycles whatever its box holds, so small
// boxes (pages that share no large power of two with a slot) starve the tensor cores.
// whole: no tile is cut, so that nothing is left to join. The split counts tiles, not steps.
struct LatentAttnP {
  const int32_t *cu, *kv_lens, *page_tables;
  const void* cache;
  int32_t B, T, H, P, box, gather, whole, num_pages, max_pages, max_kv_len, table_cap, out_32;
  float scale_log2;   // > 0
  void* out;
  float* lse;
  char* ws;
  int32_t* dev_status;
};

// The kernel for few rows a sequence (pkv_latent_rows.cu): rows of its ring slots,
// its tiling, its workspace, its launch.
int latent_rows_slot();
struct LatentTiling {
  int rows, keys, workers;   // of a tile, of a step, of the GPU
};
LatentTiling latent_rows_tiling(int num_sms);
size_t latent_rows_workspace(int latent_dim);
cudaError_t launch_latent_rows(const LatentAttnArgs& a, const LatentAttnP& p, cudaStream_t s);

// A run of steps [j0, j1) of one tile.
struct LatentSegment {
  int valid, b, L, base;      // base: keys before the sequence's first new token
  int row0, frow0, nrows;     // first packed row, first row within the sequence, rows
  int j0, j1, n;              // n: steps of the whole tile
};

// The tile that a worker's run cuts at its end: its first worker, and how many
// workers share it. nrows 0: no cut tile.
struct LatentRecord {
  int32_t parts, row0, nrows, owner;
};

// One sequence's tiles. Tile t covers rows [TM t, TM t + TM) of its q_len * H
// and needs the keys up to its last row's position, BN of them a step. In the split
// a tile counts START units, for its queries' loading and its results' storing, then one
// a step: workers with many short tiles get fewer steps. A place in a tile is an
// offset in units; one in the first START of them stands before its first step.
template <int TM, int BN, int START>
struct LatentSeq {
  int q, L, base, H, rows, tiles, whole;
  __device__ __forceinline__ int steps(int t) const {
    const int last = (min((t + 1) * TM, rows) - 1) / H;
    return (base + last + BN) / BN;
  }
  // tiles with at most v steps (steps() never falls from one tile to the next)
  __device__ __forceinline__ int tiles_within(int v) const {
    const int64_t e = (int64_t)v * BN - base;   // tokens that see at most v * BN keys
    if (e >= q) return tiles;
    if (e <= 0) return 0;
    return min(tiles - 1, (int)(e * H / TM));
  }
  __device__ __forceinline__ int64_t total() const {
    if (tiles == 0 || whole) return tiles;
    if (tiles == 1) return (L + BN - 1) / BN + START;
    const int lo = steps(0), hi = steps(tiles - 1);
    int64_t s = (int64_t)(hi + START) * tiles;
    for (int v = lo; v < hi; ++v) s -= tiles_within(v);
    return s;
  }
  // tile, and offset in it, of the sequence's unit number `at`
  __device__ __forceinline__ void seek(int64_t at, int* tile, int* off) const {
    if (tiles == 1 || whole) {
      *tile = whole ? (int)at : 0;
      *off = whole ? 0 : (int)at;
      return;
    }
    const int lo = steps(0), hi = steps(tiles - 1);
    int before = 0;
    for (int v = lo; v <= hi; ++v) {
      const int upto = v == hi ? tiles : tiles_within(v);
      const int64_t s = (int64_t)(upto - before) * (v + START);
      if (at < s) {
        *tile = before + (int)(at / (v + START));
        *off = (int)(at % (v + START));
        return;
      }
      at -= s;
      before = upto;
    }
  }
  // Sequence b; one with bad lengths has no tiles.
  __device__ __forceinline__ void load(const LatentAttnP& p, int b, bool report) {
    const int c0 = __ldg(p.cu + b);
    q = __ldg(p.cu + b + 1) - c0;
    L = __ldg(p.kv_lens + b);
    H = p.H;
    whole = p.whole;
    base = L - q;
    rows = q * H;
    tiles = (rows + TM - 1) / TM;
    if (q > 0 && (L < q || L > p.max_kv_len || L > p.table_cap)) {
      if (report) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
      tiles = 0;
    }
    if (q <= 0 || q > p.T) tiles = 0;
  }
};

// The segment of a run with `left` units to go that begins at offset `off` of a tile; not
// valid if the run ends before the tile's first step (then the run has no more segments).
template <int TM, int BN, int START>
__device__ __forceinline__ LatentSegment latent_segment(const LatentAttnP& p, const LatentSeq<TM, BN, START>& s, int b,
                                                        int tile, int off, int64_t left) {
  LatentSegment g;
  g.b = b;
  g.L = s.L;
  g.base = s.base;
  g.frow0 = tile * TM;
  g.row0 = __ldg(p.cu + b) * p.H + tile * TM;
  g.nrows = min(TM, s.rows - tile * TM);
  g.n = s.steps(tile);
  g.j0 = max(0, off - START);
  g.j1 = p.whole ? g.n : (int)min((int64_t)g.n, off - START + left);
  g.valid = g.j0 < g.j1;
  return g;
}

// Where a worker's run starts, in shared memory.
template <int NTHREADS>
struct LatentPlan {
  int64_t scan[NTHREADS / 32];
  int64_t run, each;   // units of this worker's run, and of every worker's but the last
  int b, tile, off;
};

// By all threads of a CTA, after the wait for the kernel before, which may have written
// the lengths: every CTA counts the whole tick's units and finds where its own run starts,
// and LatentRun reads the same lengths again. One thread has set pl->run and first->valid to 0 before; the results,
// the run's first segment among them, are visible after the caller's next block barrier.
template <int TM, int BN, int START, int NTHREADS>
__device__ __forceinline__ void latent_plan(const LatentAttnP& p, int worker, int workers, LatentPlan<NTHREADS>* pl,
                                            LatentSegment* first) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = tid == 0 && __ldg(p.cu) != 0;
  const int per = (p.B + NTHREADS - 1) / NTHREADS;
  const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
  int64_t mine = 0;
  LatentSeq<TM, BN, START> s;
  for (int b = b_lo; b < b_hi; ++b) {
    s.load(p, b, blockIdx.x == 0);
    bad |= s.q < 0;
    mine += s.total();
  }
  bad |= __ldg(p.cu + p.B) > p.T;
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += y;
  }
  if (lane == 31) pl->scan[warp] = scan;
  bad = __syncthreads_or(bad);
  int64_t total = 0, before = scan - mine;
#pragma unroll
  for (int w = 0; w < NTHREADS / 32; ++w) {
    if (w < warp) before += pl->scan[w];
    total += pl->scan[w];
  }
  if (bad) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.dev_status, PKV_DEV_BAD_LENGTHS);
    total = 0;
  }
  const int64_t each = (total + workers - 1) / workers;
  const int64_t lo = worker * each, hi = min(lo + each, total);
  if (lo < hi && lo >= before && lo < before + mine) {
    int64_t at = lo - before;
    for (int b = b_lo; b < b_hi; ++b) {
      s.load(p, b, false);
      const int64_t n = s.total();
      if (at < n) {
        int tile, off;
        s.seek(at, &tile, &off);
        pl->b = b;
        pl->tile = tile;
        pl->off = off;
        const LatentSegment g = latent_segment(p, s, b, tile, off, hi - lo);
        prefetch_l2(p.page_tables + (int64_t)b * p.max_pages + (int64_t)g.j0 * BN / p.P);   // wanted first
        *first = g;
        break;
      }
      at -= n;
    }
    pl->run = hi - lo;
  }
  if (tid == 0) pl->each = each;
}

// A worker's segments, one after the other, and the record of the tile that its
// run cuts at the end.
template <int TM, int BN, int START>
struct LatentRun {
  int64_t left, done, each;
  int worker, b, tile, off;
  LatentSeq<TM, BN, START> s;
  LatentRecord r;
  template <int NTHREADS>
  __device__ __forceinline__ LatentRun(const LatentAttnP& p, const LatentPlan<NTHREADS>& pl, int w) {
    left = pl.run;
    done = 0;
    each = pl.each;
    worker = w;
    b = tile = off = 0;
    s.tiles = 0;
    r = LatentRecord{0, 0, 0, 0};
    if (left > 0) {
      b = pl.b;
      tile = pl.tile;
      off = pl.off;
      s.load(p, b, false);
    }
  }
  __device__ __forceinline__ LatentSegment next(const LatentAttnP& p) {
    LatentSegment g;
    g.valid = 0;
    if (left <= 0) return g;
    // left > 0 promises one more tile, as long as nobody rewrites the lengths meanwhile
    while (tile >= s.tiles && ++b < p.B) {
      s.load(p, b, false);
      tile = 0;
    }
    if (tile >= s.tiles) return g;
    g = latent_segment(p, s, b, tile, off, left);
    if (!g.valid) return g;
    if (g.j1 < g.n) {
      // the tile's first step among the tick's units (this run starts at worker * each)
      const int64_t begin = worker * each + done - off + START;
      r.owner = (int)(begin / each);
      r.parts = (int)((begin + g.n - 1) / each) - r.owner + 1;
      r.row0 = g.row0;
      r.nrows = g.nrows;
    }
    const int used = p.whole ? 1 : g.j1 + START - off;
    left -= used;
    done += used;
    ++tile;
    off = 0;
    return g;
  }
};

}  // namespace pkv
