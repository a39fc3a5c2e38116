// C-ABI entry points of the windowed layers' calls: host-side checks, then the launches of
// pkv_norm_rope.cu, pkv_window_rows.cu, pkv_window_tiles.cu and pkv_pages.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pagedkv.h"
#include "pkv_internal.h"

using namespace pkv;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int elt_bytes(int dtype) { return dtype == PKV_F32 ? 4 : dtype == PKV_FP8_E4M3 ? 1 : 2; }
bool source_type(int dtype) { return dtype == PKV_F32 || dtype == PKV_F16 || dtype == PKV_BF16; }

// Strides of rows read or written as 16-byte vectors; the bound keeps a token's offset within 64 bits.
bool stride_ok(int64_t s, int elt) { return s >= 0 && (s * elt) % 16 == 0 && s < ((int64_t)1 << 31); }

constexpr int32_t MAX_HEADS = 4096;

// Sequences with this many new rows or more run on the tile kernel, which takes all their rows in one
// pass over the keys but does not split them; the row kernel splits keys over CTAs and reads them
// again for every 16 columns (rows x heads of a KV head). So the rule counts columns. Row / tile kernel,
// 8 KV heads of 128 in bf16, B sequences, windows of 512 and 4096 (columns alone matter: 1 to 16
// heads of a KV head give the same figures):
//   16 columns  B = 10 15 / 16 us and 47 / 57 (row)   B = 48 42 / 43 and 204 / 159 (tile at the larger)
//   24 columns  B = 6 15 / 16 and 46 / 56 (row)       B = 10 20 / 16 and 104 / 58 (tile)
//   40 columns  B = 6 20 / 16 and 103 / 57 (tile)     B = 48 74 / 43 and 396 / 160 (tile)
// Tiles for fewer than half the SMs leave the larger part idle: 16 columns more. Keys of 64 channels
// cost a row pass half as much and a tile about as much (24 columns, B = 48: 31 / 38 and 152 / 141; 40
// columns: 37 / 38 and 183 / 141; B = 6: 12 / 14 and 40 / 51). So do e4m3 keys, which a tile has to widen (32
// columns, B = 48: 44 / 72 and 207 / 207; 48: 60 / 73 and 290 / 208; 64: 77 / 73 and 383 / 207).
int32_t tile_rows(bool codes, int32_t D, int32_t group, int64_t tiles, int num_sms) {
  const int32_t columns = codes ? 48 : (D == 128 ? 16 : 32) + (2 * tiles < num_sms ? 16 : 0);
  return columns / group + 1;
}

// Whether the row kernel may be left out of a call with chunks, so that its short sequences become work tiles too. A
// row kernel that finds nothing to do costs a call 1 to 5 us (7 prompts, 28 / 4 heads of 128, window 512: 95.6 us
// without / 100.8 with; 16 prompts of 600, 32 / 8 heads: 77 / 81; one of 512 rows: 14.5 / 16.1). A short sequence costs the
// tile kernel a work tile for each KV head, whose keys one CTA walks. So both have to be few, work tiles that short
// sequences may add and steps that one takes (without / with the row kernel, in us):
//   1 row of 8000 keys beside a prompt of 600      W = 512 16.8 / 17.8   1024 19.5 / 17.5   4096 52 / 18
//   3 rows beside one of 4000                      W = 512 56 / 60       1024 82 / 78       4096 159 / 136
//   12 rows beside one of 8192                     W = 512 110 / 109     1024 156 / 152     4096 386 / 362
//   8 rows beside one of 8192, 8 heads of 8        W = 128 32.4 / 31.9   512 47 / 43        4096 162 / 143
// A call of one sequence has nothing beside it.
constexpr int64_t FEW_KEYS = 768, TILES_A_SEQUENCE = 8;
bool tiles_only(int32_t num_seqs, int32_t total_q, int32_t group, int64_t keys) {
  return num_seqs == 1 || (keys <= FEW_KEYS && total_q / (2 * (128 / group)) >= TILES_A_SEQUENCE * num_seqs);
}

// head_dim and dtypes that the calls of this file share
int check(const pkv_cache_desc* c, int32_t src_dtype, const float* k_scale, const float* v_scale) {
  if (!c) return PKV_E_NULL;
  if (c->dtype < PKV_F32 || c->dtype > PKV_FP8_E4M3 || !source_type(src_dtype)) return PKV_E_DTYPE;
  const bool codes = c->dtype == PKV_FP8_E4M3;
  if (!codes && c->dtype != src_dtype) return PKV_E_DTYPE;
  if (c->num_pages < 1 || c->page_size < 1 || c->num_kv_heads < 1 || c->num_kv_heads > MAX_HEADS) return PKV_E_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return PKV_E_SHAPE;
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX) return PKV_E_SHAPE;
  if (codes && (!k_scale || !v_scale)) return PKV_E_NULL;
  if (!codes && (k_scale || v_scale)) return PKV_E_DTYPE;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return PKV_E_ALIGN;
  return PKV_OK;
}

}  // namespace

extern "C" int pkv_norm_rope_kv_append(const pkv_norm_rope_args* args, pkv_stream_t stream) {
  if (!args) return PKV_E_NULL;
  const pkv_norm_rope_args& g = *args;
  const pkv_cache_desc& cache = g.cache;
  const int st = check(&cache, g.src_dtype, g.k_scale, g.v_scale);
  if (st != PKV_OK) return st;
  if (g.num_tokens < 0 || g.num_q_heads < 1 || g.num_q_heads > MAX_HEADS || g.max_pos < 1) return PKV_E_SHAPE;
  if (g.rotary_dim < 16 || g.rotary_dim % 16 != 0 || g.rotary_dim > cache.head_dim) return PKV_E_SHAPE;
  if (!(g.eps >= 0.f) || !isfinite(g.eps)) return PKV_E_SHAPE;
  const int elt = elt_bytes(g.src_dtype);
  const int64_t strides[] = {g.q_stride_t, g.q_stride_h, g.k_stride_t,  g.k_stride_h,
                             g.v_stride_t, g.v_stride_h, g.qo_stride_t, g.qo_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s, elt)) return PKV_E_SHAPE;
  if (g.num_tokens == 0) return PKV_OK;
  if (!g.q || !g.k || !g.v || !g.positions || !g.cos_sin || !g.slot_mapping || !g.k_cache || !g.v_cache || !g.q_out)
    return PKV_E_NULL;
  if (!aligned(g.q, 16) || !aligned(g.k, 16) || !aligned(g.v, 16) || !aligned(g.q_out, 16) || !aligned(g.k_cache, 16) ||
      !aligned(g.v_cache, 16) || !aligned(g.q_weight, 16) || !aligned(g.k_weight, 16) || !aligned(g.cos_sin, 16) ||
      !aligned(g.slot_mapping, 8) || !aligned(g.positions, 4))
    return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  NormRopeArgs a{};
  a.q = g.q;
  a.k = g.k;
  a.v = g.v;
  a.q_weight = g.q_weight;
  a.k_weight = g.k_weight;
  a.q_st = g.q_stride_t;
  a.q_sh = g.q_stride_h;
  a.k_st = g.k_stride_t;
  a.k_sh = g.k_stride_h;
  a.v_st = g.v_stride_t;
  a.v_sh = g.v_stride_h;
  a.qo_st = g.qo_stride_t;
  a.qo_sh = g.qo_stride_h;
  a.pool_slots = (int64_t)cache.num_pages * cache.page_size;
  a.eps = g.eps;
  a.positions = g.positions;
  a.cos_sin = g.cos_sin;
  a.slots = g.slot_mapping;
  a.max_pos = g.max_pos;
  a.rot = g.rotary_dim;
  a.interleaved = g.interleaved != 0;
  a.T = g.num_tokens;
  a.Hq = g.num_q_heads;
  a.Hkv = cache.num_kv_heads;
  a.D = cache.head_dim;
  a.dtype = g.src_dtype;
  a.kc = g.k_cache;
  a.vc = g.v_cache;
  a.q_out = g.q_out;
  a.k_scale = g.k_scale;
  a.v_scale = g.v_scale;
  a.dev_status = dev.status;
  const cudaError_t e = launch_norm_rope(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "norm_rope_kv_append");
}

extern "C" int pkv_window_attention(const void* q, int32_t q_dtype, const int32_t* cu_seqlens_q,
                                    const int32_t* kv_lens, const int32_t* page_tables, int32_t num_seqs,
                                    int32_t total_q, int32_t num_q_heads, int32_t max_pages_per_seq, int32_t window,
                                    int32_t sinks, const void* k_cache, const void* v_cache,
                                    const pkv_cache_desc* cache, const float* k_scale, const float* v_scale,
                                    float scale, void* out, float* lse, pkv_stream_t stream) {
  const int st = check(cache, q_dtype, k_scale, v_scale);
  if (st != PKV_OK) return st;
  const bool codes = cache->dtype == PKV_FP8_E4M3;
  if (codes && q_dtype == PKV_F32) return PKV_E_DTYPE;
  if (num_seqs < 0 || total_q < 0 || num_q_heads < 1 || num_q_heads > MAX_HEADS) return PKV_E_SHAPE;
  if (window < 1 || sinks < 0 || !(scale > 0.f) || !isfinite(scale)) return PKV_E_SHAPE;
  if (num_q_heads % cache->num_kv_heads != 0) return PKV_E_SHAPE;
  const int g = num_q_heads / cache->num_kv_heads;
  if (g > 8 && g != 16) return PKV_E_SHAPE;
  if (total_q > 0 && num_seqs > 0 && max_pages_per_seq < 1) return PKV_E_SHAPE;
  // (positions a few steps past the last key stay within 32 bits)
  if ((int64_t)max_pages_per_seq * cache->page_size > INT32_MAX - 65535) return PKV_E_SHAPE;
  if (total_q == 0 || num_seqs == 0) return PKV_OK;
  if (!q || !cu_seqlens_q || !kv_lens || !page_tables || !k_cache || !v_cache || !out) return PKV_E_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(cu_seqlens_q, 4) || !aligned(kv_lens, 4) || !aligned(page_tables, 4) || !aligned(lse, 4))
    return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  WindowArgs a{};
  a.q = q;
  a.cu = cu_seqlens_q;
  a.kv_lens = kv_lens;
  a.page_tables = page_tables;
  a.B = num_seqs;
  a.T = total_q;
  a.Hq = num_q_heads;
  a.Hkv = cache->num_kv_heads;
  a.D = cache->head_dim;
  a.P = cache->page_size;
  a.num_pages = cache->num_pages;
  a.max_pages = max_pages_per_seq;
  a.window = window;
  a.sinks = sinks;
  a.dtype = q_dtype;
  a.kv_dtype = cache->dtype;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.dev = dev;
  a.tile_min_q = INT32_MAX;
  // a call of no more rows than sequences is one of single rows (were it not, the row kernel
  // takes its chunks too)
  const int32_t many = tile_rows(codes, cache->head_dim, g, (int64_t)num_seqs * cache->num_kv_heads, dev.num_sms);
  // the most that a row sees
  const int64_t context = (int64_t)max_pages_per_seq * cache->page_size, seen = (int64_t)window + sinks;
  const int64_t keys = seen < context ? seen : context;
  if (total_q > num_seqs && total_q >= many && window_tiles_supported(cache->dtype, cache->head_dim, cache->page_size))
    a.tile_min_q = tiles_only(num_seqs, total_q, g, keys) ? 1 : many;
  cudaError_t e = cudaSuccess;
  if (a.tile_min_q != INT32_MAX) e = launch_window_tiles(a, (cudaStream_t)stream);
  if (e == cudaSuccess && a.tile_min_q > 1) e = launch_window_rows(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "window_attention");
}

extern "C" int pkv_copy_pages(void* const* caches, int32_t num_caches, int32_t num_pages, int32_t page_size,
                              int64_t slot_bytes, const int32_t* src, const int32_t* dst, const int32_t* tokens,
                              int32_t num_copies, pkv_stream_t stream) {
  if (num_caches < 0 || num_copies < 0 || num_pages < 1 || page_size < 1) return PKV_E_SHAPE;
  if (slot_bytes < 16 || slot_bytes % 16 != 0 || slot_bytes > INT32_MAX) return PKV_E_SHAPE;
  if ((int64_t)num_pages * page_size > INT32_MAX || page_size * slot_bytes > INT32_MAX) return PKV_E_SHAPE;
  if (num_caches == 0 || num_copies == 0) return PKV_OK;
  if (!caches || !src || !dst) return PKV_E_NULL;
  for (int32_t c = 0; c < num_caches; ++c) {
    if (!caches[c]) return PKV_E_NULL;
    if (!aligned(caches[c], 16)) return PKV_E_ALIGN;
  }
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(tokens, 4)) return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  CopyPagesArgs a{};
  a.caches = caches;
  a.num_caches = num_caches;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.num_copies = num_copies;
  a.slot_bytes = slot_bytes;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.dev_status = dev.status;
  const cudaError_t e = launch_copy_pages(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "copy_pages");
}

extern "C" int pkv_remap_pages(int32_t* page_tables, int64_t num_entries, const int32_t* page_map,
                               int32_t num_pages, pkv_stream_t stream) {
  if (num_entries < 0 || num_pages < 1) return PKV_E_SHAPE;
  if (num_entries == 0) return PKV_OK;
  if (!page_tables || !page_map) return PKV_E_NULL;
  if (!aligned(page_tables, 4) || !aligned(page_map, 4)) return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  const cudaError_t e = launch_remap_pages(page_tables, num_entries, page_map, num_pages, dev, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "remap_pages");
}
