// C-ABI entry points of the latent-attention calls: host-side checks, then the
// launches of pkv_latent_move.cu, pkv_latent_attn.cu and pkv_latent_prefill.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pagedkv.h"
#include "pkv_internal.h"

using namespace pkv;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Strides of rows read or written as 16-byte vectors. TMA strides end below 2^40 bytes.
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 38); }

int check_latent(const pkv_latent_desc* d) {
  if (!d) return PKV_E_NULL;
  if (d->dtype != PKV_F16 && d->dtype != PKV_BF16) return PKV_E_DTYPE;
  if (d->num_pages < 1 || d->page_size < 1) return PKV_E_SHAPE;
  if ((d->latent_dim != 256 && d->latent_dim != 512) || d->rope_dim != 64) return PKV_E_SHAPE;
  if ((int64_t)d->num_pages * d->page_size > INT32_MAX) return PKV_E_SHAPE;
  return PKV_OK;
}

constexpr int32_t MAX_HEADS = 4096;

bool scale_ok(float s) { return s > 0.f && isfinite(s); }

}  // namespace

extern "C" int pkv_latent_append(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t kr_stride,
                                 const void* q_rope, int64_t q_stride_t, int64_t q_stride_h, void* q_out,
                                 int64_t qo_stride_t, int64_t qo_stride_h, int32_t num_q_heads,
                                 const int32_t* positions, const float* cos_sin, int32_t max_pos,
                                 const int64_t* slot_mapping, int32_t num_tokens, void* cache,
                                 const pkv_latent_desc* desc, pkv_stream_t stream) {
  const int st = check_latent(desc);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || max_pos < 1 || !stride_ok(c_stride) || !stride_ok(kr_stride)) return PKV_E_SHAPE;
  if (q_rope && (num_q_heads < 1 || num_q_heads > MAX_HEADS || !stride_ok(q_stride_t) || !stride_ok(q_stride_h) ||
                 !stride_ok(qo_stride_t) || !stride_ok(qo_stride_h)))
    return PKV_E_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!c_kv || !k_rope || !positions || !cos_sin || !slot_mapping || !cache || (!q_rope) != (!q_out))
    return PKV_E_NULL;
  if (!aligned16(c_kv) || !aligned16(k_rope) || !aligned16(q_rope) || !aligned16(q_out) || !aligned16(cache) ||
      ((uintptr_t)cos_sin & 15u) || ((uintptr_t)slot_mapping & 7u) || !aligned4(positions))
    return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  LatentAppendArgs a{};
  a.c = c_kv;
  a.kr = k_rope;
  a.q = q_rope;
  a.c_st = c_stride;
  a.kr_st = kr_stride;
  a.q_st = q_stride_t;
  a.q_sh = q_stride_h;
  a.qo_st = qo_stride_t;
  a.qo_sh = qo_stride_h;
  a.q_out = q_out;
  a.cache = cache;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.slots = slot_mapping;
  a.max_pos = max_pos;
  a.T = num_tokens;
  a.Hq = q_rope ? num_q_heads : 0;
  a.dtype = desc->dtype;
  a.latent_dim = desc->latent_dim;
  a.rope_dim = desc->rope_dim;
  a.pool_slots = (int64_t)desc->num_pages * desc->page_size;
  a.dev_status = dev.status;
  a.num_sms = dev.num_sms;
  const cudaError_t e = launch_latent_append(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "latent_append");
}

extern "C" int pkv_latent_gather(const void* cache, const pkv_latent_desc* desc, const int32_t* page_tables,
                                 int32_t max_pages_per_seq, const int32_t* cu_seqlens_k, int32_t num_seqs,
                                 int32_t total_k, void* out, pkv_stream_t stream) {
  const int st = check_latent(desc);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || total_k < 0) return PKV_E_SHAPE;
  if (total_k > 0 && max_pages_per_seq < 1) return PKV_E_SHAPE;
  if (total_k == 0 || num_seqs == 0) return PKV_OK;
  if (!cache || !page_tables || !cu_seqlens_k || !out) return PKV_E_NULL;
  if (!aligned16(cache) || !aligned16(out) || !aligned4(page_tables) || !aligned4(cu_seqlens_k)) return PKV_E_ALIGN;
  DeviceView dev;
  const int ds = current_device(&dev);
  if (ds != PKV_OK) return ds;
  LatentGatherArgs a{};
  a.cache = cache;
  a.page_tables = page_tables;
  a.cu = cu_seqlens_k;
  a.B = num_seqs;
  a.total = total_k;
  a.max_pages = max_pages_per_seq;
  a.P = desc->page_size;
  a.num_pages = desc->num_pages;
  a.row_vecs = (desc->latent_dim + desc->rope_dim) / 8;
  a.out = out;
  a.dev_status = dev.status;
  a.num_sms = dev.num_sms;
  const cudaError_t e = launch_latent_gather(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "latent_gather");
}

extern "C" size_t pkv_latent_attention_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                                      const pkv_latent_desc* desc) {
  if (check_latent(desc) != PKV_OK || num_seqs < 0 || total_q < 0 || num_q_heads < 1 || num_q_heads > MAX_HEADS)
    return 0;
  return latent_attn_workspace(num_seqs, total_q, num_q_heads, desc->latent_dim);
}

extern "C" int pkv_latent_attention(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                                    const int32_t* page_tables, int32_t num_seqs, int32_t total_q,
                                    int32_t num_q_heads, int32_t max_pages_per_seq, int32_t max_kv_len,
                                    const void* cache, const pkv_latent_desc* desc, float scale, void* out,
                                    float* lse, void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  const int st = check_latent(desc);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || total_q < 0 || num_q_heads < 1 || num_q_heads > MAX_HEADS || max_kv_len < 0 || !scale_ok(scale))
    return PKV_E_SHAPE;
  // packed (token, head) rows and positions are 32-bit numbers
  if ((int64_t)total_q * num_q_heads > INT32_MAX - 256) return PKV_E_SHAPE;
  if (total_q > 0 && max_pages_per_seq < 1) return PKV_E_SHAPE;
  if ((int64_t)max_pages_per_seq * desc->page_size > INT32_MAX - 256) return PKV_E_SHAPE;
  if (total_q == 0 || num_seqs == 0) return PKV_OK;
  if (!q || !cu_seqlens_q || !kv_lens || !page_tables || !cache || !out || !workspace) return PKV_E_NULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(cache) || !aligned4(lse) || !aligned4(cu_seqlens_q) ||
      !aligned4(kv_lens) || !aligned4(page_tables))
    return PKV_E_ALIGN;
  if (((uintptr_t)workspace & 255u) != 0 ||
      workspace_bytes < latent_attn_workspace(num_seqs, total_q, num_q_heads, desc->latent_dim))
    return PKV_E_WORKSPACE;
  LatentAttnArgs a{};
  const int ds = current_device(&a.dev);
  if (ds != PKV_OK) return ds;
  a.q = q;
  a.cache = cache;
  a.cu = cu_seqlens_q;
  a.kv_lens = kv_lens;
  a.page_tables = page_tables;
  a.B = num_seqs;
  a.T = total_q;
  a.H = num_q_heads;
  a.P = desc->page_size;
  a.num_pages = desc->num_pages;
  a.max_pages = max_pages_per_seq;
  a.max_kv_len = max_kv_len;
  a.latent_dim = desc->latent_dim;
  a.dtype = desc->dtype;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.ws = (char*)workspace;
  const cudaError_t e = launch_latent_attn(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "latent_attention");
}

extern "C" size_t pkv_latent_prefill_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_heads) {
  if (num_seqs < 0 || total_q < 0 || num_heads < 1 || num_heads > MAX_HEADS) return 0;
  return latent_prefill_workspace(num_seqs, total_q, num_heads);
}

extern "C" int pkv_latent_prefill(const void* q, const int32_t* cu_seqlens_q, const void* k_nope,
                                  int64_t kn_stride_t, int64_t kn_stride_h, const void* v, int64_t v_stride_t,
                                  int64_t v_stride_h, const void* k_rope, int64_t kr_stride,
                                  const int32_t* cu_seqlens_k, int32_t num_seqs, int32_t total_q, int32_t total_k,
                                  int32_t num_heads, int32_t dtype, float scale, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  if (dtype != PKV_BF16 && dtype != PKV_F16) return PKV_E_DTYPE;
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || num_heads < 1 || num_heads > MAX_HEADS || !scale_ok(scale))
    return PKV_E_SHAPE;
  if (!stride_ok(kn_stride_t) || !stride_ok(kn_stride_h) || !stride_ok(v_stride_t) || !stride_ok(v_stride_h) ||
      !stride_ok(kr_stride))
    return PKV_E_SHAPE;
  if ((int64_t)total_q * num_heads > INT32_MAX - 256 || total_k > INT32_MAX - 256) return PKV_E_SHAPE;
  if (total_q == 0 || num_seqs == 0) return PKV_OK;
  if (total_k == 0) return PKV_E_SHAPE;   // rows without keys
  // a key row per token; a head stride of 0 (one key or value for all heads) is fine
  if (total_k > 1 && (kn_stride_t == 0 || v_stride_t == 0 || kr_stride == 0)) return PKV_E_SHAPE;
  if (!q || !cu_seqlens_q || !k_nope || !v || !k_rope || !cu_seqlens_k || !out || !workspace) return PKV_E_NULL;
  if (!aligned16(q) || !aligned16(k_nope) || !aligned16(v) || !aligned16(k_rope) || !aligned16(out) ||
      !aligned4(lse) || !aligned4(cu_seqlens_q) || !aligned4(cu_seqlens_k))
    return PKV_E_ALIGN;
  if (((uintptr_t)workspace & 255u) != 0 ||
      workspace_bytes < latent_prefill_workspace(num_seqs, total_q, num_heads))
    return PKV_E_WORKSPACE;
  LatentPrefillArgs a{};
  const int ds = current_device(&a.dev);
  if (ds != PKV_OK) return ds;
  a.q = q;
  a.kn = k_nope;
  a.v = v;
  a.kr = k_rope;
  a.kn_st = kn_stride_t;
  a.kn_sh = kn_stride_h;
  a.v_st = v_stride_t;
  a.v_sh = v_stride_h;
  a.kr_st = kr_stride;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.B = num_seqs;
  a.Tq = total_q;
  a.Tk = total_k;
  a.H = num_heads;
  a.dtype = dtype;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.ws = (char*)workspace;
  const cudaError_t e = launch_latent_prefill(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "latent_prefill");
}
