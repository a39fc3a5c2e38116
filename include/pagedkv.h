/*
 * pagedkv.h — C ABI of libpagedkv: attention over a paged KV cache for one
 * packed, continuously batched tick of decode tokens and chunked-prefill
 * tokens with grouped-query heads, on an NVIDIA GB300 (sm_103a).
 *
 * The operations follow the serving pages' description of the problem:
 *  - the KV cache is a fixed pool of fixed-size pages shared by all sequences,
 *    one tensor per layer for K and one for V, each laid out
 *    [num_pages, page_size, num_kv_heads, head_dim] (llm-serving-engine README,
 *    component table "KV Cache" row and "KV cache memory layout" figure;
 *    Helios README, "Paged attention": a fixed pool of 256-token pages);
 *  - each sequence owns a page table that maps its positions to pages
 *    (mini-vLLM, "Paged KV-cache"; Helios README, "Paged attention");
 *  - new tokens' K/V are written into their slots first, then attention reads
 *    K/V through the page tables, never copying them into dense per-sequence
 *    buffers (Helios README, "Paged attention" and its closing remark on
 *    causal paged attention on NVIDIA GPUs; Helios blog, "Prefill vs Decode");
 *  - decode tokens and prefill chunks run in one packed pass with independent
 *    positions and page tables, decode tokens first (Helios README,
 *    "Continuous batching"; Helios blog, "Continuous batching").
 *
 * Conventions shared by every call:
 *  - Ownership: the caller allocates and owns every buffer, host or device,
 *    including the attention workspace. The library allocates no device memory
 *    and keeps no per-call state. It does hold, per process, a device status
 *    word (see pkv_get_device_status) and, when enabled, CUDA events for
 *    kernel timing.
 *  - Asynchrony: device calls are enqueued on `stream` (a cudaStream_t; NULL =
 *    the legacy default stream) and return before the work runs. Outputs are
 *    valid once the stream has been synchronised.
 *  - Errors: every call returns PKV_OK (0) or a negative PKV_E_* code. Host
 *    checks run before anything is enqueued; on an error nothing is launched.
 *    Data-dependent checks that only the device can make (a slot or page id
 *    outside the pool, a kv_len longer than its page table) set bits of the
 *    device status word and skip the offending row; nothing traps or aborts.
 *  - Dtypes: K, V, Q and the attention output share one dtype (PKV_F32,
 *    PKV_F16 or PKV_BF16); accumulation is fp32; lse is fp32.
 */
#ifndef PAGEDKV_H_
#define PAGEDKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pkv_stream_t; /* same handle as cudaStream_t */

typedef enum {
  PKV_F32 = 0,
  PKV_F16 = 1,
  PKV_BF16 = 2,
  PKV_FP8_E4M3 = 3 /* caches only, with per-KV-head scales (pkv_kv_append_quant,
                      pkv_paged_attention_fp8) */
} pkv_dtype;

typedef enum {
  PKV_OK = 0,
  PKV_E_NULL = -1,      /* a required pointer is NULL */
  PKV_E_DTYPE = -2,     /* unknown dtype */
  PKV_E_SHAPE = -3,     /* a size is out of range, Hq % Hkv != 0, or head_dim unsupported */
  PKV_E_LENGTHS = -4,   /* q/kv lengths break 0 <= q_len <= kv_len (host-checked calls) */
  PKV_E_PAGES = -5,     /* a page id outside the pool, or too few pages for a length */
  PKV_E_WORKSPACE = -6, /* workspace smaller than pkv_paged_attention_workspace_size */
  PKV_E_ALIGN = -7,     /* a pointer is not 16-byte aligned */
  PKV_E_CUDA = -8,      /* a CUDA runtime call or launch failed */
  PKV_E_DEVICE = -9,    /* the current device is not an sm_103 GPU */
  PKV_E_CAPACITY = -10  /* an output buffer is too small (host-checked calls) */
} pkv_status;

/* Bits of the device status word. */
#define PKV_DEV_BAD_SLOT 0x1    /* kv_append: slot >= num_pages * page_size; that row skipped */
#define PKV_DEV_BAD_LENGTHS 0x2 /* attention: kv_len < q_len, kv_len < 1 with rows,
                                   kv_len > max_kv_len or > max_pages_per_seq * page_size:
                                   that sequence's rows are skipped; cu_seqlens_q not
                                   non-decreasing from 0 to total_q (some q_len < 0):
                                   every row of the call is skipped */
#define PKV_DEV_BAD_PAGE 0x4    /* attention: a page id needed by a row is outside the pool;
                                   that row's output is left unwritten */
#define PKV_DEV_TIMEOUT 0x8     /* a kernel's internal wait gave up (a bug, never expected);
                                   the outputs of that call are unspecified */
#define PKV_DEV_BAD_POSITION 0x10 /* rope and latent append: a position outside [0, max_pos); that row skipped */

/* One layer's K (or V) page pool: contiguous
 * [num_pages, page_size, num_kv_heads, head_dim] of `dtype`. */
typedef struct {
  int32_t num_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype; /* pkv_dtype */
} pkv_cache_desc;

/* ---------------------------------------------------------------------------
 * pkv_pack_tick — host-side packing of one tick (no device work).
 *
 * Puts decode sequences (q_len == 1) first and then the others, each group in
 * arrival order (Helios README, "Continuous batching": every tick first takes
 * one token per decoding request, then spends the rest of the budget on
 * prompts; both run in one packed forward), and builds the packed metadata.
 *
 * In (host pointers, num_seqs entries unless stated):
 *   q_lens[i]        tokens sequence i adds this tick (0 = idle, 1 = decode, >1 = chunk)
 *   kv_lens[i]       context length after this tick's tokens are written
 *   page_offsets     [num_seqs + 1], CSR offsets into page_ids
 *   page_ids         physical pages of sequence i in logical order:
 *                    page_ids[page_offsets[i] .. page_offsets[i+1])
 *   page_size, num_pages, max_pages_per_seq (width of the output table)
 *   slot_capacity    length of the slot_mapping buffer
 * Out (host pointers, caller-allocated):
 *   order[num_seqs]                   arrival index of the i-th packed sequence
 *   cu_seqlens_q[num_seqs + 1]        row offsets of the packed sequences
 *   kv_lens_out[num_seqs]             kv_len of the i-th packed sequence
 *   page_tables[num_seqs * max_pages_per_seq]  row-major, unused entries -1
 *   slot_mapping[total_q]             page * page_size + offset of each packed
 *                                     row's new token (its position is
 *                                     kv_len - q_len + i for chunk row i)
 *   total_q_out                       number of packed rows
 * Errors: PKV_E_NULL, PKV_E_SHAPE (num_seqs < 0, page_size < 1, num_pages < 1,
 * max_pages_per_seq < 1), PKV_E_LENGTHS (q_len < 0, kv_len < q_len, kv_len < 1
 * with q_len > 0), PKV_E_PAGES (page id outside [0, num_pages), fewer pages
 * than ceil(kv_len / page_size), more pages than max_pages_per_seq),
 * PKV_E_CAPACITY (total_q > slot_capacity). Outputs are unspecified on error.
 */
int pkv_pack_tick(int32_t num_seqs, const int32_t* q_lens, const int32_t* kv_lens,
                  const int32_t* page_offsets, const int32_t* page_ids,
                  int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                  int32_t slot_capacity,
                  int32_t* order, int32_t* cu_seqlens_q, int32_t* kv_lens_out,
                  int32_t* page_tables, int64_t* slot_mapping, int32_t* total_q_out);

/* pkv_tick_positions — host: position of every packed row (kv_len - q_len + i
 * for row i of a sequence), from cu_seqlens_q[num_seqs + 1] and kv_lens
 * (host pointers), into positions[capacity]. PKV_E_LENGTHS for q_len < 0,
 * kv_len < q_len or cu[0] != 0; PKV_E_CAPACITY if the rows do not fit. */
int pkv_tick_positions(int32_t num_seqs, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                       int32_t* positions, int32_t capacity);

/* ---------------------------------------------------------------------------
 * pkv_kv_append — write each new token's K and V rows into its slot
 * (Helios blog, "Prefill vs Decode": a decode step writes its new token's
 * slot; Helios README, "Paged attention": decode stores straight into the
 * shared pool; llm-serving-engine README, engine step trace: a prefill chunk
 * stores its K/V starting at the chunk's first position).
 *
 *   k, v          device, [num_tokens, num_kv_heads, head_dim], contiguous, cache dtype
 *   slot_mapping  device, int64 [num_tokens]; row t goes to page slot / page_size,
 *                 offset slot % page_size; a negative slot skips the row
 *   k_cache, v_cache  device, the pools described by `cache`
 * Bit-exact copy. Duplicate non-negative slots in one call are a caller error
 * (which row lands is unspecified). A slot >= num_pages * page_size sets
 * PKV_DEV_BAD_SLOT and skips the row. num_tokens == 0 is a no-op.
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE, PKV_E_ALIGN (k, v, caches must
 * be 16-byte aligned), PKV_E_CUDA.
 */
int pkv_kv_append(const void* k, const void* v, const int64_t* slot_mapping, int32_t num_tokens,
                  void* k_cache, void* v_cache, const pkv_cache_desc* cache, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * Rotary position embedding fused into the append (Helios blog, "torch.sdpa
 * and Flash Attention": RoPE is applied to Q and K before attention;
 * llm-serving-engine README, component table "RoPE from scratch": cached
 * sin/cos tables). Half-split form: for pair i < d/2 of a head row x at
 * position p, with a = p * base^(-2i/d),
 *   x'_i = x_i cos a - x_{i+d/2} sin a,   x'_{i+d/2} = x_{i+d/2} cos a + x_i sin a.
 *
 * pkv_rope_table (host): fills cos_sin[max_pos][head_dim/2][2] (float) with
 * (cos a, sin a), computed in double. PKV_E_SHAPE unless base > 1, head_dim
 * even >= 2, max_pos >= 1.
 *
 * pkv_rope_kv_append (device): for each new token t at position positions[t]
 * (int32, device), rotates its K rows and writes them to slot slot_mapping[t]
 * (as pkv_kv_append; a negative slot skips K and V), copies its V rows to the
 * slot unrotated, and writes its rotated Q rows [num_tokens, num_q_heads,
 * head_dim] to q_out (q_out may equal q: in place). cos_sin is the device copy
 * of the table above. A position outside [0, max_pos) sets
 * PKV_DEV_BAD_POSITION and skips that token's Q and K rows. Rotation in fp32,
 * results rounded to the cache dtype. Errors as pkv_kv_append, plus PKV_E_SHAPE
 * for an odd head_dim or num_q_heads < 1.
 */
int pkv_rope_table(double base, int32_t head_dim, int32_t max_pos, float* cos_sin);
int pkv_rope_kv_append(const void* q, const void* k, const void* v, const int32_t* positions,
                       const float* cos_sin, int32_t max_pos, const int64_t* slot_mapping, int32_t num_tokens,
                       int32_t num_q_heads, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                       void* q_out, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * pkv_paged_attention_workspace_size — bytes of device workspace that
 * pkv_paged_attention needs for these sizes (0 on invalid sizes).
 * The workspace holds the device-side work plan and the split-KV partial
 * results; its contents need no initialisation and are not preserved.
 */
size_t pkv_paged_attention_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                          const pkv_cache_desc* cache, int32_t max_kv_len);

/* ---------------------------------------------------------------------------
 * pkv_paged_attention — attention of every packed query row over its
 * sequence's pages (Helios blog, "torch.sdpa and Flash Attention":
 * softmax(Q K^T * scale) V with grouped-query heads sharing KV heads;
 * llm-serving-engine README, engine step trace: a prefill chunk after cached
 * K/V uses a rectangular causal mask, a decode row attends the full context).
 *
 *   q             device, [total_q, num_q_heads, head_dim], cache dtype, contiguous
 *   cu_seqlens_q  device, int32 [num_seqs + 1]; cu[0] = 0, non-decreasing, cu[num_seqs] = total_q
 *   kv_lens       device, int32 [num_seqs]; context length INCLUDING this tick's
 *                 tokens (append first, then attend)
 *   page_tables   device, int32 [num_seqs, max_pages_per_seq], row-major
 *   max_kv_len    host upper bound on every kv_lens entry (sizes the work plan)
 *   scale         multiplies q.k before the softmax
 *   out           device, [total_q, num_q_heads, head_dim], cache dtype
 *   lse           device, fp32 [total_q, num_q_heads], natural log of
 *                 sum_j exp(scale * q.k_j); may be NULL
 *   workspace     device, >= pkv_paged_attention_workspace_size(...) bytes, 256-byte aligned
 * Row i of sequence b (q_len = cu[b+1] - cu[b], kv_len = kv_lens[b]) attends
 * keys 0 .. kv_len - q_len + i. q head h reads KV head h / (num_q_heads /
 * num_kv_heads). Page-table entries past ceil(kv_len / page_size) and slots at
 * positions >= kv_len are never read and may hold anything (NaN, -1).
 * Rows of sequences with bad lengths or pages (see the device status bits)
 * are skipped.
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE (num_q_heads % num_kv_heads != 0,
 * a group num_q_heads / num_kv_heads outside 1..8 and 16, head_dim not 64,
 * 128 or 256, sizes < 0), PKV_E_ALIGN, PKV_E_WORKSPACE, PKV_E_DEVICE, PKV_E_CUDA.
 * head_dim 64 and 128 run decode rows on the TMA-staged decode kernel and
 * chunks on the tensor-core prefill kernels; at head_dim 256 every row (decode
 * and chunk) runs on the TMA-staged decode kernel over 16-bit caches and on the
 * CUDA-core rows kernel over fp32 caches.
 */
int pkv_paged_attention(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                        const int32_t* page_tables, int32_t num_seqs, int32_t total_q,
                        int32_t num_q_heads, int32_t max_pages_per_seq, int32_t max_kv_len,
                        const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                        float scale, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * FP8 (e4m3) KV cache. mini-vLLM, "Quantization": 8-bit weights widened
 * before every matmul saved memory but slowed decode, and the page names a
 * fused low-precision kernel as the missing step. Here the cache holds one
 * byte per element and the attention kernel widens the codes in registers, so
 * a decode step reads half the bytes of a 16-bit cache.
 *
 * Cache dtype PKV_FP8_E4M3: same [num_pages, page_size, num_kv_heads,
 * head_dim] layout, one e4m3 code per element (1 sign, 4 exponent bits with
 * bias 7, 3 mantissa bits; largest finite 448; no infinities). Element
 * (slot, h, i) stands for code * k_scale[h] (K) or code * v_scale[h] (V);
 * k_scale, v_scale are device float [num_kv_heads], owned by the caller,
 * finite and > 0.
 *
 * pkv_kv_append_quant: as pkv_kv_append, but k, v are [num_tokens,
 * num_kv_heads, head_dim] of src_dtype (PKV_F32/F16/BF16) and each element x
 * is stored as e4m3(x / scale[h]): the quotient in IEEE float32 (correctly
 * rounded), then the nearest e4m3 value, ties to even, saturating to +-448
 * (NaN stays NaN). Bit-exact against that definition. head_dim must be a
 * multiple of 16. Errors as pkv_kv_append; PKV_E_DTYPE unless the cache is
 * PKV_FP8_E4M3 (pkv_kv_append and pkv_rope_kv_append answer PKV_E_DTYPE for an
 * fp8 cache).
 *
 * pkv_paged_attention_fp8: as pkv_paged_attention over an fp8 cache; q and
 * out are q_dtype (PKV_BF16 or PKV_F16), lse as there. Scores are
 * (q . code) * k_scale[h] * scale and the output is (sum p_j code_j) *
 * v_scale[h] / sum p_j. q is rounded to fp16 for the products with the codes
 * (every e4m3 value is exact in fp16), so bf16 queries must lie within fp16's
 * range. head_dim must be 128; page_size as for the 16-bit decode path. Decode
 * rows and short chunks run on the TMA-staged row kernel; a chunk of 64 rows
 * or more runs on the tensor-core prefill kernel (scale > 0, page_size a
 * multiple or divisor of 128, any group size), which widens each K/V tile to fp16
 * in shared memory before its MMAs; other chunks go row by row.
 * Errors as pkv_paged_attention, plus PKV_E_DTYPE for another cache or query
 * type and PKV_E_NULL for missing scales. pkv_paged_attention answers
 * PKV_E_DTYPE for an fp8 cache. The workspace size is
 * pkv_paged_attention_workspace_size with the fp8 cache descriptor.
 */
int pkv_kv_append_quant(const void* k, const void* v, int32_t src_dtype, const int64_t* slot_mapping,
                        int32_t num_tokens, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                        const float* k_scale, const float* v_scale, pkv_stream_t stream);
int pkv_paged_attention_fp8(const void* q, int32_t q_dtype, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                            const int32_t* page_tables, int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                            int32_t max_pages_per_seq, int32_t max_kv_len, const void* k_cache,
                            const void* v_cache, const pkv_cache_desc* cache, const float* k_scale,
                            const float* v_scale, float scale, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * Host page pool and prefix cache (no device work; host memory only).
 *
 * A fixed pool of page ids with per-page reference counts, and a cache of
 * complete prompt blocks keyed by a hash chained over the blocks before them
 * (Helios README, "Paged attention": pages come from a free list and return
 * to the pool when the last request or prefix-cache entry holding them lets
 * go; Helios blog, "Prefix caching": complete page-size prompt blocks are
 * hashed with the previous block's hash, a request reuses the longest matching
 * chain's pages, partial blocks are not stored, entries have a sliding TTL and
 * eviction takes unused leaf blocks first).
 *  - pkv_pool_alloc hands out the lowest free ids first, each with count 1;
 *    PKV_E_CAPACITY (nothing taken) when fewer than n pages are free.
 *  - pkv_pool_retain / pkv_pool_release add / drop one reference per listed
 *    page (a page may be listed several times); a page whose count reaches 0
 *    is free again. PKV_E_PAGES (nothing changed) for an id outside the pool,
 *    a free page, or more releases than references.
 *  - pkv_prefix_lookup walks tokens[0 .. n_tokens) block by block (page_size
 *    tokens each) and returns the number of leading blocks found in the cache
 *    (at most max_pages); their page ids go to pages[] and each gets one more
 *    reference, now owned by the caller; their last-use time becomes `now`.
 *  - pkv_prefix_insert stores every complete block of tokens not yet cached,
 *    on the caller's page for that block (pages[b] for block b); the cache
 *    takes one reference per stored page. Returns the number of new entries.
 *  - pkv_prefix_evict drops unused leaf entries (the cache holds the only
 *    reference and no cached block continues them): first every entry unused
 *    for more than `ttl` (sliding), then, oldest last use first, until at
 *    least want_free pages are free or nothing is evictable. Returns the
 *    number of entries dropped.
 * The pool object is not thread-safe; callers serialise access.
 */
typedef struct pkv_pool pkv_pool;
int pkv_pool_create(int32_t num_pages, int32_t page_size, pkv_pool** out);
void pkv_pool_destroy(pkv_pool* pool);
int pkv_pool_alloc(pkv_pool* pool, int32_t n, int32_t* pages);
int pkv_pool_retain(pkv_pool* pool, const int32_t* pages, int32_t n);
int pkv_pool_release(pkv_pool* pool, const int32_t* pages, int32_t n);
int pkv_pool_free_count(const pkv_pool* pool);
int pkv_pool_refcount(const pkv_pool* pool, int32_t page);
int pkv_prefix_lookup(pkv_pool* pool, const int32_t* tokens, int32_t n_tokens, double now, int32_t* pages,
                      int32_t max_pages);
int pkv_prefix_insert(pkv_pool* pool, const int32_t* tokens, int32_t n_tokens, const int32_t* pages,
                      int32_t n_pages, double now);
int pkv_prefix_evict(pkv_pool* pool, double now, double ttl, int32_t want_free);
int pkv_prefix_size(const pkv_pool* pool);

/* ---------------------------------------------------------------------------
 * pkv_paged_attention_no_alloc — pkv_paged_attention without a workspace
 * argument, for callers that cannot allocate device memory (for example code
 * running inside a memory pool's or custom allocator's own callbacks, or a
 * plug-in that is handed only the tensors it reads and writes). The serving
 * pages have no counterpart of this call; it is a deployment convenience.
 *
 * Arguments, results, layouts and errors are those of pkv_paged_attention,
 * minus workspace/workspace_bytes. The scratch the call needs (its work plan
 * and split-KV partial results) lives in a fixed array of
 * PKV_NO_ALLOC_SCRATCH_BYTES inside the library's device image, which every
 * GPU that loads the library holds until the process exits. The call itself
 * calls no cudaMalloc, cudaFree or allocating library routine.
 *  - Limit: sizes whose work plan does not fit the array (very many packed
 *    rows) return PKV_E_WORKSPACE; the split-KV partials get the room that is
 *    left, and the split size grows until they fit.
 *  - Set-up: the first call on each device looks up the array's device address
 *    (with that device current); make that first call before any stream
 *    capture.
 *  - Sharing: every call on a device uses the same array, which keeps the last
 *    call's contents; each call rewrites every counter and control word it
 *    reads before using it. Calls that overlap on the GPU (for example on two
 *    streams at once) race on the array and give undefined results: serialise
 *    them.
 */
#define PKV_NO_ALLOC_SCRATCH_BYTES (16u << 20)

int pkv_paged_attention_no_alloc(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                                 const int32_t* page_tables, int32_t num_seqs, int32_t total_q,
                                 int32_t num_q_heads, int32_t max_pages_per_seq, int32_t max_kv_len,
                                 const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                                 float scale, void* out, float* lse, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * Latent attention: keys and values of all heads from one shared vector a token.
 *
 * A latent cache keeps for each token a latent part c (latent_dim values) and a
 * rotary key part r (rope_dim values), one row [c, r] shared by every head, in
 * the same kind of page pool as above: contiguous
 * [num_pages, page_size, latent_dim + rope_dim], PKV_BF16 or PKV_F16. Per token
 * that is 576 values at latent_dim 512, against 2 * heads * head_dim for a K/V
 * cache. Models attend over it in two forms with equal results in exact
 * arithmetic:
 *  - absorbed (pkv_latent_attention), for decode rows: the key up-projection is
 *    multiplied into the query beforehand, so a head's query is latent_dim +
 *    rope_dim wide, every head attends the cached rows themselves, and the
 *    output is the weighted sum of the latent parts (the caller applies the
 *    value up-projection to it);
 *  - expanded (pkv_latent_prefill), for chunks: the caller gathers the cached
 *    rows (pkv_latent_gather), up-projects the latent parts to a 128-wide key
 *    and a 128-wide value per head, and attends over those and the shared
 *    rotary key part. Per (query, key) pair and head it computes 320 products
 *    against the absorbed form's 1088.
 * The calls follow the conventions above (ownership, asynchrony, errors, the
 * device status word). Page tables, cu_seqlens and kv_lens are those of
 * pkv_pack_tick; every causal rule is bottom-right: row i of a sequence with
 * q_len rows and kv_len keys sees keys 0 .. kv_len - q_len + i.
 *
 * latent_dim is 256 or 512 and rope_dim 64 (PKV_E_SHAPE otherwise). Any
 * page_size >= 1 is taken; rows of pages that are a multiple of 32 long move by
 * TMA, others by 16-byte copies of threads: in decode of 64 sequences of 1000-4000 keys, against
 * pages of 64, pages of 16 and 8 are 1-8 % slower at latent_dim 512 and 3-9 % at 256, pages
 * of one row 12 % and 24-32 %. */
typedef struct {
  int32_t num_pages;
  int32_t page_size;
  int32_t latent_dim; /* 256 or 512 */
  int32_t rope_dim;   /* 64 */
  int32_t dtype;      /* PKV_F16 or PKV_BF16 */
} pkv_latent_desc;

/* pkv_latent_append — write new tokens' rows [c, rotated r] into their slots,
 * and rotate the rotary parts of the tick's queries.
 *
 *   c_kv       device, latent part of token t at c_kv + t * c_stride (elements of the
 *              cache dtype, latent_dim of them)
 *   k_rope     device, rotary key part of token t at k_rope + t * kr_stride, not yet rotated
 *   q_rope     device or NULL, rotary part of head h of token t at
 *              q_rope + t * q_stride_t + h * q_stride_h, not yet rotated
 *   q_out      device, where its rotation goes: q_out + t * qo_stride_t + h *
 *              qo_stride_h; may be q_rope itself with the same strides (in place), and must
 *              not overlap it otherwise. NULL with a NULL q_rope.
 *   positions, cos_sin, max_pos, slot_mapping  as pkv_rope_kv_append (half-split
 *              rotation over rope_dim values, in fp32, rounded once). Weights made for rotating
 *              neighbours (x0, x1), (x2, x3), .. need the rotary columns of both the query and
 *              the key projection reordered once, when they are loaded: the even ones first,
 *              then the odd ones. Scores are the same.
 * Strides are in elements and may be any multiple of 8 (views of wider
 * projection outputs); c_kv, k_rope, q_rope, q_out, cos_sin and cache must be 16-byte
 * aligned. A negative slot skips the token's cache row (its queries are still
 * rotated); a slot past the pool sets PKV_DEV_BAD_SLOT and skips the row. A
 * position outside [0, max_pos) sets PKV_DEV_BAD_POSITION and skips the token
 * altogether, the latent part included. Duplicate slots are a caller error.
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE (also a stride that is negative or not a multiple of 8,
 * num_q_heads < 1 with queries), PKV_E_ALIGN, PKV_E_DEVICE, PKV_E_CUDA. */
int pkv_latent_append(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t kr_stride,
                      const void* q_rope, int64_t q_stride_t, int64_t q_stride_h, void* q_out,
                      int64_t qo_stride_t, int64_t qo_stride_h, int32_t num_q_heads, const int32_t* positions,
                      const float* cos_sin, int32_t max_pos, const int64_t* slot_mapping, int32_t num_tokens,
                      void* cache, const pkv_latent_desc* desc, pkv_stream_t stream);

/* pkv_latent_gather — copy the cached rows of every sequence, in order, into
 * one packed tensor (bit for bit).
 *
 *   page_tables   device, int32 [num_seqs, max_pages_per_seq]
 *   cu_seqlens_k  device, int32 [num_seqs + 1]; sequence b's rows 0 .. cu[b+1] - cu[b] - 1
 *                 go to out rows cu[b] .. cu[b+1] - 1
 *   total_k       rows of `out`; rows from cu[num_seqs] on are left as they were
 *   out           device, contiguous [total_k, latent_dim + rope_dim], cache dtype, not
 *                 overlapping the cache
 * cu_seqlens_k that does not start at 0, decreases, or ends past total_k sets
 * PKV_DEV_BAD_LENGTHS and copies nothing; so does a sequence longer than its
 * page table, for that sequence. A page id outside the pool sets
 * PKV_DEV_BAD_PAGE and skips the rows of that page.
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE, PKV_E_ALIGN, PKV_E_DEVICE, PKV_E_CUDA. */
int pkv_latent_gather(const void* cache, const pkv_latent_desc* desc, const int32_t* page_tables,
                      int32_t max_pages_per_seq, const int32_t* cu_seqlens_k, int32_t num_seqs, int32_t total_k,
                      void* out, pkv_stream_t stream);

/* pkv_latent_attention — the absorbed form over the pages.
 *
 *   q             device, contiguous [total_q, num_q_heads, latent_dim + rope_dim], cache dtype:
 *                 the absorbed part first, then the rotated rotary part
 *   cu_seqlens_q, kv_lens, page_tables, max_kv_len, lse  as pkv_paged_attention, but for
 *                 cu[num_seqs], which may be less than total_q: rows from there on
 *                 are padding, may hold anything and are left as they were
 *   scale         > 0 and finite; multiplies q . [c, r] before the softmax
 *   out           device, contiguous [total_q, num_q_heads, latent_dim], cache dtype
 *   workspace     device, >= pkv_latent_attention_workspace_size(...) bytes, 256-byte
 *                 aligned; needs no initialisation; one for the largest call serves smaller
 *                 ones. Calls that may overlap (two streams, two captured graphs replayed
 *                 side by side) need one each.
 * Sums and softmax statistics are fp32; the softmax weights are rounded to the
 * cache dtype for the products with the latent parts. Keys of a sequence are
 * split over the GPU by the tick's total work, so the order of a row's fp32 sums
 * depends on the other rows of the tick (the same call gives the same bits).
 * Bad lengths skip the sequence's rows as in pkv_paged_attention (bad
 * cu_seqlens_q: every row). A page id outside the pool sets PKV_DEV_BAD_PAGE, and the
 * rows that need the page, with up to 127 (token, head) rows of the sequence beside
 * them, are left unwritten. Slots that no sequence owns may hold anything. A NaN in
 * a sequence's own row reaches every row that sees it, and a NaN or an infinity may
 * reach earlier rows of the same chunk (0 * NaN, as in a product with a masked weight
 * matrix). A row all of whose scores are -inf is NaN, with an lse of -inf. num_q_heads is at most 4096.
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE, PKV_E_ALIGN, PKV_E_WORKSPACE, PKV_E_DEVICE, PKV_E_CUDA. */
size_t pkv_latent_attention_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                           const pkv_latent_desc* desc);
int pkv_latent_attention(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                         const int32_t* page_tables, int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                         int32_t max_pages_per_seq, int32_t max_kv_len, const void* cache,
                         const pkv_latent_desc* desc, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, pkv_stream_t stream);

/* pkv_latent_prefill — the expanded form over packed keys and values.
 *
 *   q             device, contiguous [total_q, num_heads, 192]: 128 values against k_nope,
 *                 then 64 rotated values against k_rope
 *   k_nope, v     device, key and value of head h of packed key row t at + t * stride_t +
 *                 h * stride_h, 128 values each (views of one up-projection output will do)
 *   k_rope        device, shared rotary key part of row t at + t * kr_stride, 64 values
 *   cu_seqlens_q, cu_seqlens_k  device, int32 [num_seqs + 1]: rows of q / of the keys by
 *                 sequence; from 0, non-decreasing, ending at or before total_q /
 *                 total_k (rows behind are padding, may hold anything and are left as they were)
 *   dtype         PKV_BF16 or PKV_F16, of q, k_nope, v, k_rope and out
 *   scale         > 0 and finite
 *   out           device, contiguous [total_q, num_heads, 128]
 *   lse           device, fp32 [total_q, num_heads] or NULL
 *   workspace     device, >= pkv_latent_prefill_workspace_size(...) bytes, 256-byte aligned;
 *                 needs no initialisation; one for the largest call serves smaller ones;
 *                 one for each of calls that may overlap
 * Sequence b has kv_len = cu_k[b+1] - cu_k[b] >= q_len keys; the last q_len of
 * them are the chunk's own. A sequence with rows and fewer keys than rows sets
 * PKV_DEV_BAD_LENGTHS and is skipped; a cu_seqlens array that breaks the rules
 * above skips every row. Strides are in elements, multiples of 8; pointers
 * 16-byte aligned. Values of other sequences' rows never reach a row, NaN or not; a
 * NaN in a sequence's own key or value reaches every row that sees it, and a NaN or
 * an infinity may reach earlier rows of the same chunk (0 * NaN). A row all of whose
 * scores are -inf is NaN, with an lse of -inf. Sums and softmax statistics are fp32; the
 * softmax weights are rounded to dtype for the products with the values. Calls of few tiles
 * split their keys over the GPU by the tick's total work: the order of a row's
 * fp32 sums then depends on the other rows (the same call gives the same bits).
 * Errors: PKV_E_NULL, PKV_E_DTYPE, PKV_E_SHAPE, PKV_E_ALIGN, PKV_E_WORKSPACE, PKV_E_DEVICE, PKV_E_CUDA. */
size_t pkv_latent_prefill_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_heads);
int pkv_latent_prefill(const void* q, const int32_t* cu_seqlens_q, const void* k_nope, int64_t kn_stride_t,
                       int64_t kn_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h,
                       const void* k_rope, int64_t kr_stride, const int32_t* cu_seqlens_k, int32_t num_seqs,
                       int32_t total_q, int32_t total_k, int32_t num_heads, int32_t dtype, float scale, void* out,
                       float* lse, void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * Status and instrumentation. */

/* Human-readable text for a pkv_status code (static storage). */
const char* pkv_status_string(int status);

/* Text of the CUDA error behind the calling thread's last PKV_E_CUDA
 * (thread-local storage, valid until that thread's next failing call). */
const char* pkv_last_error(void);

/* Waits for `stream`, then returns in *code the OR of the PKV_DEV_* bits set
 * on the current device since the last call, and clears them. */
int pkv_get_device_status(int32_t* code, pkv_stream_t stream);

/* Kernel timing: when enabled (1), every kernel the library launches is
 * bracketed by CUDA events on its launch stream; pkv_kernel_times waits for
 * the recorded work and returns, per kernel name, the number of launches and
 * the summed device time, then clears the record. Disabled (0) by default. */
int pkv_set_kernel_timing(int enable);
/* Fills up to `max` entries; returns the number of kernels recorded (>= 0) or
 * a negative pkv_status. names[i] points at static storage. */
int pkv_kernel_times(const char** names, int32_t* launches, double* total_ms, int32_t max);

/* Self-test of the failure path (the pages have no counterpart; it checks the
 * library's own error handling). Enqueues on `stream` one CTA laid out like
 * the prefill kernel's (a producer warp, an MMA-issuer thread, eight softmax
 * warps), each waiting, through the bounded pipeline wait that every decode and
 * prefill kernel of the library uses, on a barrier that nothing ever completes.
 * The producer warp waits with a limit of limit_us microseconds, gives up
 * first, raises the CTA's abort flag and records PKV_DEV_TIMEOUT in the CTA's
 * error word and in the device status word (read and cleared by
 * pkv_get_device_status); the other warps see the flag and return. The CUDA
 * context stays usable.
 *  - result: device int32[2] or NULL. [0] = the CTA's error word
 *    (PKV_DEV_TIMEOUT), [1] = warps that left their wait without the barrier
 *    (10 when every warp drained). Cleared on `stream` before the launch.
 *  - limit_us must lie in [1, 1000000], else PKV_E_SHAPE and nothing is
 *    launched; PKV_E_ALIGN if result is not 4-byte aligned; PKV_E_CUDA if the
 *    launch fails. */
int pkv_selftest_bounded_wait(int32_t limit_us, int32_t* result, pkv_stream_t stream);

/* Library version string. */
const char* pkv_version(void);

#ifdef __cplusplus
}
#endif
#endif /* PAGEDKV_H_ */
