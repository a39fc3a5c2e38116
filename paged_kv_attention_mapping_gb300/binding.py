"""Thin ctypes binding of libpagedkv (declared in include/pagedkv.h).

Argument marshalling only: torch tensors become device pointers and the
current torch stream becomes the cudaStream_t; every step of the computation
runs in the library's kernels. There is no fallback: if the library is missing
or cannot be loaded, every call raises.
"""
from __future__ import annotations

import array
import ctypes
import functools
import itertools
import os
import struct
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

PKV_F32, PKV_F16, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2, 3
DEV_BAD_SLOT, DEV_BAD_LENGTHS, DEV_BAD_PAGE, DEV_TIMEOUT, DEV_BAD_POSITION = 0x1, 0x2, 0x4, 0x8, 0x10

EXPORTED = (
    "pkv_pack_tick",
    "pkv_kv_append",
    "pkv_paged_attention_workspace_size",
    "pkv_paged_attention",
    "pkv_paged_attention_no_alloc",
    "pkv_status_string",
    "pkv_get_device_status",
    "pkv_selftest_bounded_wait",
    "pkv_set_kernel_timing",
    "pkv_kernel_times",
    "pkv_version",
    "pkv_last_error",
    "pkv_pool_create",
    "pkv_pool_destroy",
    "pkv_pool_alloc",
    "pkv_pool_retain",
    "pkv_pool_release",
    "pkv_pool_free_count",
    "pkv_pool_refcount",
    "pkv_prefix_lookup",
    "pkv_prefix_insert",
    "pkv_prefix_evict",
    "pkv_prefix_size",
    "pkv_rope_table",
    "pkv_rope_kv_append",
    "pkv_tick_positions",
    "pkv_kv_append_quant",
    "pkv_paged_attention_fp8",
    "pkv_latent_append",
    "pkv_latent_gather",
    "pkv_latent_attention_workspace_size",
    "pkv_latent_attention",
    "pkv_latent_prefill_workspace_size",
    "pkv_latent_prefill",
    "pkv_norm_rope_kv_append",
    "pkv_rope_table_scaled",
    "pkv_window_attention",
    "pkv_copy_pages",
    "pkv_remap_pages",
    "pkv_pool_fork",
    "pkv_pool_fork_window",
    "pkv_pool_compact",
    "pkv_pool_trim",
    "pkv_pack_tick_window",
)


class PagedKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f"; {lib().pkv_last_error().decode()}" if status == -8 else ""
        super().__init__(f"{where}: {status_string(status)} (status {status}){detail}")


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class LatentDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


# pkv_norm_rope_args: pointers, strides, pointers, sizes, the cache's description
_NORM_ROPE_ARGS = struct.Struct("@4P8q9P6if5i")


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original_max_pos", ctypes.c_double), ("attention_factor", ctypes.c_double)]


_lib = None


def lib():
    """Load libpagedkv.so (built by paged_kv_attention_mapping_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libpagedkv.so is not built ({LIB_PATH}); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'` first")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    P32, P64 = ctypes.POINTER(i32), ctypes.POINTER(i64)
    L.pkv_pack_tick.argtypes = [i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.pkv_pack_tick.restype = ctypes.c_int
    L.pkv_kv_append.argtypes = [vp, vp, vp, i32, vp, vp, ctypes.POINTER(CacheDesc), vp]
    L.pkv_kv_append.restype = ctypes.c_int
    L.pkv_paged_attention_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(CacheDesc), i32]
    L.pkv_paged_attention_workspace_size.restype = sz
    L.pkv_paged_attention.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                      ctypes.POINTER(CacheDesc), ctypes.c_float, vp, vp, vp, sz, vp]
    L.pkv_paged_attention.restype = ctypes.c_int
    L.pkv_paged_attention_no_alloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                               ctypes.POINTER(CacheDesc), ctypes.c_float, vp, vp, vp]
    L.pkv_paged_attention_no_alloc.restype = ctypes.c_int
    L.pkv_status_string.argtypes = [ctypes.c_int]
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_get_device_status.argtypes = [P32, vp]
    L.pkv_get_device_status.restype = ctypes.c_int
    L.pkv_selftest_bounded_wait.argtypes = [i32, vp, vp]
    L.pkv_selftest_bounded_wait.restype = ctypes.c_int
    L.pkv_set_kernel_timing.argtypes = [ctypes.c_int]
    L.pkv_set_kernel_timing.restype = ctypes.c_int
    L.pkv_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_char_p), P32, ctypes.POINTER(ctypes.c_double), i32]
    L.pkv_kernel_times.restype = ctypes.c_int
    L.pkv_last_error.argtypes = []
    L.pkv_last_error.restype = ctypes.c_char_p
    L.pkv_pool_create.argtypes = [i32, i32, ctypes.POINTER(vp)]
    L.pkv_pool_create.restype = ctypes.c_int
    L.pkv_pool_destroy.argtypes = [vp]
    L.pkv_pool_destroy.restype = None
    for name in ("pkv_pool_alloc", "pkv_pool_retain", "pkv_pool_release"):
        getattr(L, name).argtypes = [vp, P32, i32] if name != "pkv_pool_alloc" else [vp, i32, P32]
        getattr(L, name).restype = ctypes.c_int
    L.pkv_pool_free_count.argtypes = [vp]
    L.pkv_pool_free_count.restype = ctypes.c_int
    L.pkv_pool_refcount.argtypes = [vp, i32]
    L.pkv_pool_refcount.restype = ctypes.c_int
    L.pkv_prefix_lookup.argtypes = [vp, P32, i32, ctypes.c_double, P32, i32]
    L.pkv_prefix_lookup.restype = ctypes.c_int
    L.pkv_prefix_insert.argtypes = [vp, P32, i32, P32, i32, ctypes.c_double]
    L.pkv_prefix_insert.restype = ctypes.c_int
    L.pkv_prefix_evict.argtypes = [vp, ctypes.c_double, ctypes.c_double, i32]
    L.pkv_prefix_evict.restype = ctypes.c_int
    L.pkv_prefix_size.argtypes = [vp]
    L.pkv_prefix_size.restype = ctypes.c_int
    L.pkv_rope_table.argtypes = [ctypes.c_double, i32, i32, ctypes.POINTER(ctypes.c_float)]
    L.pkv_rope_table.restype = ctypes.c_int
    L.pkv_rope_kv_append.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, ctypes.POINTER(CacheDesc), vp, vp]
    L.pkv_rope_kv_append.restype = ctypes.c_int
    L.pkv_kv_append_quant.argtypes = [vp, vp, i32, vp, i32, vp, vp, ctypes.POINTER(CacheDesc), vp, vp, vp]
    L.pkv_kv_append_quant.restype = ctypes.c_int
    L.pkv_paged_attention_fp8.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                          ctypes.POINTER(CacheDesc), vp, vp, ctypes.c_float, vp, vp, vp, sz, vp]
    L.pkv_paged_attention_fp8.restype = ctypes.c_int
    L.pkv_tick_positions.argtypes = [i32, P32, P32, P32, i32]
    L.pkv_tick_positions.restype = ctypes.c_int
    PL = ctypes.POINTER(LatentDesc)
    L.pkv_latent_append.argtypes = [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, i32, vp, vp, i32, vp, i32, vp, PL,
                                    vp]
    L.pkv_latent_append.restype = ctypes.c_int
    L.pkv_latent_gather.argtypes = [vp, PL, vp, i32, vp, i32, i32, vp, vp]
    L.pkv_latent_gather.restype = ctypes.c_int
    L.pkv_latent_attention_workspace_size.argtypes = [i32, i32, i32, PL]
    L.pkv_latent_attention_workspace_size.restype = sz
    L.pkv_latent_attention.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, PL, ctypes.c_float, vp, vp, vp,
                                       sz, vp]
    L.pkv_latent_attention.restype = ctypes.c_int
    L.pkv_latent_prefill_workspace_size.argtypes = [i32, i32, i32]
    L.pkv_latent_prefill_workspace_size.restype = sz
    L.pkv_latent_prefill.argtypes = [vp, vp, vp, i64, i64, vp, i64, i64, vp, i64, vp, i32, i32, i32, i32, i32,
                                     ctypes.c_float, vp, vp, vp, sz, vp]
    L.pkv_latent_prefill.restype = ctypes.c_int
    PC, f32 = ctypes.POINTER(CacheDesc), ctypes.c_float
    L.pkv_norm_rope_kv_append.argtypes = [ctypes.c_char_p, vp]
    L.pkv_norm_rope_kv_append.restype = ctypes.c_int
    L.pkv_rope_table_scaled.argtypes = [ctypes.c_double, i32, ctypes.POINTER(RopeScaling), i32,
                                        ctypes.POINTER(f32)]
    L.pkv_rope_table_scaled.restype = ctypes.c_int
    L.pkv_window_attention.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, PC, vp, vp, f32, vp,
                                       vp, vp]
    L.pkv_window_attention.restype = ctypes.c_int
    L.pkv_copy_pages.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, i32, vp]
    L.pkv_copy_pages.restype = ctypes.c_int
    L.pkv_remap_pages.argtypes = [vp, i64, vp, i32, vp]
    L.pkv_remap_pages.restype = ctypes.c_int
    L.pkv_pool_fork.argtypes = [vp, P32, i32, i32, P32, P32, P32, P32]
    L.pkv_pool_fork.restype = ctypes.c_int
    L.pkv_pool_fork_window.argtypes = [vp, P32, i32, i32, i32, i32, P32, P32, P32, P32]
    L.pkv_pool_fork_window.restype = ctypes.c_int
    L.pkv_pool_compact.argtypes = [vp, i32, P32, P32, P32]
    L.pkv_pool_compact.restype = ctypes.c_int
    L.pkv_pool_trim.argtypes = [vp, P32, i32, i32, i32, i32]
    L.pkv_pool_trim.restype = ctypes.c_int
    L.pkv_pack_tick_window.argtypes = [i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.pkv_pack_tick_window.restype = ctypes.c_int
    L.pkv_version.argtypes = []
    L.pkv_version.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


def version() -> str:
    return lib().pkv_version().decode()


def _check(status: int, where: str):
    if status != 0:
        raise PagedKVError(status, where)


# ---------------------------------------------------------------------------
# host packing

def _count(n):
    """A window or a number of sinks as a 32-bit argument: contexts are shorter than 2^31, so what is
    larger means the same; what is negative is refused by the call, not wrapped."""
    return -1 if n < 0 else n if n < 2147483648 else 2147483647


def pack_tick(q_lens: Sequence[int], kv_lens: Sequence[int], pages: Sequence[Sequence[int]], page_size: int,
              num_pages: int, max_pages_per_seq: Optional[int] = None, window: Optional[int] = None, sinks: int = 0):
    """Host packing of one tick (pkv_pack_tick). Returns numpy arrays:
    order, cu_seqlens_q, kv_lens, page_tables [B, W] (-1 padded), slot_mapping.
    With a `window` (pkv_pack_tick_window) pages that no row of the tick sees may be -1."""
    B = len(q_lens)
    counts = [len(p) for p in pages]
    offs = np.zeros(B + 1, dtype=np.int32)
    if B:
        np.cumsum(counts, out=offs[1:])
    ids = np.fromiter(itertools.chain.from_iterable(pages), dtype=np.int32, count=int(offs[-1]))
    return pack_tick_flat(np.asarray(q_lens, dtype=np.int32), np.asarray(kv_lens, dtype=np.int32), offs, ids,
                          page_size, num_pages, max_pages_per_seq, window=window, sinks=sinks)


def pack_tick_flat(q_lens, kv_lens, page_offsets, page_ids, page_size: int, num_pages: int,
                   max_pages_per_seq: Optional[int] = None, out: Optional[dict] = None, window: Optional[int] = None,
                   sinks: int = 0):
    """pack_tick on flat int32 arrays, the form a scheduler keeps its block
    tables in: sequence b owns page_ids[page_offsets[b]:page_offsets[b + 1]].

    `out` may hold preallocated (for example pinned) numpy arrays to write into:
    order [>= B], cu_seqlens_q [B + 1], kv_lens [>= B], page_tables [B, W] and
    slot_mapping [>= sum of q_lens] (int64), so that a serving loop packs each
    tick without allocating. Returns the same dict as pack_tick (views of `out`)."""
    ql = np.ascontiguousarray(q_lens, dtype=np.int32)
    kl = np.ascontiguousarray(kv_lens, dtype=np.int32)
    offs = np.ascontiguousarray(page_offsets, dtype=np.int32)
    ids = np.ascontiguousarray(page_ids, dtype=np.int32)
    B = int(ql.shape[0])
    if offs.shape[0] != B + 1:
        raise ValueError("page_offsets must have num_seqs + 1 entries")
    if ids.size == 0:
        ids = np.zeros(1, dtype=np.int32)
    if max_pages_per_seq is not None:
        W = int(max_pages_per_seq)
    else:
        W = int(np.max(np.diff(offs))) if B else 1
    W = max(W, 1)
    cap = int(max(int(ql.clip(min=0).sum()), 1))
    if out is None:
        out = dict(order=np.zeros(max(B, 1), dtype=np.int32), cu_seqlens_q=np.zeros(B + 1, dtype=np.int32),
                   kv_lens=np.zeros(max(B, 1), dtype=np.int32), page_tables=np.zeros((max(B, 1), W), dtype=np.int32),
                   slot_mapping=np.zeros(cap, dtype=np.int64))
    order, cu, kv_out, tables, slots = (out["order"], out["cu_seqlens_q"], out["kv_lens"], out["page_tables"],
                                        out["slot_mapping"])
    if (order.dtype != np.int32 or cu.dtype != np.int32 or kv_out.dtype != np.int32 or tables.dtype != np.int32
            or slots.dtype != np.int64):
        raise ValueError("pack_tick_flat: out arrays must be int32 (slot_mapping int64)")
    if (order.size < max(B, 1) or cu.size < B + 1 or kv_out.size < max(B, 1) or tables.ndim != 2
            or tables.shape[0] < max(B, 1) or tables.shape[1] != W or slots.size < cap):
        raise ValueError("pack_tick_flat: out arrays too small for this tick")
    for a in (order, cu, kv_out, tables, slots):
        if not a.flags.c_contiguous:
            raise ValueError("pack_tick_flat: out arrays must be C-contiguous")
    total = np.zeros(1, dtype=np.int32)
    given = (B, ql.ctypes.data if B else None, kl.ctypes.data if B else None, offs.ctypes.data, ids.ctypes.data,
             int(page_size), int(num_pages), W, cap)
    wanted = (order.ctypes.data, cu.ctypes.data, kv_out.ctypes.data, tables.ctypes.data, slots.ctypes.data,
              total.ctypes.data)
    if window is None:
        _check(lib().pkv_pack_tick(*given, *wanted), "pkv_pack_tick")
    else:
        _check(lib().pkv_pack_tick_window(*given, _count(int(window)), _count(int(sinks)), *wanted), "pkv_pack_tick_window")
    T = int(total[0])
    return dict(order=order[:B], cu_seqlens_q=cu[:B + 1], kv_lens=kv_out[:B], page_tables=tables[:B],
                slot_mapping=slots[:T])


# ---------------------------------------------------------------------------
# device calls (torch tensors)

@functools.lru_cache(maxsize=None)
def _code_of(dtype) -> int:
    import torch
    m = {torch.float32: PKV_F32, torch.float16: PKV_F16, torch.bfloat16: PKV_BF16,
         torch.uint8: PKV_FP8_E4M3}
    if hasattr(torch, "float8_e4m3fn"):
        m[torch.float8_e4m3fn] = PKV_FP8_E4M3
    if dtype not in m:
        raise TypeError(f"unsupported dtype {dtype}")
    return m[dtype]


def _dtype_code(t) -> int:
    return _code_of(t.dtype)


def cache_desc(k_cache) -> CacheDesc:
    if k_cache.dim() != 4 or not k_cache.is_contiguous():
        raise ValueError("cache must be a contiguous [num_pages, page_size, num_kv_heads, head_dim] tensor")
    N, P, H, D = k_cache.shape
    return CacheDesc(N, P, H, D, _dtype_code(k_cache))


def _stream_ptr(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def kv_append(k, v, slot_mapping, k_cache, v_cache, stream=None):
    """Write new tokens' K/V rows into their slots (pkv_kv_append)."""
    for t in (k, v, slot_mapping, k_cache, v_cache):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("kv_append needs contiguous CUDA tensors")
    import torch
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    desc = cache_desc(k_cache)
    st = lib().pkv_kv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), int(k.shape[0]), _ptr(k_cache), _ptr(v_cache),
                             ctypes.byref(desc), _stream_ptr(stream))
    _check(st, "pkv_kv_append")


def workspace_size(num_seqs: int, total_q: int, num_q_heads: int, k_cache, max_kv_len: int) -> int:
    desc = cache_desc(k_cache)
    n = lib().pkv_paged_attention_workspace_size(int(num_seqs), int(total_q), int(num_q_heads), ctypes.byref(desc),
                                                 int(max_kv_len))
    if n == 0:
        raise PagedKVError(-3, "pkv_paged_attention_workspace_size")
    return int(n)


def alloc_workspace(num_seqs, total_q, num_q_heads, k_cache, max_kv_len):
    import torch
    n = workspace_size(num_seqs, total_q, num_q_heads, k_cache, max_kv_len)
    return torch.empty(n, dtype=torch.uint8, device=k_cache.device)


def _check_attention_args(where, q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, out, lse,
                          extra=(), q_matches_cache=True):
    """The checks every attention call makes before any pointer reaches the
    library: CUDA, contiguous, int32 index tensors, consistent dtypes and shapes."""
    import torch
    for t in (cu_seqlens_q, kv_lens, page_tables):
        if t.dtype != torch.int32:
            raise TypeError(f"{where}: index tensors must be int32")
    if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
        raise TypeError(f"{where}: k_cache and v_cache must share one dtype and shape")
    if q_matches_cache and q.dtype != k_cache.dtype:
        raise TypeError(f"{where}: q, k_cache and v_cache must share one dtype")
    for t in (q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache) + tuple(extra):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{where} needs contiguous CUDA tensors")
    if q.dim() != 3 or page_tables.dim() != 2 or cu_seqlens_q.dim() != 1 or kv_lens.dim() != 1:
        raise ValueError(f"{where}: q [T, Hq, d], cu_seqlens_q [B+1], kv_lens [B], page_tables [B, W]")
    B = int(cu_seqlens_q.shape[0]) - 1
    if B < 0 or int(kv_lens.shape[0]) < B or int(page_tables.shape[0]) < B:
        raise ValueError(f"{where}: cu_seqlens_q, kv_lens and page_tables disagree on the number of sequences")
    if out is not None:
        if not out.is_cuda or not out.is_contiguous() or out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError(f"{where}: out must be a contiguous CUDA tensor shaped and typed like q")
    if lse is not None:
        if (not lse.is_cuda or not lse.is_contiguous() or lse.dtype != torch.float32
                or tuple(lse.shape) != tuple(q.shape[:2])):
            raise ValueError(f"{where}: lse must be a contiguous float32 CUDA tensor [T, Hq]")


def paged_attention(q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, scale: float, max_kv_len: int,
                    out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Attention of packed query rows over their pages (pkv_paged_attention).

    q [T, Hq, d] (cache dtype); cu_seqlens_q int32 [B+1]; kv_lens int32 [B];
    page_tables int32 [B, W]; caches [N, P, Hkv, d]. Returns (out, lse)."""
    import torch
    _check_attention_args("paged_attention", q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, out, lse)
    T, Hq, D = q.shape
    B = int(cu_seqlens_q.shape[0]) - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, T, Hq, k_cache, max_kv_len)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("paged_attention: workspace must be a contiguous CUDA tensor")
    desc = cache_desc(k_cache)
    st = lib().pkv_paged_attention(_ptr(q), _ptr(cu_seqlens_q), _ptr(kv_lens), _ptr(page_tables), B, int(T), int(Hq),
                                   int(page_tables.shape[1]), int(max_kv_len), _ptr(k_cache), _ptr(v_cache),
                                   ctypes.byref(desc), ctypes.c_float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                   int(workspace.numel() * workspace.element_size()), _stream_ptr(stream))
    _check(st, "pkv_paged_attention")
    return out, lse


def paged_attention_no_alloc(q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, scale: float,
                             max_kv_len: int, out=None, lse=None, want_lse: bool = True, stream=None):
    """pkv_paged_attention_no_alloc: as paged_attention, but the library uses its
    own fixed device scratch array instead of a caller workspace (for callers
    that cannot allocate device memory). Output buffers may still be passed in;
    when they are not, this wrapper allocates them with torch (the C call
    itself never allocates)."""
    import torch
    _check_attention_args("paged_attention_no_alloc", q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache,
                          out, lse)
    T, Hq, D = q.shape
    B = int(cu_seqlens_q.shape[0]) - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    desc = cache_desc(k_cache)
    st = lib().pkv_paged_attention_no_alloc(_ptr(q), _ptr(cu_seqlens_q), _ptr(kv_lens), _ptr(page_tables), B,
                                            int(T), int(Hq), int(page_tables.shape[1]), int(max_kv_len),
                                            _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), ctypes.c_float(scale),
                                            _ptr(out), _ptr(lse), _stream_ptr(stream))
    _check(st, "pkv_paged_attention_no_alloc")
    return out, lse


def kv_append_quant(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Quantise new tokens' K/V rows to e4m3 codes of x / scale[head] and write
    them into their slots of an fp8 cache (pkv_kv_append_quant). Caches are
    uint8 (or float8_e4m3fn) [N, P, Hkv, d]; scales float32 [Hkv] on the device."""
    import torch
    for t in (k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("kv_append_quant needs contiguous CUDA tensors")
    if slot_mapping.dtype != torch.int64 or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise TypeError("slot_mapping int64, scales float32")
    desc = cache_desc(k_cache)
    st = lib().pkv_kv_append_quant(_ptr(k), _ptr(v), _dtype_code(k), _ptr(slot_mapping), int(k.shape[0]),
                                   _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), _ptr(k_scale), _ptr(v_scale),
                                   _stream_ptr(stream))
    _check(st, "pkv_kv_append_quant")


def paged_attention_fp8(q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, k_scale, v_scale, scale: float,
                        max_kv_len: int, out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Attention over an fp8 e4m3 cache (pkv_paged_attention_fp8): q/out bf16 or
    f16 [T, Hq, d]; caches uint8 codes [N, P, Hkv, d]; element = code * scale[head]."""
    import torch
    _check_attention_args("paged_attention_fp8", q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, out, lse,
                          extra=(k_scale, v_scale), q_matches_cache=False)
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise TypeError("paged_attention_fp8: scales must be float32")
    T, Hq, D = q.shape
    B = int(cu_seqlens_q.shape[0]) - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, T, Hq, k_cache, max_kv_len)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("paged_attention_fp8: workspace must be a contiguous CUDA tensor")
    desc = cache_desc(k_cache)
    st = lib().pkv_paged_attention_fp8(_ptr(q), _dtype_code(q), _ptr(cu_seqlens_q), _ptr(kv_lens),
                                       _ptr(page_tables), B, int(T), int(Hq), int(page_tables.shape[1]),
                                       int(max_kv_len), _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc),
                                       _ptr(k_scale), _ptr(v_scale), ctypes.c_float(scale), _ptr(out), _ptr(lse),
                                       _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                       _stream_ptr(stream))
    _check(st, "pkv_paged_attention_fp8")
    return out, lse


def tick_positions(cu_seqlens_q, kv_lens) -> np.ndarray:
    """Position of every packed row (pkv_tick_positions), host int32 array."""
    cu = np.ascontiguousarray(cu_seqlens_q, dtype=np.int32)
    kl = np.ascontiguousarray(kv_lens, dtype=np.int32)
    out = np.zeros(max(int(cu[-1]), 1), dtype=np.int32)
    P32 = ctypes.POINTER(ctypes.c_int32)
    _check(lib().pkv_tick_positions(len(kl), cu.ctypes.data_as(P32), kl.ctypes.data_as(P32),
                                    out.ctypes.data_as(P32), len(out)), "pkv_tick_positions")
    return out[:int(cu[-1])]


def rope_table(base: float, head_dim: int, max_pos: int) -> np.ndarray:
    """Host cos/sin table [max_pos, head_dim/2, 2] float32 (pkv_rope_table)."""
    out = np.zeros((max_pos, head_dim // 2, 2), dtype=np.float32)
    _check(lib().pkv_rope_table(float(base), int(head_dim), int(max_pos),
                                out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))), "pkv_rope_table")
    return out


def rope_kv_append(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out=None, stream=None):
    """Rotate K and write it with V to the slots; rotate Q into q_out
    (pkv_rope_kv_append). cos_sin: device float32 [max_pos, d/2, 2]."""
    import torch
    for t in (q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("rope_kv_append needs contiguous CUDA tensors")
    if positions.dtype != torch.int32 or slot_mapping.dtype != torch.int64 or cos_sin.dtype != torch.float32:
        raise TypeError("positions int32, slot_mapping int64, cos_sin float32")
    if q_out is None:
        q_out = torch.empty_like(q)
    desc = cache_desc(k_cache)
    st = lib().pkv_rope_kv_append(_ptr(q), _ptr(k), _ptr(v), _ptr(positions), _ptr(cos_sin), int(cos_sin.shape[0]),
                                  _ptr(slot_mapping), int(k.shape[0]), int(q.shape[1]), _ptr(k_cache),
                                  _ptr(v_cache), ctypes.byref(desc), _ptr(q_out), _stream_ptr(stream))
    _check(st, "pkv_rope_kv_append")
    return q_out


# ---------------------------------------------------------------------------
# latent attention

LATENT_NOPE, LATENT_ROPE, LATENT_V = 128, 64, 128


# The smallest ticks are a few microseconds of GPU work, so these checks are written
# for few attribute reads: a tensor's shape, strides or type is read once.

_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


@functools.lru_cache(maxsize=256)
def _latent_desc_of(shape, dtype):
    N, P, R = shape
    return R - LATENT_ROPE, ctypes.byref(LatentDesc(N, P, R - LATENT_ROPE, LATENT_ROPE, _code_of(dtype)))


def _latent_desc(where, cache):
    """The cache's latent_dim and its descriptor, as an argument."""
    if cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError(f"{where}: the latent cache must be a contiguous [num_pages, page_size, latent_dim + 64] tensor")
    return _latent_desc_of(cache.shape, cache.dtype)


def _on_one_device(where, first, *rest) -> int:
    """The index of the CUDA device that every tensor is on (None: not given)."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"{where} needs CUDA tensors")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: all tensors must be on one CUDA device")
    return dev


def _rows_only(where, *last):
    """Refuses views whose last stride is not 1."""
    for x in last:
        if x != 1:
            raise ValueError(f"{where}: tensors of rows must be contiguous in their last dimension")


def _bad_out(where, width):
    return ValueError(f"{where}: out must be a contiguous [T, H, {width}] tensor of q's dtype, lse a contiguous "
                      "float32 tensor [T, H]")


def _lent(t, stream):
    """A tensor allocated here for a call on `stream`: its memory is not handed
    out again before that stream's work on it is done."""
    if stream is not None:
        t.record_stream(stream)
    return t


def latent_append(c_kv, k_rope, positions, cos_sin, slot_mapping, cache, q_rope=None, q_out=None, stream=None):
    """Write new tokens into a latent cache, rotating on the way (pkv_latent_append).

    c_kv [T, latent_dim] and k_rope [T, 64] (strided rows allowed), positions
    int32 [T], cos_sin float32 [max_pos, 32, 2] (rope_table), slot_mapping int64
    [T], cache [N, P, latent_dim + 64]. With q_rope [T, H, 64] its rotation goes
    to q_out (strided views allowed; q_out may be q_rope; a new tensor when it is
    None). Returns q_out (None without q_rope)."""
    torch = _torch or _load_torch()
    where = "latent_append"
    latent_dim, desc = _latent_desc(where, cache)
    dev = _on_one_device(where, cache, c_kv, k_rope, positions, cos_sin, slot_mapping, q_rope, q_out)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return latent_append(c_kv, k_rope, positions, cos_sin, slot_mapping, cache, q_rope, q_out, stream)
    if (positions.dtype is not torch.int32 or slot_mapping.dtype is not torch.int64
            or cos_sin.dtype is not torch.float32):
        raise TypeError(f"{where}: positions int32, slot_mapping int64, cos_sin float32")
    if not (positions.is_contiguous() and slot_mapping.is_contiguous() and cos_sin.is_contiguous()):
        raise ValueError(f"{where}: positions, slot_mapping and cos_sin must be contiguous")
    dtype, tokens, table = cache.dtype, slot_mapping.shape, cos_sin.shape
    if len(tokens) != 1 or positions.shape != tokens or len(table) != 3 or table[1:] != (LATENT_ROPE // 2, 2):
        raise ValueError(f"{where}: positions and slot_mapping must be [T], cos_sin [max_pos, {LATENT_ROPE // 2}, 2]")
    T, = tokens
    if (c_kv.dtype is not dtype or k_rope.dtype is not dtype or c_kv.shape != (T, latent_dim)
            or k_rope.shape != (T, LATENT_ROPE)):
        raise ValueError(f"{where}: c_kv must be [T, {latent_dim}], k_rope [T, {LATENT_ROPE}], of the cache's dtype")
    (c_st, c_1), (kr_st, kr_1) = c_kv.stride(), k_rope.stride()
    _rows_only(where, c_1, kr_1)
    q = qo = None
    q_st = q_sh = qo_st = qo_sh = H = 0
    if q_rope is not None:
        shape = q_rope.shape
        if q_out is None:
            q_out = _lent(torch.empty(shape, dtype=dtype, device=q_rope.device), stream)
        if (q_rope.dtype is not dtype or q_out.dtype is not dtype or len(shape) != 3 or shape[0] != T
                or shape[2] != LATENT_ROPE or q_out.shape != shape):
            raise ValueError(f"{where}: q_rope and q_out must be [T, H, {LATENT_ROPE}] of the cache's dtype")
        H = shape[1]
        (q_st, q_sh, q_1), (qo_st, qo_sh, qo_1) = q_rope.stride(), q_out.stride()
        _rows_only(where, q_1, qo_1)
        if (T > 1 and qo_st == 0) or (H > 1 and qo_sh == 0):
            raise ValueError(f"{where}: q_out must not be a broadcast view")
        if H == 1:
            q_sh = qo_sh = 0
        q, qo = q_rope.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError(f"{where}: q_out without q_rope")
    if T == 1:   # (a dimension of one entry may have any stride)
        c_st = kr_st = q_st = qo_st = 0
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = lib().pkv_latent_append(c_kv.data_ptr(), c_st, k_rope.data_ptr(), kr_st, q, q_st, q_sh, qo, qo_st, qo_sh, H,
                                 positions.data_ptr(), cos_sin.data_ptr(), table[0], slot_mapping.data_ptr(), T,
                                 cache.data_ptr(), desc, on)
    if st:
        _check(st, "pkv_latent_append")
    return q_out


def latent_gather(cache, page_tables, cu_seqlens_k, total_k: int, out=None, stream=None):
    """Cached rows of every sequence, packed (pkv_latent_gather): out [total_k,
    latent_dim + 64], sequence b in rows cu_seqlens_k[b] .. cu_seqlens_k[b + 1].
    out[:, :latent_dim] is what the up-projection reads, out[:, latent_dim:] the
    k_rope of latent_prefill."""
    torch = _torch or _load_torch()
    where = "latent_gather"
    latent_dim, desc = _latent_desc(where, cache)
    if page_tables.dtype is not torch.int32 or cu_seqlens_k.dtype is not torch.int32:
        raise TypeError(f"{where}: index tensors must be int32")
    dev = _on_one_device(where, cache, page_tables, cu_seqlens_k, out)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return latent_gather(cache, page_tables, cu_seqlens_k, total_k, out, stream)
    tables, cu = page_tables.shape, cu_seqlens_k.shape
    if len(tables) != 2 or len(cu) != 1 or not 1 <= cu[0] <= tables[0] + 1:
        raise ValueError(f"{where}: page_tables [B, W] and cu_seqlens_k [B + 1] disagree")
    if not (page_tables.is_contiguous() and cu_seqlens_k.is_contiguous()):
        raise ValueError(f"{where}: index tensors must be contiguous")
    total_k, R = int(total_k), latent_dim + LATENT_ROPE
    if out is None:
        out = _lent(torch.empty((total_k, R), dtype=cache.dtype, device=cache.device), stream)
    elif out.dtype is not cache.dtype or out.shape != (total_k, R) or not out.is_contiguous():
        raise ValueError(f"{where}: out must be a contiguous [total_k, {R}] tensor of the cache's dtype")
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = lib().pkv_latent_gather(cache.data_ptr(), desc, page_tables.data_ptr(), tables[1], cu_seqlens_k.data_ptr(),
                                 cu[0] - 1, total_k, out.data_ptr(), on)
    if st:
        _check(st, "pkv_latent_gather")
    return out


def latent_workspace_size(num_seqs: int, total_q: int, num_q_heads: int, cache) -> int:
    _, desc = _latent_desc("latent_workspace_size", cache)
    n = lib().pkv_latent_attention_workspace_size(int(num_seqs), int(total_q), int(num_q_heads), desc)
    if n == 0:
        raise PagedKVError(-3, "pkv_latent_attention_workspace_size")
    return int(n)


def alloc_latent_workspace(num_seqs: int, total_q: int, num_q_heads: int, cache):
    import torch
    return torch.empty(latent_workspace_size(num_seqs, total_q, num_q_heads, cache), dtype=torch.uint8,
                       device=cache.device)


def latent_attention(q, cu_seqlens_q, kv_lens, page_tables, cache, scale: float, max_kv_len: int, out=None,
                     lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Absorbed latent attention over the pages (pkv_latent_attention).

    q [T, H, latent_dim + 64] (cache dtype), cu_seqlens_q int32 [B + 1], kv_lens
    int32 [B], page_tables int32 [B, W], cache [N, P, latent_dim + 64]. Returns
    (out [T, H, latent_dim], lse [T, H])."""
    torch = _torch or _load_torch()
    where = "latent_attention"
    width, desc = _latent_desc(where, cache)
    i32, dtype = torch.int32, cache.dtype
    if cu_seqlens_q.dtype is not i32 or kv_lens.dtype is not i32 or page_tables.dtype is not i32:
        raise TypeError(f"{where}: index tensors must be int32")
    if q.dtype is not dtype:
        raise TypeError(f"{where}: q and cache must share one dtype")
    dev = _on_one_device(where, q, cu_seqlens_q, kv_lens, page_tables, cache, out, lse, workspace)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return latent_attention(q, cu_seqlens_q, kv_lens, page_tables, cache, scale, max_kv_len, out, lse, workspace,
                                    want_lse, stream)
    shape, tables, cu, lens = q.shape, page_tables.shape, cu_seqlens_q.shape, kv_lens.shape
    if len(shape) != 3 or shape[2] != width + LATENT_ROPE or not q.is_contiguous():
        raise ValueError(f"{where}: q must be a contiguous [T, H, {width + LATENT_ROPE}] tensor")
    T, H, _ = shape
    if len(cu) != 1 or len(lens) != 1 or len(tables) != 2 or not 0 <= cu[0] - 1 <= min(lens[0], tables[0]):
        raise ValueError(f"{where}: cu_seqlens_q [B + 1], kv_lens [B] and page_tables [B, W] disagree")
    if not (cu_seqlens_q.is_contiguous() and kv_lens.is_contiguous() and page_tables.is_contiguous()):
        raise ValueError(f"{where}: index tensors must be contiguous")
    B = cu[0] - 1
    if out is None:
        out = _lent(torch.empty((T, H, width), dtype=dtype, device=q.device), stream)
    elif out.dtype is not dtype or out.shape != (T, H, width) or not out.is_contiguous():
        raise _bad_out(where, width)
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, H) or not lse.is_contiguous():
            raise _bad_out(where, width)
    elif want_lse:
        lse = _lent(torch.empty((T, H), dtype=torch.float32, device=q.device), stream)
    if workspace is None:
        workspace = _lent(alloc_latent_workspace(B, T, H, cache), stream)
    elif not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace must be contiguous")
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = lib().pkv_latent_attention(q.data_ptr(), cu_seqlens_q.data_ptr(), kv_lens.data_ptr(), page_tables.data_ptr(), B,
                                    T, H, tables[1], int(max_kv_len), cache.data_ptr(), desc, scale, out.data_ptr(),
                                    None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, on)
    if st:
        _check(st, "pkv_latent_attention")
    return out, lse


def latent_prefill_workspace_size(num_seqs: int, total_q: int, num_heads: int) -> int:
    n = lib().pkv_latent_prefill_workspace_size(int(num_seqs), int(total_q), int(num_heads))
    if n == 0:
        raise PagedKVError(-3, "pkv_latent_prefill_workspace_size")
    return int(n)


def alloc_latent_prefill_workspace(num_seqs: int, q):
    import torch
    return torch.empty(latent_prefill_workspace_size(num_seqs, q.shape[0], q.shape[1]), dtype=torch.uint8,
                       device=q.device)


def latent_prefill(q, cu_seqlens_q, k_nope, v, k_rope, cu_seqlens_k, scale: float, out=None, lse=None,
                   workspace=None, want_lse: bool = True, stream=None):
    """Expanded latent attention of chunks over packed keys (pkv_latent_prefill).

    q [Tq, H, 192]; k_nope and v [Tk, H, 128], k_rope [Tk, 64] (strided rows
    allowed: views of the up-projection's output and of the gathered rows);
    cu_seqlens_q, cu_seqlens_k int32 [B + 1]. Returns (out [Tq, H, 128], lse [Tq, H])."""
    torch = _torch or _load_torch()
    where = "latent_prefill"
    if cu_seqlens_q.dtype is not torch.int32 or cu_seqlens_k.dtype is not torch.int32:
        raise TypeError(f"{where}: index tensors must be int32")
    dev = _on_one_device(where, q, cu_seqlens_q, k_nope, v, k_rope, cu_seqlens_k, out, lse, workspace)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return latent_prefill(q, cu_seqlens_q, k_nope, v, k_rope, cu_seqlens_k, scale, out, lse, workspace, want_lse,
                                  stream)
    shape, dtype, rope, cu = q.shape, q.dtype, k_rope.shape, cu_seqlens_q.shape
    if len(shape) != 3 or shape[2] != LATENT_NOPE + LATENT_ROPE or not q.is_contiguous():
        raise ValueError(f"{where}: q must be a contiguous [T, H, {LATENT_NOPE + LATENT_ROPE}] tensor")
    if len(cu) != 1 or cu[0] < 1 or cu_seqlens_k.shape != cu:
        raise ValueError(f"{where}: cu_seqlens_q and cu_seqlens_k must both be [B + 1]")
    if not (cu_seqlens_q.is_contiguous() and cu_seqlens_k.is_contiguous()):
        raise ValueError(f"{where}: index tensors must be contiguous")
    Tq, H, _ = shape
    B, Tk = cu[0] - 1, rope[0] if len(rope) == 2 else -1
    if Tk < 0 or rope[1] != LATENT_ROPE or k_nope.shape != (Tk, H, LATENT_NOPE) or v.shape != (Tk, H, LATENT_V):
        raise ValueError(f"{where}: k_nope, v [Tk, H, 128] and k_rope [Tk, 64] disagree")
    if k_nope.dtype is not dtype or v.dtype is not dtype or k_rope.dtype is not dtype:
        raise ValueError(f"{where}: q, k_nope, v and k_rope must share one dtype")
    (kn_st, kn_sh, kn_1), (v_st, v_sh, v_1), (kr_st, kr_1) = k_nope.stride(), v.stride(), k_rope.stride()
    _rows_only(where, kn_1, v_1, kr_1)
    if Tk == 1:   # (a dimension of one entry may have any stride)
        kn_st = v_st = kr_st = 0
    if H == 1:
        kn_sh = v_sh = 0
    if out is None:
        out = _lent(torch.empty((Tq, H, LATENT_V), dtype=dtype, device=q.device), stream)
    elif out.dtype is not dtype or out.shape != (Tq, H, LATENT_V) or not out.is_contiguous():
        raise _bad_out(where, LATENT_V)
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (Tq, H) or not lse.is_contiguous():
            raise _bad_out(where, LATENT_V)
    elif want_lse:
        lse = _lent(torch.empty((Tq, H), dtype=torch.float32, device=q.device), stream)
    if workspace is None:
        workspace = _lent(alloc_latent_prefill_workspace(B, q), stream)
    elif not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace must be contiguous")
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = lib().pkv_latent_prefill(q.data_ptr(), cu_seqlens_q.data_ptr(), k_nope.data_ptr(), kn_st, kn_sh, v.data_ptr(),
                                  v_st, v_sh, k_rope.data_ptr(), kr_st, cu_seqlens_k.data_ptr(), B, Tq, Tk, H,
                                  _code_of(dtype), scale, out.data_ptr(), None if lse is None else lse.data_ptr(),
                                  workspace.data_ptr(), workspace.nbytes, on)
    if st:
        _check(st, "pkv_latent_prefill")
    return out, lse


# ---------------------------------------------------------------------------
# layers with a window

@functools.lru_cache(maxsize=256)
def _cache_desc_of(shape, dtype):
    """Heads, head_dim, the descriptor as an argument and whether the cache holds codes."""
    if len(shape) != 4:
        raise ValueError("a cache must be [num_pages, page_size, num_kv_heads, head_dim]")
    return shape[2], shape[3], ctypes.byref(CacheDesc(*shape, _code_of(dtype))), _code_of(dtype) == PKV_FP8_E4M3


def _bad_device(where, dev):
    return ValueError(f"{where} needs CUDA tensors" if dev < 0 else f"{where}: all tensors must be on one CUDA device")


def _caches(where, k_cache, v_cache):
    shape, dtype = k_cache.shape, k_cache.dtype
    if v_cache.dtype is not dtype or v_cache.shape != shape or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError(f"{where}: k_cache and v_cache must be contiguous and share one shape [num_pages, page_size, "
                         "num_kv_heads, head_dim] and one dtype")
    return _cache_desc_of(shape, dtype)


def _scales(where, k_scale, v_scale, heads, dev, codes):
    """Pointers of an e4m3 cache's scales."""
    if not codes or k_scale is None or v_scale is None:
        raise ValueError(f"{where}: an e4m3 cache needs k_scale and v_scale, other caches take none")
    for t in (k_scale, v_scale):
        if t.get_device() != dev:
            raise _bad_device(where, dev)
        if t.dtype is not _torch.float32 or t.shape != (heads,) or not t.is_contiguous():
            raise ValueError(f"{where}: scales must be contiguous float32 [num_kv_heads]")
    return k_scale.data_ptr(), v_scale.data_ptr()


def _heads(where, name, t, dtype, T, H, D):
    """Strides of tokens and heads of [T, H, D] rows."""
    if t.dtype is not dtype or t.shape != (T, H, D):
        raise ValueError(f"{where}: {name} must be [{T}, {H}, {D}] of dtype {dtype}")
    st, sh, s1 = t.stride()
    if s1 != 1:
        raise ValueError(f"{where}: {name} must be contiguous in its last dimension")
    # (a dimension of one entry may have any stride)
    return (st if T > 1 else 0), (sh if H > 1 else 0)


def norm_rope_kv_append(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, k_scale=None, v_scale=None, q_out=None,
                        stream=None):
    """Norm queries and keys per head, rotate them, and append keys and values, in one
    pass (pkv_norm_rope_kv_append).

    q [T, Hq, d], k and v [T, Hkv, d] of one dtype (strided views allowed); q_weight,
    k_weight [d] of that dtype or None (not normed); cos_sin float32 [max_pos, r / 2, 2]
    (rope_table, rope_table_scaled): the first r values of a head are rotated, in pairs
    r / 2 apart or, interleaved, of neighbours; positions int32 [T]; slot_mapping int64 [T];
    caches [N, P, Hkv, d] of that dtype, or e4m3 codes with float32 scales [Hkv]. The
    queries go to q_out (strided views allowed; q_out may be q; a new tensor when it is
    None). Returns q_out."""
    torch = _torch or _load_torch()
    where = "norm_rope_kv_append"
    dev = q.get_device()
    if (dev < 0 or k.get_device() != dev or v.get_device() != dev or positions.get_device() != dev
            or cos_sin.get_device() != dev or slot_mapping.get_device() != dev or k_cache.get_device() != dev
            or v_cache.get_device() != dev or (q_out is not None and q_out.get_device() != dev)):
        raise _bad_device(where, dev)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return norm_rope_kv_append(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight,
                                       eps, interleaved, k_scale, v_scale, q_out, stream)
    Hkv, D, _, codes = _caches(where, k_cache, v_cache)
    ks = vs = qw = kw = 0
    if codes or k_scale is not None or v_scale is not None:
        ks, vs = _scales(where, k_scale, v_scale, Hkv, dev, codes)
    if (positions.dtype is not torch.int32 or slot_mapping.dtype is not torch.int64
            or cos_sin.dtype is not torch.float32):
        raise TypeError(f"{where}: positions int32, slot_mapping int64, cos_sin float32")
    if not (positions.is_contiguous() and slot_mapping.is_contiguous() and cos_sin.is_contiguous()):
        raise ValueError(f"{where}: positions, slot_mapping and cos_sin must be contiguous")
    dtype, tokens, table = q.dtype, slot_mapping.shape, cos_sin.shape
    if not codes and dtype is not k_cache.dtype:
        raise TypeError(f"{where}: q, k, v and the caches must share one dtype (but for e4m3 caches)")
    if len(tokens) != 1 or positions.shape != tokens or len(table) != 3 or table[2] != 2:
        raise ValueError(f"{where}: positions and slot_mapping must be [T], cos_sin [max_pos, r / 2, 2]")
    T, = tokens
    if q.dim() != 3:
        raise ValueError(f"{where}: q must be [T, Hq, {D}]")
    Hq = q.shape[1]
    if q_out is None:
        q_out = _lent(torch.empty(q.shape, dtype=dtype, device=q.device), stream)
    qo_t, qo_h = _heads(where, "q_out", q_out, dtype, T, Hq, D)
    if (T > 1 and qo_t == 0) or (Hq > 1 and qo_h == 0):
        raise ValueError(f"{where}: q_out must not be a broadcast view")
    q_t, q_h = _heads(where, "q", q, dtype, T, Hq, D)
    k_t, k_h = _heads(where, "k", k, dtype, T, Hkv, D)
    v_t, v_h = _heads(where, "v", v, dtype, T, Hkv, D)
    for w in (q_weight, k_weight):
        if w is not None:
            if w.get_device() != dev:
                raise _bad_device(where, dev)
            if w.dtype is not dtype or w.shape != (D,) or not w.is_contiguous():
                raise ValueError(f"{where}: norm weights must be contiguous [{D}] of q's dtype")
    if q_weight is not None:
        qw = q_weight.data_ptr()
    if k_weight is not None:
        kw = k_weight.data_ptr()
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    args = _NORM_ROPE_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), q_t, q_h, k_t, k_h, v_t, v_h, qo_t, qo_h, qw, kw,
        positions.data_ptr(), cos_sin.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ks, vs,
        _code_of(dtype), T, Hq, table[0], 2 * table[1], 1 if interleaved else 0, eps, *k_cache.shape,
        _code_of(k_cache.dtype))
    st = (_lib or lib()).pkv_norm_rope_kv_append(args, on)
    if st:
        _check(st, "pkv_norm_rope_kv_append")
    return q_out


ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def rope_table_scaled(base: float, rotary_dim: int, max_pos: int, kind: str = "plain", factor: float = 1.0,
                      low: float = 1.0, high: float = 32.0, original_max_pos: float = 0.0,
                      attention_factor: float = 0.0) -> np.ndarray:
    """Host cos/sin table [max_pos, rotary_dim/2, 2] float32 of stretched angles
    (pkv_rope_table_scaled): kind "plain", "linear", "base", "bands" or "ramp"."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"rope_table_scaled: kind must be one of {', '.join(ROPE_KINDS)}")
    scaling = RopeScaling(ROPE_KINDS[kind], float(factor), float(low), float(high), float(original_max_pos),
                          float(attention_factor))
    out = np.zeros((max(int(max_pos), 1), max(int(rotary_dim) // 2, 1), 2), dtype=np.float32)
    _check(lib().pkv_rope_table_scaled(float(base), int(rotary_dim), ctypes.byref(scaling), int(max_pos),
                                       out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))), "pkv_rope_table_scaled")
    return out


def window_attention(q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, scale: float, window: int, sinks: int = 0,
                     k_scale=None, v_scale=None, out=None, lse=None, want_lse: bool = True, stream=None):
    """Attention of packed rows over their pages through a sliding window with sinks
    (pkv_window_attention): the row at position p sees the keys p - window + 1 .. p and
    the first `sinks` keys.

    q [T, Hq, d]; cu_seqlens_q int32 [B + 1]; kv_lens int32 [B]; page_tables int32 [B, W];
    caches [N, P, Hkv, d] of q's dtype, or e4m3 codes (q bf16 or f16) with float32 scales
    [Hkv]. out must not overlap q. Returns (out [T, Hq, d], lse [T, Hq])."""
    torch = _torch or _load_torch()
    where = "window_attention"
    i32 = torch.int32
    if cu_seqlens_q.dtype is not i32 or kv_lens.dtype is not i32 or page_tables.dtype is not i32:
        raise TypeError(f"{where}: index tensors must be int32")
    dev = q.get_device()
    if (dev < 0 or cu_seqlens_q.get_device() != dev or kv_lens.get_device() != dev or page_tables.get_device() != dev
            or k_cache.get_device() != dev or v_cache.get_device() != dev
            or (out is not None and out.get_device() != dev) or (lse is not None and lse.get_device() != dev)):
        raise _bad_device(where, dev)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return window_attention(q, cu_seqlens_q, kv_lens, page_tables, k_cache, v_cache, scale, window, sinks,
                                    k_scale, v_scale, out, lse, want_lse, stream)
    Hkv, D, desc, codes = _caches(where, k_cache, v_cache)
    ks = vs = None
    if codes or k_scale is not None or v_scale is not None:
        ks, vs = _scales(where, k_scale, v_scale, Hkv, dev, codes)
    shape, dtype, tables, cu, lens = q.shape, q.dtype, page_tables.shape, cu_seqlens_q.shape, kv_lens.shape
    if not codes and dtype is not k_cache.dtype:
        raise TypeError(f"{where}: q and the caches must share one dtype (but for e4m3 caches)")
    if len(shape) != 3 or shape[2] != D or not q.is_contiguous():
        raise ValueError(f"{where}: q must be a contiguous [T, Hq, {D}] tensor")
    T, Hq, _ = shape
    if len(cu) != 1 or len(lens) != 1 or len(tables) != 2 or not 0 <= cu[0] - 1 <= min(lens[0], tables[0]):
        raise ValueError(f"{where}: cu_seqlens_q [B + 1], kv_lens [B] and page_tables [B, W] disagree")
    if not (cu_seqlens_q.is_contiguous() and kv_lens.is_contiguous() and page_tables.is_contiguous()):
        raise ValueError(f"{where}: index tensors must be contiguous")
    if out is None:
        out = _lent(torch.empty(shape, dtype=dtype, device=q.device), stream)
    elif out.dtype is not dtype or out.shape != shape or not out.is_contiguous():
        raise _bad_out(where, D)
    lse_ptr = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous():
            raise _bad_out(where, D)
        lse_ptr = lse.data_ptr()
    elif want_lse:
        lse = _lent(torch.empty((T, Hq), dtype=torch.float32, device=q.device), stream)
        lse_ptr = lse.data_ptr()
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = (_lib or lib()).pkv_window_attention(
        q.data_ptr(), _code_of(dtype), cu_seqlens_q.data_ptr(), kv_lens.data_ptr(), page_tables.data_ptr(), cu[0] - 1, T,
        Hq, tables[1], _count(window), _count(sinks), k_cache.data_ptr(), v_cache.data_ptr(), desc, ks, vs, scale,
        out.data_ptr(), lse_ptr, on)
    if st:
        _check(st, "pkv_window_attention")
    return out, lse


def copy_pages(caches, src, dst, tokens=None, stream=None):
    """Copy pages within each of several caches of one pool's page ids (pkv_copy_pages).

    caches: contiguous tensors of one size in bytes (keys and values of all layers,
    latent caches), all with the N pages of P slots of the first, [N, P, ...]; src, dst int32
    [n] on their device: page dst[i] gets page src[i] in every cache (negative: no copy),
    with tokens int32 [n] only its first tokens[i] slots. No page may be dst of one copy and
    src or dst of another."""
    torch = _torch or _load_torch()
    where = "copy_pages"
    caches = list(caches)
    if not caches:
        return
    dev = src.get_device()
    devices = {c.get_device() for c in caches}
    devices.add(dst.get_device())
    if dev < 0 or devices != {dev} or (tokens is not None and tokens.get_device() != dev):
        raise _bad_device(where, min(dev, *devices))
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return copy_pages(caches, src, dst, tokens, stream)
    first = caches[0]
    shape = first.shape
    # (sets of all caches' attributes: the cheapest way to compare many of them)
    if len({c.nbytes for c in caches}) != 1 or not all([c.is_contiguous() for c in caches]):
        raise ValueError(f"{where}: caches must be contiguous and of one size in bytes")
    if len(shape) < 3 or 0 in shape:
        raise ValueError(f"{where}: a cache must be [num_pages, page_size, ...]")
    n = src.shape
    if src.dtype is not torch.int32 or dst.dtype is not torch.int32 or (tokens is not None
                                                                       and tokens.dtype is not torch.int32):
        raise TypeError(f"{where}: src, dst and tokens must be int32")
    if len(n) != 1 or dst.shape != n or (tokens is not None and tokens.shape != n):
        raise ValueError(f"{where}: src, dst and tokens must be [n]")
    if not (src.is_contiguous() and dst.is_contiguous() and (tokens is None or tokens.is_contiguous())):
        raise ValueError(f"{where}: src, dst and tokens must be contiguous")
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    ptrs = array.array("Q", [c.data_ptr() for c in caches])
    st = lib().pkv_copy_pages(ptrs.buffer_info()[0], len(ptrs), shape[0], shape[1], first.nbytes // (shape[0] * shape[1]),
                              src.data_ptr(), dst.data_ptr(), _ptr(tokens), n[0], on)
    if st:
        _check(st, "pkv_copy_pages")


def remap_pages(page_tables, page_map, stream=None):
    """Rewrite page tables in place for pages that have moved (pkv_remap_pages): entry
    e >= 0 becomes page_map[e]. page_tables int32 (any shape, contiguous), page_map int32
    [num_pages]. Returns page_tables."""
    torch = _torch or _load_torch()
    where = "remap_pages"
    dev = _on_one_device(where, page_tables, page_map)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return remap_pages(page_tables, page_map, stream)
    if page_tables.dtype is not torch.int32 or page_map.dtype is not torch.int32:
        raise TypeError(f"{where}: page_tables and page_map must be int32")
    if page_map.dim() != 1 or not (page_tables.is_contiguous() and page_map.is_contiguous()):
        raise ValueError(f"{where}: page_tables and page_map [num_pages] must be contiguous")
    on = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    st = lib().pkv_remap_pages(page_tables.data_ptr(), page_tables.numel(), page_map.data_ptr(), page_map.shape[0], on)
    if st:
        _check(st, "pkv_remap_pages")
    return page_tables


def selftest_bounded_wait(limit_us: int, result=None, stream=None) -> None:
    """Enqueue the failure-path self-test (pkv_selftest_bounded_wait): a CTA laid
    out like the prefill kernel's waits on barriers that nothing completes; the
    producer warp gives up after ~limit_us and sets PKV_DEV_TIMEOUT, the other
    warps drain through the abort flag. `result`: optional device int32 [2]
    tensor (error word, warps that returned)."""
    if result is not None:
        import torch
        if not result.is_cuda or result.dtype != torch.int32 or result.numel() < 2 or not result.is_contiguous():
            raise ValueError("selftest_bounded_wait: result must be a contiguous int32 CUDA tensor of 2 entries")
    _check(lib().pkv_selftest_bounded_wait(int(limit_us), _ptr(result), _stream_ptr(stream)),
           "pkv_selftest_bounded_wait")


def device_status(stream=None) -> int:
    """OR of the device status bits since the last call (then cleared)."""
    code = ctypes.c_int32(0)
    _check(lib().pkv_get_device_status(ctypes.byref(code), _stream_ptr(stream)), "pkv_get_device_status")
    return int(code.value)


def set_kernel_timing(enable: bool):
    _check(lib().pkv_set_kernel_timing(1 if enable else 0), "pkv_set_kernel_timing")


def kernel_times(max_kernels: int = 32):
    """{kernel name: (launches, total ms)} recorded since the last call."""
    names = (ctypes.c_char_p * max_kernels)()
    launches = (ctypes.c_int32 * max_kernels)()
    total = (ctypes.c_double * max_kernels)()
    n = lib().pkv_kernel_times(names, launches, total, max_kernels)
    if n < 0:
        raise PagedKVError(n, "pkv_kernel_times")
    return {names[i].decode(): (int(launches[i]), float(total[i])) for i in range(n)}


# ---------------------------------------------------------------------------
# host page pool and prefix cache

class PagePool:
    """The library's host page pool (pkv_pool_*, pkv_prefix_*)."""

    def __init__(self, num_pages: int, page_size: int):
        self._h = ctypes.c_void_p()
        _check(lib().pkv_pool_create(int(num_pages), int(page_size), ctypes.byref(self._h)), "pkv_pool_create")
        self.num_pages, self.page_size = int(num_pages), int(page_size)

    def close(self):
        if self._h:
            lib().pkv_pool_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _arr(xs):
        a = np.ascontiguousarray(np.asarray(xs, dtype=np.int32))
        return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def alloc(self, n: int):
        a = np.zeros(max(n, 1), dtype=np.int32)
        _check(lib().pkv_pool_alloc(self._h, int(n), a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))), "pkv_pool_alloc")
        return [int(x) for x in a[:n]]

    def retain(self, pages):
        a, p = self._arr(pages)
        _check(lib().pkv_pool_retain(self._h, p, len(a)), "pkv_pool_retain")

    def release(self, pages):
        a, p = self._arr(pages)
        _check(lib().pkv_pool_release(self._h, p, len(a)), "pkv_pool_release")

    def free_count(self) -> int:
        return int(lib().pkv_pool_free_count(self._h))

    def refcount(self, page: int) -> int:
        r = lib().pkv_pool_refcount(self._h, int(page))
        if r < 0:
            raise PagedKVError(r, "pkv_pool_refcount")
        return int(r)

    def lookup(self, tokens, now: float, max_pages: int = 1 << 20):
        t, tp = self._arr(tokens if len(tokens) else [0])
        n_max = min(max_pages, len(tokens) // self.page_size)
        out = np.zeros(max(n_max, 1), dtype=np.int32)
        n = lib().pkv_prefix_lookup(self._h, tp, len(tokens), float(now),
                                    out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(n_max))
        if n < 0:
            raise PagedKVError(n, "pkv_prefix_lookup")
        return [int(x) for x in out[:n]]

    def insert(self, tokens, pages, now: float) -> int:
        t, tp = self._arr(tokens if len(tokens) else [0])
        a, ap = self._arr(pages if len(pages) else [0])
        n = lib().pkv_prefix_insert(self._h, tp, len(tokens), ap, len(pages), float(now))
        if n < 0:
            raise PagedKVError(n, "pkv_prefix_insert")
        return int(n)

    def evict(self, now: float, ttl: float, want_free: int = 0) -> int:
        n = lib().pkv_prefix_evict(self._h, float(now), float(ttl), int(want_free))
        if n < 0:
            raise PagedKVError(n, "pkv_prefix_evict")
        return int(n)

    def cache_size(self) -> int:
        return int(lib().pkv_prefix_size(self._h))

    # A call of these changes nothing when it raises.

    def fork(self, pages, kv_len: int, window: Optional[int] = None, sinks: int = 0):
        """Pages of a sequence forked after kv_len tokens (pkv_pool_fork): (the child's
        pages, None or the (src, dst, tokens) that copy_pages has to copy). With a `window`
        (pkv_pool_fork_window) a -1 page that the child's next rows see is refused."""
        a, p = self._arr(pages if len(pages) else [0])
        used = -(-int(kv_len) // self.page_size)
        child, cp = self._arr(np.zeros(max(used, len(pages), 1)))
        what = np.zeros(3, dtype=np.int32)
        P32 = ctypes.POINTER(ctypes.c_int32)
        at = [what[i:].ctypes.data_as(P32) for i in range(3)]
        if window is None:
            n = lib().pkv_pool_fork(self._h, p, len(pages), int(kv_len), cp, *at)
        else:
            n = lib().pkv_pool_fork_window(self._h, p, len(pages), int(kv_len), _count(int(window)), _count(int(sinks)), cp,
                                           *at)
        if n < 0:
            raise PagedKVError(n, "pkv_pool_fork" if window is None else "pkv_pool_fork_window")
        return [int(x) for x in child[:used]], (tuple(int(x) for x in what) if n else None)

    def compact(self, max_moves: int = 1 << 30):
        """Move held pages to the lowest free ids (pkv_pool_compact): int32 arrays src,
        dst of the moves and page_map [num_pages], for copy_pages and remap_pages."""
        m = max(min(int(max_moves), self.num_pages), 0) if max_moves >= 0 else int(max_moves)
        src, sp = self._arr(np.zeros(max(m, 1)))
        dst, dp = self._arr(np.zeros(max(m, 1)))
        page_map, mp = self._arr(np.zeros(self.num_pages))
        n = lib().pkv_pool_compact(self._h, m, sp, dp, mp)
        if n < 0:
            raise PagedKVError(n, "pkv_pool_compact")
        return src[:n], dst[:n], page_map

    def trim(self, pages, kv_len: int, window: int, sinks: int = 0):
        """Let go of the pages that no row at position kv_len or later sees through a
        window with sinks (pkv_pool_trim): the list with -1 in their places."""
        a, p = self._arr(pages if len(pages) else [0])
        a = a.copy()
        n = lib().pkv_pool_trim(self._h, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(pages), int(kv_len),
                                _count(int(window)), _count(int(sinks)))
        if n < 0:
            raise PagedKVError(n, "pkv_pool_trim")
        return [int(x) for x in a[:len(pages)]]
