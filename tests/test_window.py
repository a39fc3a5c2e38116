"""Layers with a window: the oracle against torch and closed forms, the calls' refusals
and the host pool's forks, compaction and trimming, and (GPU) norm, rotation and append,
window attention and page copies against the oracle in 64 bits, alone and as a serving
loop runs them.

Tolerances. u is half a step of the stored type (bf16 2^-8, f16 2^-11, f32 2^-24), up
half a step of the softmax weights' type (bf16 caches 2^-8; f16 and e4m3 caches f16 2^-11;
f32: not rounded). A score is an fp32 sum of D products, off by at most D 2^-23 scale
sum_d |q_d k_d| =: ds (2^-23: the tensor core may truncate), which moves every weight by a
factor exp(+-ds) before and, through the sum, as much after: 2 ds sum_j w_j |v_j|. f16
weights carry a power of two of at least 2^7: below 2^-14 they are off by up to 2^-25, so by
2^-32 of the largest weight, max|v| a key. Over e4m3 caches bf16 queries go to f16 with their
largest value at 2^8 or above: what falls below f16's normal range is off by 2^-25, 2^-33 of
that value, each channel. The output's fp32 sums over L keys add at most (L + 64) 2^-23 of
sum_j w_j |v_j|, the exponentials' and the final scaling's errors stay below 2^-20. lse moves
by ds, by its sum's relative error (L + 64) 2^-23, and by 2^-20 plus two roundings of its size.

Norm and rotation: the fp32 sum of D squares is off by at most D 2^-24, half of it after
the root; root, two products, the rotation's two products and sum are one rounding each: (D / 2
+ 8) 2^-24 of the size of what is added, and u of the result.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as F
from oracle import window as O
from paged_kv_attention_mapping_gb300 import binding

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"f32": binding.PKV_F32, "f16": binding.PKV_F16, "bf16": binding.PKV_BF16, "e4m3": binding.PKV_FP8_E4M3}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
# f16's steps below 2^-14 are 2^-24 whatever the value, half of one is 2^-25: not u |x|
# (bf16 and f32 have fp32's exponents)
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
UP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -11, "f32": 0.0}


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_mapping_gb300 import build
    build.build()
    return binding.lib()


@pytest.fixture(scope="module")
def dev(lib):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    binding.device_status()
    return d


# ---------------------------------------------------------------------------
# oracle pins (CPU)

@pytest.mark.parametrize("n,L,W,S", [(1, 1, 1, 0), (5, 11, 3, 0), (5, 11, 3, 2), (11, 11, 4, 1), (3, 20, 100, 7), (4, 9, 1, 9)])
def test_oracle_attention_matches_torch(n, L, W, S):
    g = np.random.default_rng(n * 100 + L)
    q, k, v = g.standard_normal((n, 6, 16)), g.standard_normal((L, 2, 16)), g.standard_normal((L, 2, 16))
    mask = torch.ones(n, L, dtype=torch.bool).tril(L - n)
    mask &= torch.ones(n, L, dtype=torch.bool).triu(L - n - W + 1) | (torch.arange(L) < S)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).transpose(0, 1)
    kk, vv = (t(x).repeat_interleave(3, 0) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(t(q), kk, vv, mask, scale=0.3).transpose(0, 1)
    lse = torch.logsumexp((0.3 * t(q) @ kk.transpose(1, 2)).masked_fill(~mask, -math.inf), -1).T
    out, got, mass, dot = O.attend(q, k, v, 0.3, W, S)
    assert np.abs(out - want.numpy()).max() < 1e-12 and np.abs(got - lse.numpy()).max() < 1e-12
    assert (mass + 1e-12 >= np.abs(out)).all() and (dot >= 0).all()


def test_oracle_attention_reads_only_what_is_seen():
    g = np.random.default_rng(0)
    k, v = g.standard_normal((20, 1, 8)), g.standard_normal((20, 1, 8))
    k[2:13], v[2:13] = np.nan, np.nan
    out, lse, _, _ = O.attend(g.standard_normal((3, 2, 8)), k, v, 1.0, 5, 2)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    out, lse, _, _ = O.attend(np.ones((1, 1, 8)), k, v, 1.0, 1, 0)   # one key: its value
    assert np.array_equal(out[0, 0], v[19, 0]) and np.isclose(lse[0, 0], k[19, 0].sum())


def test_oracle_norm_and_rotation():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    assert np.allclose(O.norm(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0), [[[1.2, 3.2, 0.0, 0.0]]])
    assert O.norm(x, None, 1.0) is not None and np.array_equal(O.norm(x, None, 1.0), x)
    quarter = np.array([[[0.0, 1.0], [0.0, 1.0]]])        # a turn by 90 degrees: (a, b) -> (-b, a)
    y = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    assert np.allclose(O.rotate(y, quarter, False)[0], [[[-3.0, -4.0, 1.0, 2.0, 5.0]]])
    assert np.allclose(O.rotate(y, quarter, True)[0], [[[-2.0, 1.0, -4.0, 3.0, 5.0]]])


# ---------------------------------------------------------------------------
# tables of the rotation (CPU)

@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("plain", dict(attention_factor=0.5)), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("bands", dict(factor=8.0, low=1.0, high=4.0, original_max_pos=8192)),
    ("ramp", dict(factor=4.0, low=1.0, high=32.0, original_max_pos=4096)),
    ("ramp", dict(factor=16.0, low=1.0, high=1.5, original_max_pos=64, attention_factor=1.0)),
    ("ramp", dict(factor=1.0, low=1.0, high=32.0, original_max_pos=1))])
@pytest.mark.parametrize("r,base", [(16, 10000.0), (64, 500000.0), (128, 1e6)])
def test_tables_match_the_definitions(lib, r, base, kind, kw):
    got = binding.rope_table_scaled(base, r, 300, kind, **kw)
    a = dict(factor=1.0, low=1.0, high=32.0, original_max_pos=0.0, attention_factor=0.0)
    a.update(kw)
    f, m = O.angles(base, r, kind, a["factor"], a["low"], a["high"], a["original_max_pos"], a["attention_factor"])
    p = np.arange(300)[:, None] * f
    # a float's half step; the angles in double are off by a few 2^-53 of up to 300
    want = np.stack([np.cos(p), np.sin(p)], -1) * m
    assert got.shape == want.shape and np.abs(got - want).max() <= 2.0 ** -24 * m + 1e-12
    if kind == "plain" and not kw:
        assert np.array_equal(got, binding.rope_table(base, r, 300))


def test_table_refusals(lib):
    def call(r=64, max_pos=8, kind="ramp", **kw):
        a = dict(factor=2.0, low=1.0, high=2.0, original_max_pos=64.0)
        a.update(kw)
        return binding.rope_table_scaled(a.pop("base", 10000.0), r, max_pos, kind, **a)
    call()
    for bad in (dict(r=63), dict(r=0), dict(max_pos=0), dict(factor=0.5), dict(factor=math.nan), dict(low=0.0),
                dict(low=2.0), dict(high=math.inf), dict(original_max_pos=0.0), dict(attention_factor=-1.0),
                dict(attention_factor=math.nan), dict(base=1.0), dict(base=math.inf), dict(r=2, kind="base")):
        with pytest.raises(binding.PagedKVError):
            call(**bad)
    with pytest.raises(ValueError):
        call(kind="cubic")


# ---------------------------------------------------------------------------
# the page pool and packing (CPU)

def test_fork_shares_full_pages_and_copies_the_last(lib):
    pool = binding.PagePool(8, 4)
    parent = pool.alloc(3)
    child, copy = pool.fork(parent, 10)
    assert child == [0, 1, 3] and copy == (2, 3, 2)
    assert [pool.refcount(i) for i in range(5)] == [2, 2, 1, 1, 0]
    child2, copy2 = pool.fork(parent, 8)                   # ends at a page's end: nothing to copy
    assert child2 == [0, 1] and copy2 is None and pool.refcount(0) == 3
    assert pool.fork(parent, 0) == ([], None)
    pool.release(child)
    pool.release(child2)
    pool.release(parent)
    assert pool.free_count() == 8


def test_fork_of_trimmed_pages(lib):
    pool = binding.PagePool(8, 4)
    parent = pool.trim(pool.alloc(4), 14, 5, 0)            # the next row sees keys 10 .. 14
    assert parent == [-1, -1, 2, 3]
    child, copy = pool.fork(parent, 14)
    assert child == [-1, -1, 2, 0] and copy == (3, 0, 2)


def test_fork_refusals_change_nothing(lib):
    pool = binding.PagePool(4, 4)
    a = pool.alloc(4)
    for pages, n in ((a, 15), (a, 17), ([0, 1, 2, 9], 16), ([0, 1, 2, -1], 15), ([0, 1], -1)):
        with pytest.raises(binding.PagedKVError):
            pool.fork(pages, n)
    assert [pool.refcount(i) for i in range(4)] == [1] * 4
    pool.release([3])
    with pytest.raises(binding.PagedKVError):
        pool.fork([0, 1, 3], 12)                           # a page that nobody holds
    assert pool.fork([0, 1, 2], 10)[1] == (2, 3, 2)


@pytest.mark.parametrize("seed", range(5))
def test_compact_moves_the_highest_pages_down(lib, seed):
    rng = np.random.default_rng(seed)
    N = 40
    pool = binding.PagePool(N, 4)
    pool.alloc(N)
    held = np.flatnonzero(rng.random(N) < 0.4)
    pool.release([i for i in range(N) if i not in held])
    extra = [int(i) for i in held if rng.random() < 0.3]
    pool.retain(extra)
    count = {int(i): 1 + (int(i) in extra) for i in held}
    moves = int(rng.integers(0, 30))
    src, dst, page_map = pool.compact(moves)
    assert len(src) == len(dst) <= moves and not set(src.tolist()) & set(dst.tolist())
    assert all(d < s for s, d in zip(src, dst)) and page_map.tolist() != [] and len(page_map) == N
    want = np.arange(N)
    want[src] = dst
    assert np.array_equal(page_map, want)
    for old, c in count.items():
        assert pool.refcount(int(page_map[old])) == c
    assert pool.free_count() == N - len(held)
    if moves >= len(held):
        assert sorted(page_map[held].tolist()) == list(range(len(held)))
    assert pool.alloc(1)[0] == min(set(range(N)) - {int(page_map[i]) for i in held})


def test_compact_takes_prefix_entries_along(lib):
    pool = binding.PagePool(6, 2)
    pages = pool.alloc(6)
    pool.insert([1, 2, 3, 4], [4, 5], now=0.0)
    pool.release(pages)                                    # only the prefix cache holds 4 and 5
    src, dst, _ = pool.compact()
    assert src.tolist() == [5, 4] and dst.tolist() == [0, 1]
    assert pool.lookup([1, 2, 3, 4], now=1.0) == [1, 0]
    pool.release([0, 1])
    assert pool.evict(now=9.0, ttl=1.0) == 2 and pool.free_count() == 6


@pytest.mark.parametrize("P", [1, 4, 7])
@pytest.mark.parametrize("W,S", [(1, 0), (5, 0), (5, 3), (16, 4), (100, 0)])
def test_trim_keeps_what_a_later_row_sees(lib, P, W, S):
    for L in (0, 1, 5, 16, 23, 24, 40):
        n = -(-(L + 1) // P)
        pool = binding.PagePool(64, P)
        pages = pool.alloc(n)
        got = pool.trim(pages, L, W, S)
        seen = O.visible(1, L + 1, W, S)[0]                # the row at position L
        for j in range(n):
            # (a page of the sinks stays although not all of them may be seen yet)
            keep = seen[j * P:(j + 1) * P].any() or j * P < S
            assert got[j] == (pages[j] if keep else -1), (L, j)
        assert pool.free_count() == 64 - sum(p >= 0 for p in got)
        assert pool.trim(got, L, W, S) == got


def test_trim_refusals_change_nothing(lib):
    pool = binding.PagePool(8, 2)
    a = pool.alloc(4)
    for pages, L, W, S in ((a, 7, 0, 0), (a, 7, 2, -1), (a, -1, 2, 0), ([0, 9, 2, 3], 7, 2, 0), ([0, 0, 0, 3], 7, 2, 0)):
        with pytest.raises(binding.PagedKVError):
            pool.trim(pages, L, W, S)
    assert pool.free_count() == 4 and pool.refcount(0) == 1


def test_packing_takes_freed_pages_behind_the_window(lib):
    kw = dict(page_size=4, num_pages=10)
    a = binding.pack_tick([1, 3], [20, 5], [[0, -1, -1, 3, 4], [7, 8]], window=6, sinks=2, **kw)
    assert a["page_tables"].tolist() == [[0, -1, -1, 3, 4], [7, 8, -1, -1, -1]]
    assert a["slot_mapping"].tolist() == [19, 30, 31, 32]
    # the row at position 19 sees keys 14 .. 19 and 0, 1
    for pages in ([-1, -1, -1, 3, 4], [0, -1, -1, -1, 4], [0, -1, -1, 3, -1], [0, -2, -1, 3, 4], [0, 10, 2, 3, 4]):
        with pytest.raises(binding.PagedKVError):
            binding.pack_tick([1], [20], [pages], window=6, sinks=2, **kw)
    with pytest.raises(binding.PagedKVError):
        binding.pack_tick([1], [20], [[0, -1, -1, 3, 4]], **kw)
    for w, s in ((0, 0), (1, -1)):
        with pytest.raises(binding.PagedKVError):
            binding.pack_tick([1], [4], [[0]], window=w, sinks=s, **kw)
    plain, wide = (binding.pack_tick([2, 1], [9, 4], [[5, 6, 1], [2]], **kw, **x) for x in ({}, dict(window=99)))
    assert all(np.array_equal(plain[k], wide[k]) for k in plain)


# ---------------------------------------------------------------------------
# refusals on the host (no device work happens before them)

FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104)


def _desc(N=4, P=16, H=2, D=64, t="bf16"):
    return binding.CacheDesc(N, P, H, D, CODES[t])


def _append(lib, desc=None, q=FAKE, qs=(512, 64), k=FAKE, ks=(128, 64), v=FAKE, t="bf16", qw=None, kw=None, eps=1e-6,
            pos=FAKE, cs=FAKE, max_pos=8, rot=64, slots=FAKE, T=2, H=8, kc=FAKE, sc=None, qo=FAKE):
    d = desc or _desc()
    at = lambda x: 0 if x is None else x.value
    args = binding._NORM_ROPE_ARGS.pack(at(q), at(k), at(v), at(qo), *qs, *ks, 128, 64, 512, 64, at(qw), at(kw), at(pos),
                                        at(cs), at(slots), at(kc), FAKE.value, at(sc), at(sc), CODES[t], T, H, max_pos, rot,
                                        0, eps, d.num_pages, d.page_size, d.num_kv_heads, d.head_dim, d.dtype)
    return lib.pkv_norm_rope_kv_append(args, None)


def _attend(lib, desc=None, q=FAKE, t="bf16", cu=FAKE, B=1, T=2, H=8, W=4, window=8, sinks=0, kc=FAKE, ks=None, vs=None,
            scale=0.1, out=FAKE, lse=None):
    d = desc or _desc()
    return lib.pkv_window_attention(q, CODES[t], cu, FAKE, FAKE, B, T, H, W, window, sinks, kc, FAKE, ctypes.byref(d), ks,
                                    vs, scale, out, lse, None)


@pytest.mark.parametrize("kw,status", [(dict(N=0), -3), (dict(P=0), -3), (dict(H=0), -3), (dict(D=96), -3), (dict(D=32), -3),
                                       (dict(N=1 << 20, P=1 << 12), -3), (dict(t="f16"), -2)])
def test_bad_caches_are_refused(lib, kw, status):
    assert _append(lib, desc=_desc(**kw)) == status and _attend(lib, desc=_desc(**kw)) == status


def test_append_refusals(lib):
    assert lib.pkv_norm_rope_kv_append(None, None) == -1
    for kw in (dict(T=-1), dict(H=0), dict(H=5000), dict(max_pos=0), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=80),
               dict(eps=-1.0), dict(eps=math.nan), dict(qs=(510, 64)), dict(qs=(512, -64)), dict(ks=(1 << 31, 64))):
        assert _append(lib, **kw) == -3, kw
    for name in ("q", "k", "v", "pos", "cs", "slots", "kc", "qo"):
        assert _append(lib, **{name: None}) == -1, name
    for name in ("q", "k", "v", "qw", "kw", "cs", "kc", "qo"):
        assert _append(lib, **{name: ODD}) == -7, name
    assert _append(lib, slots=ctypes.c_void_p(4100)) == -7 and _append(lib, pos=ctypes.c_void_p(4098)) == -7
    assert _append(lib, sc=FAKE) == -2 and _append(lib, desc=_desc(t="e4m3")) == -1
    assert _append(lib, t="e4m3", desc=_desc(t="e4m3"), sc=FAKE) == -2
    assert _append(lib, T=0) == 0


def test_attention_refusals(lib):
    for kw in (dict(B=-1), dict(T=-1), dict(H=0), dict(H=7), dict(H=18), dict(H=64), dict(W=0), dict(W=1 << 28),
               dict(window=0), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert _attend(lib, **kw) == -3, kw
    assert _attend(lib, q=None) == -1 and _attend(lib, cu=None) == -1 and _attend(lib, out=None) == -1
    assert _attend(lib, q=ODD) == -7 and _attend(lib, out=ODD) == -7 and _attend(lib, kc=ODD) == -7
    assert _attend(lib, lse=ctypes.c_void_p(4098)) == -7
    e4m3 = _desc(t="e4m3")
    assert _attend(lib, desc=e4m3) == -1 and _attend(lib, desc=e4m3, ks=FAKE) == -1
    assert _attend(lib, desc=e4m3, ks=FAKE, vs=FAKE, t="f32") == -2 and _attend(lib, ks=FAKE, vs=FAKE) == -2
    assert _attend(lib, T=0) == 0 and _attend(lib, B=0) == 0


def test_page_call_refusals(lib):
    def copy(caches=(4096, 8192), n=3, pages=8, P=16, slot=256, src=FAKE, dst=FAKE, tokens=None):
        a = (ctypes.c_void_p * max(len(caches), 1))(*caches)
        return lib.pkv_copy_pages(a, len(caches), pages, P, slot, src, dst, tokens, n, None)
    for kw in (dict(n=-1), dict(pages=0), dict(P=0), dict(slot=0), dict(slot=24), dict(pages=1 << 20, P=1 << 12),
               dict(P=1 << 16, slot=1 << 16)):
        assert copy(**kw) == -3, kw
    assert copy(src=None) == -1 and copy(dst=None) == -1 and copy(caches=(4096, None)) == -1
    assert copy(caches=(4096, 4104)) == -7 and copy(tokens=ctypes.c_void_p(4098)) == -7
    assert copy(n=0) == 0 and copy(caches=()) == 0
    remap = lambda t=FAKE, n=4, m=FAKE, pages=8: lib.pkv_remap_pages(t, n, m, pages, None)
    assert remap(n=-1) == -3 and remap(pages=0) == -3 and remap(t=None) == -1 and remap(m=None) == -1
    assert remap(t=ctypes.c_void_p(4098)) == -7 and remap(n=0) == 0


def test_binding_refuses_wrong_tensors(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    kc, q, k = z(4, 16, 2, 64), z(1, 8, 64), z(1, 2, 64)
    cu, kv, pt = torch.tensor([0, 1], dtype=i32), z(1, t=i32), z(1, 1, t=i32)
    with pytest.raises(ValueError):                                        # host tensors
        binding.window_attention(q, cu, kv, pt, kc, kc, 0.1, 4)
    with pytest.raises(TypeError):
        binding.window_attention(q, cu.long(), kv, pt, kc, kc, 0.1, 4)
    with pytest.raises(ValueError):
        binding.norm_rope_kv_append(q, k, k, z(1, t=i32), z(4, 32, 2, t=f32), z(1, t=i64), kc, kc)
    with pytest.raises(ValueError):
        binding.copy_pages([kc], z(1, t=i32), z(1, t=i32))
    with pytest.raises(ValueError):
        binding.remap_pages(pt, z(4, t=i32))
    assert binding.copy_pages([], None, None) is None


# ---------------------------------------------------------------------------
# GPU

def _cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _host(t):
    return t.double().cpu().numpy()


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


class Problem:
    """Sequences over scattered pages. Slots that no row sees hold NaN, and tables are -1
    where no row sees a key of the page."""

    def __init__(self, dev, t, cache, Hq, Hkv, D, P, W, S, q_lens, kv_lens, seed=0, spread=1.0, pad=0):
        self.__dict__.update(dev=dev, t=t, cache=cache, Hq=Hq, Hkv=Hkv, D=D, P=P, W=W, S=S, q_lens=list(q_lens),
                             kv_lens=list(kv_lens), scale=spread / math.sqrt(D), pad=pad)
        g = torch.Generator(device="cpu").manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-L // P) for L in kv_lens]
        self.N = sum(need) + 2
        perm = rng.permutation(self.N).astype(np.int32)
        self.tables = np.full((len(q_lens), max(max(need), 1)), -1, np.int32)
        self.seen = np.zeros((self.N, P), bool)
        at = 0
        for b, (n, L) in enumerate(zip(q_lens, kv_lens)):
            ids = perm[at:at + need[b]]
            at += need[b]
            v = O.visible(n, L, W, S).any(0) if n else np.zeros(L, bool)
            for j in np.flatnonzero(v):
                self.tables[b, j // P] = ids[j // P]
                self.seen[ids[j // P], j % P] = True
        shape = (self.N, P, Hkv, D)
        hidden = torch.from_numpy(~self.seen)
        self.ks = self.vs = None
        if cache == "e4m3":
            self.ks, self.vs = (torch.rand(Hkv, generator=g) * 0.02 + 0.005 for _ in range(2))
            self.kc, self.vc = ((torch.randn(shape, generator=g) * 80).to(torch.float8_e4m3fn).view(torch.uint8)
                                for _ in range(2))
            for c in (self.kc, self.vc):
                c[hidden] = 0x7f
        else:
            self.kc, self.vc = (torch.randn(shape, generator=g).to(TYPES[t]) for _ in range(2))
            for c in (self.kc, self.vc):
                c[hidden] = math.nan
        self.q = torch.randn((sum(q_lens) + pad, Hq, D), generator=g).to(TYPES[t])
        self.kc, self.vc, self.q = (x.to(dev) for x in (self.kc, self.vc, self.q))
        if self.ks is not None:
            self.ks, self.vs = self.ks.to(dev), self.vs.to(dev)

    def run(self, **kw):
        return binding.window_attention(self.q, _i32(_cum(self.q_lens), self.dev), _i32(self.kv_lens, self.dev),
                                        _i32(self.tables, self.dev), self.kc, self.vc, self.scale, self.W, sinks=self.S,
                                        k_scale=self.ks, v_scale=self.vs, **kw)

    def values(self, c, scale):
        """Cached values [N, P, Hkv, D] in 64 bits."""
        if scale is None:
            return _host(c)
        return _host(c.view(torch.float8_e4m3fn).float()) * _host(scale)[:, None]

    def want(self, b):
        """The oracle's answer for sequence b, with the bounds of out and lse."""
        n, L = self.q_lens[b], self.kv_lens[b]
        q0 = int(_cum(self.q_lens)[b])
        q = _host(self.q[q0:q0 + n])
        ids = self.tables[b, np.arange(L) // self.P]
        j = np.arange(L) % self.P
        k, v = ((x := self.values(c, s))[np.where(ids < 0, 0, ids), j] for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
        k[ids < 0], v[ids < 0] = np.nan, np.nan
        out, lse, mass, dot = O.attend(q, k, v, self.scale, self.W, self.S)
        u, up = U[self.t], UP[self.cache]
        keys = min(self.W + self.S, L)
        ds = self.D * 2.0 ** -23 * dot
        if self.cache == "e4m3" and self.t == "bf16":
            ds = ds + self.D * 2.0 ** -33 * np.abs(q).max(-1) * np.nanmax(np.abs(k)) * self.scale
        small = keys * 2.0 ** -32 * np.nanmax(np.abs(v)) if up == 2.0 ** -11 else 0.0
        tol = u * np.abs(out) + (up + 2 * ds[..., None] + (keys + 64) * 2.0 ** -23 + 2.0 ** -20) * mass + small
        return out, lse, tol * (1 + u) + TINY[self.t], ds + (keys + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)

    def check(self, out, lse, seqs=None):
        cu = _cum(self.q_lens)
        o, l = _host(out), None if lse is None else _host(lse)
        for b in range(len(self.q_lens)) if seqs is None else seqs:
            if not self.q_lens[b]:
                continue
            wo, wl, to, tl = self.want(b)
            s = slice(cu[b], cu[b + 1])
            worst = (np.abs(o[s] - wo) / to).max()
            assert worst <= 1.0, (b, worst)          # (a NaN fails)
            if l is not None:
                worst = (np.abs(l[s] - wl) / tl).max()
                assert worst <= 1.0, (b, worst)


def _some(rng, n, lo, hi):
    return [int(x) for x in rng.integers(lo, hi + 1, n)]


_R = np.random.default_rng(17)
CASES = [
    # type, cache, Hq, Hkv, D, P, window, sinks, q_lens, kv_lens
    ("bf16", "bf16", 8, 2, 64, 16, 5, 0, [1], [1]),
    ("bf16", "bf16", 8, 8, 64, 16, 1, 0, [1, 1], [1, 40]),
    ("f16", "f16", 32, 4, 64, 16, 128, 4, [1] * 9, [1, 2, 5, 100, 131, 132, 133, 500, 1000]),
    ("bf16", "bf16", 32, 8, 128, 256, 300, 4, [1] * 5, [3, 299, 300, 305, 2000]),
    ("bf16", "bf16", 16, 1, 128, 64, 1000, 20, [1, 1], [4000, 900]),
    ("f16", "f16", 16, 1, 256, 24, 90, 3, [1, 2, 5], [200, 95, 1000]),
    ("bf16", "bf16", 6, 2, 256, 100, 257, 0, [1, 3, 4], [800, 3, 500]),
    ("bf16", "bf16", 5, 1, 128, 1, 33, 1, [1, 4, 0, 7], [50, 4, 9, 200]),
    ("f16", "f16", 7, 1, 64, 8, 64, 130, [2, 1, 9], [100, 131, 400]),
    ("bf16", "bf16", 3, 3, 128, 16, 40, 0, [16, 17, 1], [16, 300, 41]),
    ("bf16", "bf16", 12, 2, 64, 32, 2 ** 31 - 1, 0, [1, 5], [700, 300]),
    ("bf16", "bf16", 12, 2, 64, 32, 1, 2 ** 31 - 1, [1, 5], [700, 300]),
    ("f16", "f16", 8, 1, 128, 64, 8000, 64, [1], [20000]),
    ("bf16", "e4m3", 8, 2, 128, 16, 70, 4, [1, 3, 1], [300, 80, 1]),
    ("f16", "e4m3", 16, 2, 64, 24, 128, 0, [1, 2], [129, 700]),
    ("bf16", "e4m3", 4, 4, 256, 64, 200, 7, [5, 1], [400, 900]),
    ("bf16", "e4m3", 16, 1, 128, 256, 3000, 1, [1], [9000]),
    ("f32", "f32", 8, 2, 64, 16, 9, 2, [1, 3, 0, 20], [1, 30, 5, 200]),
    ("f32", "f32", 5, 1, 128, 24, 100, 0, [1, 2], [99, 400]),
    ("f32", "f32", 16, 1, 256, 64, 500, 4, [1, 1], [3000, 30]),
    # chunks
    ("bf16", "bf16", 8, 2, 64, 16, 50, 3, [200, 1, 64, 129], [200, 90, 300, 129]),
    ("bf16", "bf16", 32, 8, 128, 256, 128, 4, [300, 33], [300, 700]),
    ("f16", "f16", 28, 4, 128, 16, 200, 0, [150, 260, 1, 1], [150, 400, 10, 500]),
    ("f16", "f16", 10, 2, 64, 128, 33, 200, [100, 257], [400, 600]),
    ("bf16", "bf16", 4, 4, 128, 64, 300, 1, [270, 40], [270, 1000]),
    ("bf16", "bf16", 16, 1, 128, 32, 150, 0, [90, 20], [300, 20]),
    ("bf16", "bf16", 6, 1, 64, 8, 100, 10, [64, 100], [64, 333]),
    ("bf16", "bf16", 9, 3, 128, 384, 700, 4, [300], [800]),
    ("bf16", "bf16", 4, 2, 256, 64, 100, 4, [70], [300]),
    ("bf16", "bf16", 4, 2, 128, 24, 100, 4, [70, 3], [300, 50]),
    ("bf16", "e4m3", 8, 2, 128, 64, 100, 5, [200, 1, 40], [300, 400, 40]),
    ("f16", "e4m3", 7, 1, 128, 16, 300, 0, [130], [500]),
    ("f32", "f32", 8, 2, 128, 16, 40, 3, [70], [120]),
    # more sequences than a warp searches in one round, idle ones among them
    ("bf16", "bf16", 4, 2, 64, 16, 20, 1, _some(_R, 200, 0, 2), [3 + x for x in _some(_R, 200, 0, 90)]),
    ("f16", "f16", 8, 1, 64, 16, 30, 0, [1] * 1100, [1 + x for x in _some(_R, 1100, 0, 60)]),
]


def _id(c):
    return f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-w{c[6]}-s{c[7]}-n{len(c[8])}-q{max(c[8])}-k{max(c[9])}"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_attention_matches_the_oracle(dev, case):
    p = Problem(dev, *case)
    out, lse = p.run()
    assert binding.device_status() == 0
    p.check(out, lse, None if len(p.q_lens) <= 200 else range(0, len(p.q_lens), 7))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_attention_of_drawn_shapes(dev, seed):
    r = np.random.default_rng(1000 + seed)
    t = str(r.choice(["bf16", "f16", "f32"], p=[0.45, 0.4, 0.15]))
    cache = "e4m3" if t != "f32" and r.random() < 0.3 else t
    Hkv = int(r.choice([1, 2, 4]))
    Hq = Hkv * int(r.choice([1, 2, 3, 4, 5, 6, 7, 8, 16]))
    n = int(r.integers(1, 7))
    q = [int(r.choice([0, 1, 1, 2, 5, 17, 70, 200])) for _ in range(n)]
    q[0] = max(q[0], 1)
    kv = [max(x, 1) + int(r.choice([0, 0, 3, 100, 500])) for x in q]
    p = Problem(dev, t, cache, Hq, Hkv, int(r.choice([64, 128, 256], p=[0.4, 0.4, 0.2])),
                int(r.choice([1, 8, 16, 24, 64, 128, 256])), int(r.choice([1, 7, 64, 129, 400])),
                int(r.choice([0, 1, 4, 40, 128, 200])), q, kv, seed=seed)
    out, lse = p.run()
    assert binding.device_status() == 0
    p.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[2], CASES[13], CASES[17], CASES[20], CASES[30]], ids=_id)
def test_rows_behind_the_last_sequence_and_an_unwanted_lse(dev, case):
    p = Problem(dev, *case, pad=37)
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
    p.run(out=out, lse=lse)
    end = sum(p.q_lens)
    p.check(out, lse)
    assert (out[end:] == 7).all() and (lse[end:] == 7).all()
    again, none = p.run(want_lse=False)
    assert none is None and torch.equal(again[:end], out[:end])
    assert binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[3], CASES[12], CASES[16], CASES[19], CASES[21], CASES[30]], ids=_id)
def test_the_same_call_gives_the_same_bits(dev, case):
    p = Problem(dev, *case)
    first = p.run()
    for _ in range(3):
        again = p.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,Hq,Hkv,D,q,kv", [("bf16", "bf16", 8, 2, 64, 1, 300), ("f16", "f16", 8, 1, 128, 150, 300),
                                                   ("f32", "f32", 4, 2, 64, 3, 50), ("bf16", "e4m3", 8, 2, 128, 1, 40),
                                                   ("bf16", "e4m3", 8, 2, 128, 90, 200)])
def test_a_nan_reaches_the_rows_that_see_it(dev, t, cache, Hq, Hkv, D, q, kv):
    p = Problem(dev, t, cache, Hq, Hkv, D, 16, 40, 2, [q, q], [kv, kv])
    at = kv - 1                                            # the last key of sequence 0, KV head 0
    c = p.kc[p.tables[0, at // 16], at % 16, 0]
    c[5] = 0x7f if cache == "e4m3" else math.nan
    out, lse = p.run()
    g = Hq // Hkv
    assert torch.isnan(out[q - 1, :g]).all() and torch.isnan(lse[q - 1, :g]).all()
    assert torch.isfinite(out[q - 1, g:]).all() and torch.isfinite(out[q:]).all()
    assert binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,Hq,Hkv,D,q,kv,W", [("bf16", 8, 2, 64, 1, 300, 40), ("f16", 8, 1, 128, 150, 300, 40),
                                               ("f32", 4, 2, 64, 3, 50, 9), ("bf16", 8, 1, 128, 1, 5000, 4000),
                                               ("bf16", 8, 2, 64, 70, 70, 400)])
def test_rows_whose_scores_are_all_minus_infinity(dev, t, Hq, Hkv, D, q, kv, W):
    p = Problem(dev, t, t, Hq, Hkv, D, 16, W, 2, [q, 1], [kv, 9])
    p.q[:q].abs_()
    for j in np.flatnonzero(O.visible(q, kv, W, 2).any(0)):
        p.kc[p.tables[0, j // 16], j % 16] = -math.inf
    out, lse = p.run()
    assert torch.isnan(out[:q]).all() and (lse[:q] == -math.inf).all()
    p.check(out, lse, [1])


@pytest.mark.gpu
@pytest.mark.parametrize("t,Hq,Hkv,D,q,kv", [("bf16", 8, 2, 64, 1, 300), ("f16", 8, 1, 128, 150, 300), ("f32", 4, 2, 64, 3, 50)])
def test_some_scores_of_minus_infinity(dev, t, Hq, Hkv, D, q, kv):
    # the first keys of each row's window are -inf, with the type's lowest value beside them: no
    # weight, and the maximum starts late
    p = Problem(dev, t, t, Hq, Hkv, D, 16, 40, 0, [q], [kv])
    p.q.abs_()
    lo = kv - q - 39
    low = -torch.finfo(TYPES[t]).max
    for j in range(max(lo, 0), kv - q):
        p.kc[p.tables[0, j // 16], j % 16] = -math.inf if j % 2 else (low if t != "bf16" else -3e38)
    out, lse = p.run()
    keep = Problem(dev, t, t, Hq, Hkv, D, 16, 40, 0, [q], [kv])
    keep.q, keep.vc = p.q, p.vc
    # rows see only the chunk's own keys then: the same as a window that begins there
    wo, wl = [], []
    for i in range(q):
        ids = [(int(keep.tables[0, j // 16]), j % 16) for j in range(kv - q, kv - q + i + 1) if j > kv - q + i - 40]
        k = np.stack([_host(p.kc[a, b]) for a, b in ids])
        v = np.stack([_host(p.vc[a, b]) for a, b in ids])
        o, l, mass, dot = O.attend(_host(p.q[i:i + 1]), k, v, p.scale, 10 ** 6, 0)
        tol = U[t] * np.abs(o) + (UP[t] + 2 * D * 2.0 ** -23 * dot[..., None] + 2.0 ** -16) * mass + 2.0 ** -20
        assert (np.abs(_host(out[i:i + 1]) - o) <= tol).all(), i
        assert np.abs(_host(lse[i:i + 1]) - l).max() <= D * 2.0 ** -23 * dot.max() + 2.0 ** -16


@pytest.mark.gpu
@pytest.mark.parametrize("q", [1, 4, 100])
@pytest.mark.parametrize("t,D,P", [("bf16", 128, 64), ("f32", 64, 16), ("f16", 256, 24)])
def test_bad_data_skips_the_sequence(dev, t, D, P, q):
    kv, n = [200, 150, 300, 220], [q] * 4
    p = Problem(dev, t, t, 8, 2, D, P, 60, 3, n, kv)
    good, glse = p.run()
    p.check(good, glse)
    cu = _cum(n)

    def run(kv=kv, tables=p.tables, cu=cu):
        out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
        binding.window_attention(p.q, _i32(cu, dev), _i32(kv, dev), _i32(tables, dev), p.kc, p.vc, p.scale, p.W, sinks=p.S,
                                 out=out, lse=lse)
        return out, lse, binding.device_status()

    for bad in (q - 1, p.tables.shape[1] * P + 1, -5):      # fewer keys than rows; more than the table holds
        out, lse, st = run(kv=[200, bad, 300, 220])
        assert st == binding.DEV_BAD_LENGTHS and (out[cu[1]:cu[2]] == 7).all() and (lse[cu[1]:cu[2]] == 7).all()
        assert torch.equal(out[:cu[1]], good[:cu[1]]) and torch.equal(out[cu[2]:], good[cu[2]:])
    for page, entry in ((kv[2] - 1) // P, p.N), ((kv[2] - 1) // P, -1), (0, 1 << 30):
        tables = p.tables.copy()
        tables[2, page] = entry
        out, lse, st = run(tables=tables)
        assert st == binding.DEV_BAD_PAGE
        last = cu[3] - 1                                    # the last row needs the last page and the sinks' page
        assert (out[last] == 7).all() and (lse[last] == 7).all()
        assert torch.equal(out[:cu[2]], good[:cu[2]]) and torch.equal(out[cu[3]:], good[cu[3]:])
    for bad in ([1, q, 2 * q, 3 * q, 4 * q], [0, 2 * q, q, 3 * q, 4 * q], [0, q, 2 * q, 3 * q, 4 * q + 1], [0, -9, q, q, q]):
        assert run(cu=bad)[2] & binding.DEV_BAD_LENGTHS


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,q", [("bf16", "bf16", 1), ("bf16", "bf16", 100), ("bf16", "e4m3", 1), ("f32", "f32", 1)])
def test_pages_beyond_four_gigabytes(dev, t, cache, q):
    P, Hkv, D = 256, 8, 128
    elt = {"f32": 4, "bf16": 2, "e4m3": 1}[cache]
    far = (5 << 30) // (P * Hkv * D * elt)
    p = Problem(dev, t, cache, 16, Hkv, D, P, 300, 2, [q, q], [700, 400])
    kc = torch.zeros((far + p.N, P, Hkv, D), dtype=p.kc.dtype, device=dev)
    vc = torch.zeros_like(kc)
    kc[far:], vc[far:] = p.kc, p.vc
    out, lse = binding.window_attention(p.q, _i32(_cum(p.q_lens), dev), _i32(p.kv_lens, dev),
                                        _i32(np.where(p.tables < 0, -1, p.tables + far), dev), kc, vc, p.scale, p.W,
                                        sinks=p.S, k_scale=p.ks, v_scale=p.vs)
    p.check(out, lse)
    assert binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,q", [("f16", "f16", 1), ("f16", "f16", 130), ("f16", "e4m3", 1), ("f16", "e4m3", 100)])
def test_small_f16_weights_are_not_lost(dev, t, cache, q):
    # one key of weight 1 and thousands of weight 2^-17 each, whose values alone are not zero
    n, W = 6000, 5000
    p = Problem(dev, t, cache, 8, 1, 128, 64, W, 0, [q], [n], spread=math.sqrt(128))
    p.q.zero_()
    p.q[:, :, 0] = 1.0
    if cache == "e4m3":
        p.ks.fill_(1.0)
        p.vs.fill_(1.0)
        to = lambda x: torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).item()
    else:
        to = lambda x: x
    for c, first in ((p.kc, 0.0), (p.vc, 1.0)):
        c[torch.from_numpy(p.seen)] = to(0.0)
        c[..., 0][torch.from_numpy(p.seen)] = to(first)
    j = n - q - 1                                           # seen by every row
    p.kc[p.tables[0, j // 64], j % 64, 0, 0] = to(12.0)
    p.vc[p.tables[0, j // 64], j % 64, 0, 0] = to(0.0)
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.gpu
def test_more_sequences_than_threads_and_a_long_idle_tail(dev):
    q = [0] * 3000 + [1, 0, 2, 40, 0, 1] + [0] * 2000
    kv = [5] * 3000 + [30, 7, 50, 40, 0, 1] + [0] * 2000
    p = Problem(dev, "bf16", "bf16", 8, 2, 64, 16, 20, 1, q, kv)
    out, lse = p.run()
    p.check(out, lse)
    assert binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_a_wide_window_equals_plain_paged_attention(dev, t, cache):
    p = Problem(dev, t, cache, 16, 4, 128, 64, 10 ** 6, 0, [1, 70, 1, 3], [500, 170, 1, 90])
    out, lse = p.run()
    p.check(out, lse)
    args = (p.q, _i32(_cum(p.q_lens), dev), _i32(p.kv_lens, dev), _i32(p.tables, dev), p.kc, p.vc)
    if cache == "e4m3":
        ro, rl = binding.paged_attention_fp8(*args, p.ks, p.vs, p.scale, 500)
    else:
        ro, rl = binding.paged_attention(*args, p.scale, 500)
    # both are within bounds of the same values
    for b in range(4):
        s = slice(_cum(p.q_lens)[b], _cum(p.q_lens)[b + 1])
        _, _, to, tl = p.want(b)
        u = {"bf16": 2.0 ** -8, "f32": 2.0 ** -20}[t]
        assert (np.abs(_host(out[s]) - _host(ro[s])) <= 2 * to + 4 * u * np.abs(_host(p.vc[p.seen].float()).max()
                if cache != "e4m3" else 448 * _host(p.vs).max())).all()
        assert (np.abs(_host(lse[s]) - _host(rl[s])) <= 2 * tl + 1e-3).all()


# --- norm, rotation, append

APPEND = [
    # type, cache, T, Hq, Hkv, D, P, rot, interleaved, norms
    ("bf16", "bf16", 1, 8, 2, 64, 16, 64, False, "qk"),
    ("bf16", "bf16", 70, 32, 8, 128, 256, 128, False, "qk"),
    ("f16", "f16", 33, 5, 1, 128, 24, 64, True, "qk"),
    ("bf16", "bf16", 9, 28, 4, 128, 1, 16, False, ""),
    ("f16", "f16", 200, 3, 3, 64, 16, 48, False, "k"),
    ("bf16", "bf16", 20, 16, 1, 256, 64, 128, True, "q"),
    ("f16", "f16", 20, 7, 1, 256, 64, 256, False, "qk"),
    ("f32", "f32", 13, 4, 4, 64, 16, 32, True, "qk"),
    ("f32", "f32", 40, 6, 2, 128, 16, 128, False, "qk"),
    ("f32", "f32", 11, 6, 2, 256, 8, 256, False, "qk"),
    ("f32", "f32", 11, 6, 2, 256, 8, 160, False, "qk"),
    ("f32", "f32", 11, 6, 2, 256, 8, 80, True, ""),
    ("bf16", "e4m3", 50, 16, 2, 128, 16, 128, False, "qk"),
    ("f16", "e4m3", 50, 8, 8, 64, 32, 32, True, "k"),
    ("f32", "e4m3", 17, 4, 2, 256, 16, 256, False, "qk"),
    ("f32", "e4m3", 17, 4, 2, 64, 16, 64, True, "qk"),
]


def _append_inputs(dev, t, cache, T, Hq, Hkv, D, P, rot, seed=3, std=2.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    pages = -(-T // P) + 2
    x = dict(q=(n(T, Hq, D) * std).to(TYPES[t]), k=(n(T, Hkv, D) * std).to(TYPES[t]), v=(n(T, Hkv, D) * std).to(TYPES[t]),
             qw=(1 + 0.2 * n(D)).to(TYPES[t]), kw=(1 + 0.2 * n(D)).to(TYPES[t]),
             pos=torch.randint(0, 500, (T,), generator=g, dtype=torch.int32),
             slots=torch.randperm(pages * P, generator=g)[:T],
             cs=torch.from_numpy(binding.rope_table_scaled(10000.0, rot, 500, "ramp", factor=4.0, original_max_pos=256)))
    if T > 5:
        x["slots"][3] = -1
    if cache == "e4m3":
        x["ks"], x["vs"] = (torch.rand(Hkv, generator=g) * 0.02 + 0.004 for _ in range(2))
        x["kc"], x["vc"] = (torch.randint(0, 127, (pages, P, Hkv, D), generator=g, dtype=torch.uint8) for _ in range(2))
    else:
        x["ks"] = x["vs"] = None
        x["kc"], x["vc"] = (n(pages, P, Hkv, D).to(TYPES[t]) for _ in range(2))
    return {k: None if v is None else v.to(dev) for k, v in x.items()}


def _check_append(x, x0, got_q, t, cache, interleaved, norms, eps):
    D = x0["q"].shape[-1]
    cs = _host(x0["cs"])[_host(x0["pos"]).astype(int)]
    grow = (D / 2 + 8) * 2.0 ** -24

    def rotated(name, w):
        return O.rotate(O.norm(_host(x0[name]), None if w is None else _host(w), eps), cs, interleaved)

    y, size = rotated("q", x0["qw"] if "q" in norms else None)
    assert (np.abs(_host(got_q) - y) / (U[t] * np.abs(y) + (1 + U[t]) * grow * size + TINY[t] + 2.0 ** -140)).max() <= 1
    y, size = rotated("k", x0["kw"] if "k" in norms else None)
    slots = x0["slots"].cpu().numpy()
    P = x0["kc"].shape[1]
    kc, vc = x["kc"].cpu(), x["vc"].cpu()
    k0, v0 = x0["kc"].cpu().clone(), x0["vc"].cpu().clone()
    for i, s in enumerate(slots):
        if s < 0:
            continue
        a, b = int(s) // P, int(s) % P
        if cache == "e4m3":
            sk = x0["ks"].cpu().numpy()
            got = kc[a, b].view(torch.float8_e4m3fn).double().numpy() * sk[:, None].astype(np.float64)
            want = np.clip(y[i] / sk[:, None], -448, 448) * sk[:, None].astype(np.float64)
            # half a step of the code (2^-4 relative, 2^-10 below the normal range) and the quotient's rounding
            tol = (2.0 ** -4 + 2.0 ** -23) * np.abs(want) + 2.0 ** -10 * sk[:, None] + 1.1 * grow * size[i]
            assert (np.abs(got - want) <= tol).all(), i
            wv = F.quantize(x0["v"][i].float().cpu().numpy(), x0["vs"].cpu().numpy())
            assert np.array_equal(vc[a, b].numpy(), wv), i
        else:
            tol = U[t] * np.abs(y[i]) + (1 + U[t]) * grow * size[i] + TINY[t] + 2.0 ** -140
            assert (np.abs(_host(kc[a, b]) - y[i]) / tol).max() <= 1, i
            assert torch.equal(vc[a, b], x0["v"][i].cpu()), i
        k0[a, b], v0[a, b] = kc[a, b], vc[a, b]
    assert torch.equal(k0, kc) and torch.equal(v0, vc)      # nothing else was written


@pytest.mark.gpu
@pytest.mark.parametrize("view", ["rows", "views", "in place"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append_matches_the_oracle(dev, case, view):
    t, cache, T, Hq, Hkv, D, P, rot, inter, norms = case
    x = _append_inputs(dev, t, cache, T, Hq, Hkv, D, P, rot)
    x0 = {k: None if v is None else v.clone() for k, v in x.items()}
    q, k, v, qo = x["q"], x["k"], x["v"], None
    if view != "rows":
        big = torch.zeros((T, Hq + 2 * Hkv + 1, D), dtype=q.dtype, device=dev)
        big[:, :Hq], big[:, Hq:Hq + Hkv], big[:, Hq + Hkv:-1] = q, k, v
        q, k, v = big[:, :Hq], big[:, Hq:Hq + Hkv], big[:, Hq + Hkv:-1]
        qo = q if view == "in place" else torch.zeros((Hq, T + 3, D), dtype=q.dtype, device=dev)[:, :T].transpose(0, 1)
    got = binding.norm_rope_kv_append(q, k, v, x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                      q_weight=x["qw"] if "q" in norms else None, k_weight=x["kw"] if "k" in norms else None,
                                      eps=1e-5, interleaved=inter, k_scale=x["ks"], v_scale=x["vs"], q_out=qo)
    assert binding.device_status() == 0 and (qo is None or got is qo)
    _check_append(x, x0, got, t, cache, inter, norms, 1e-5)


@pytest.mark.gpu
def test_append_agrees_with_the_plain_rotation(dev):
    # no norm, whole heads in halves: what rope_kv_append computes, up to its order of operations
    x = _append_inputs(dev, "f32", "f32", 40, 8, 2, 64, 16, 64)
    kc, vc = x["kc"].clone(), x["vc"].clone()
    x["slots"][3] = int((set(range(kc.shape[0] * 16)) - set(x["slots"].tolist())).pop())
    got = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"])
    want = binding.rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], kc, vc)
    top = 1.2 * float(x["q"].abs().max().maximum(x["k"].abs().max()))
    assert (got - want).abs().max() <= 4 * 2.0 ** -24 * 2 * top
    assert (x["kc"] - kc).abs().max() <= 4 * 2.0 ** -24 * 2 * top and torch.equal(x["vc"], vc)


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache", [("bf16", "bf16"), ("f32", "f32"), ("f16", "e4m3")])
def test_append_bad_tokens(dev, t, cache):
    x = _append_inputs(dev, t, cache, 12, 8, 2, 64, 16, 32)
    x["pos"][2], x["pos"][5], x["slots"][7], x["slots"][3] = -1, 500, x["kc"].shape[0] * 16, 1 << 40
    q_out = torch.full_like(x["q"], 7.0)
    k0, v0 = x["kc"].clone(), x["vc"].clone()
    args = (x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"])
    binding.norm_rope_kv_append(*args, x["kc"], x["vc"], q_weight=x["qw"], k_weight=x["kw"], k_scale=x["ks"],
                                v_scale=x["vs"], q_out=q_out)
    assert binding.device_status() == binding.DEV_BAD_POSITION | binding.DEV_BAD_SLOT
    assert (q_out[[2, 5]] == 7).all() and (q_out[[7, 3]] != 7).any()
    for i in (2, 5):
        s = int(x["slots"][i])
        assert torch.equal(x["kc"].flatten(0, 1)[s], k0.flatten(0, 1)[s])
        assert torch.equal(x["vc"].flatten(0, 1)[s], v0.flatten(0, 1)[s])
    written = [int(s) for i, s in enumerate(x["slots"]) if i not in (2, 3, 5, 7)]
    rest = [s for s in range(k0.shape[0] * 16) if s not in written]
    assert torch.equal(x["kc"].flatten(0, 1)[rest], k0.flatten(0, 1)[rest])


@pytest.mark.gpu
def test_append_of_zeros_and_large_values(dev):
    x = _append_inputs(dev, "f16", "f16", 4, 2, 2, 64, 16, 64)
    x["q"].zero_()
    x["k"].fill_(60000.0)                                   # squares beyond f16, not beyond fp32
    out = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                      q_weight=x["qw"], k_weight=x["kw"], eps=0.0)
    assert torch.isnan(out).all()                           # 0 / 0
    out = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                      q_weight=x["qw"], k_weight=x["kw"], eps=1e-6)
    assert (out == 0).all()
    k = x["kc"].flatten(0, 1)[x["slots"]]
    assert torch.isfinite(k).all() and k.abs().max() < 4


# --- pages

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shape,n,layers", [
    (torch.bfloat16, (9, 16, 2, 64), 1, 2), (torch.float16, (40, 1, 1, 64), 15, 3), (torch.uint8, (30, 24, 1, 16), 11, 5),
    (torch.float32, (12, 256, 8, 128), 5, 1), (torch.bfloat16, (20, 64, 576), 9, 4), (torch.bfloat16, (7, 5, 8), 3, 300)])
@pytest.mark.parametrize("part", [False, True])
def test_copies_are_bit_exact(dev, dtype, shape, n, layers, part):
    g = torch.Generator().manual_seed(n)
    caches = [torch.randint(0, 256, (*shape[:-1], shape[-1] * torch.empty(0, dtype=dtype).element_size()), generator=g,
                            dtype=torch.uint8).view(dtype).to(dev) for _ in range(layers)]
    perm = torch.randperm(shape[0], generator=g).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    tokens = torch.randint(0, shape[1] + 1, (n,), generator=g, dtype=torch.int32) if part else None
    if n > 4:
        src[1], dst[2] = -1, -7
        src[3] = dst[3]
    raw = lambda c: c.reshape(*shape[:2], -1).view(torch.uint8).cpu()
    want = []
    for c in caches:
        w = raw(c).clone()
        for i in range(n):
            if src[i] >= 0 and dst[i] >= 0:
                m = shape[1] if tokens is None else int(tokens[i])
                w[dst[i], :m] = raw(c)[src[i], :m]
        want.append(w)
    assert binding.copy_pages(caches, src.to(dev), dst.to(dev), None if tokens is None else tokens.to(dev)) is None
    assert binding.device_status() == 0
    for c, w in zip(caches, want):
        assert torch.equal(raw(c), w)


@pytest.mark.gpu
def test_copies_with_bad_ids_and_counts(dev):
    c = torch.arange(6 * 4 * 8, dtype=torch.float32, device=dev).view(6, 4, 8)
    c0 = c.clone()
    binding.copy_pages([c], _i32([0, 6], dev), _i32([1, 2], dev))
    assert binding.device_status() == binding.DEV_BAD_PAGE
    assert torch.equal(c[1], c0[0]) and torch.equal(c[2:], c0[2:])
    binding.copy_pages([c], _i32([2, 3], dev), _i32([1 << 30, 5], dev))
    assert binding.device_status() == binding.DEV_BAD_PAGE and torch.equal(c[5], c0[3])
    c.copy_(c0)
    binding.copy_pages([c], _i32([0, 1, 2], dev), _i32([3, 4, 5], dev), _i32([5, -1, 4], dev))
    assert binding.device_status() == binding.DEV_BAD_LENGTHS
    assert torch.equal(c[3:5], c0[3:5]) and torch.equal(c[5], c0[2])


@pytest.mark.gpu
def test_copies_beyond_four_gigabytes(dev):
    c = torch.zeros((5 << 20, 1, 1024), dtype=torch.uint8, device=dev)
    c[5] = 3
    c[-1] = 9
    binding.copy_pages([c], _i32([5, c.shape[0] - 1], dev), _i32([c.shape[0] - 2, 7], dev))
    assert (c[-2] == 3).all() and (c[7] == 9).all() and int(c[-3].sum()) == 0 and binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 1000, 3_000_001])
def test_tables_are_rewritten(dev, n):
    g = torch.Generator().manual_seed(n)
    t = torch.randint(-2, 50, (n,), generator=g, dtype=torch.int32)
    m = torch.randperm(50, generator=g).to(torch.int32)
    m[7] = -1
    got = binding.remap_pages(t.to(dev), m.to(dev))
    assert torch.equal(got.cpu(), torch.where(t >= 0, m[t.long().clamp(min=0)], t)) and binding.device_status() == 0


@pytest.mark.gpu
def test_tables_with_bad_entries(dev):
    t = _i32([[0, 3, -1], [9, 2, 1]], dev)
    binding.remap_pages(t, _i32([2, 1, 0, 4], dev))
    assert binding.device_status() == binding.DEV_BAD_PAGE
    assert t.tolist() == [[2, 3, -1], [9, 0, 1]]             # an id and a target outside the pool stay


# --- graphs, streams

@pytest.mark.gpu
def test_graphs_replay_with_new_lengths_and_side_by_side(dev):
    a = Problem(dev, "bf16", "bf16", 8, 2, 128, 64, 50, 3, [1] * 6, [40, 300, 1, 90, 64, 65])
    b = Problem(dev, "bf16", "bf16", 8, 2, 128, 64, 50, 3, [100, 1, 60], [160, 90, 60], seed=5)
    st = []
    for p in (a, b):
        s = dict(cu=_i32(_cum(p.q_lens), dev), kv=_i32(p.kv_lens, dev), pt=_i32(p.tables, dev), out=torch.empty_like(p.q),
                 lse=torch.empty(p.q.shape[:2], device=dev))
        call = lambda p=p, s=s: binding.window_attention(p.q, s["cu"], s["kv"], s["pt"], p.kc, p.vc, p.scale, p.W,
                                                         sinks=p.S, out=s["out"], lse=s["lse"])
        call()
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            call()
        st.append(s)
    streams = [torch.cuda.Stream() for _ in st]
    for _ in range(5):
        for p, s in zip((a, b), st):
            s["out"].fill_(9)
        torch.cuda.synchronize()
        for s, on in zip(st, streams):
            with torch.cuda.stream(on):
                s["graph"].replay()
        torch.cuda.synchronize()
        for p, s in zip((a, b), st):
            p.check(s["out"], s["lse"])
    # new lengths, pages and row counts in place: fewer rows than were captured
    c = Problem(dev, "bf16", "bf16", 8, 2, 128, 64, 50, 3, [0, 30, 61], [9, 30, 150], seed=6, pad=b.q.shape[0] - 91)
    s = st[1]
    pt = np.full(s["pt"].shape, -1, np.int32)
    pt[:, :c.tables.shape[1]] = c.tables[:, :pt.shape[1]]
    n = min(b.N, c.N)
    assert c.N <= b.N and (c.tables < n).all()
    b.kc[:c.N], b.vc[:c.N] = c.kc, c.vc
    b.q.copy_(c.q)
    s["cu"].copy_(_i32(_cum(c.q_lens), dev))
    s["kv"].copy_(_i32(c.kv_lens, dev))
    s["pt"].copy_(_i32(pt, dev))
    s["out"].fill_(9)
    s["graph"].replay()
    torch.cuda.synchronize()
    c.check(s["out"], s["lse"])
    assert (s["out"][91:] == 9).all() and binding.device_status() == 0


@pytest.mark.gpu
def test_another_stream_in_order(dev):
    on = torch.cuda.Stream()
    x = _append_inputs(dev, "bf16", "bf16", 200, 32, 8, 128, 64, 128)
    p = Problem(dev, "bf16", "bf16", 8, 2, 64, 16, 30, 0, [1] * 50, [60] * 50)
    torch.cuda.synchronize()
    want, _ = p.run()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(on):
            got, _ = p.run(stream=on)
            moved = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                                stream=on)
            again, _ = p.run(stream=on)
        on.synchronize()
        assert torch.equal(got, want) and torch.equal(again, want) and moved.shape == x["q"].shape


# --- a serving loop

@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,Hq,Hkv,D,P,W,S", [("bf16", "bf16", 8, 2, 64, 16, 40, 3), ("f16", "e4m3", 8, 2, 128, 8, 25, 0),
                                                    ("f32", "f32", 4, 4, 64, 4, 20, 6)])
def test_a_serving_loop(dev, t, cache, Hq, Hkv, D, P, W, S):
    """Prompts, decode ticks, forks, trimming and compaction, through the public calls; each
    tick's attention is checked against the oracle on every key of each sequence's history."""
    rng = np.random.default_rng(2)
    g = torch.Generator().manual_seed(2)
    N, layers = 96, 2
    pool = binding.PagePool(N, P)
    shape = (N, P, Hkv, D)
    dt = torch.uint8 if cache == "e4m3" else TYPES[t]
    caches = [torch.zeros(shape, dtype=dt, device=dev) for _ in range(2 * layers)]
    sc = (lambda: (torch.rand(Hkv, generator=g) * 0.01 + 0.01).to(dev)) if cache == "e4m3" else (lambda: None)
    scales = [sc() for _ in range(2 * layers)]
    table = torch.from_numpy(binding.rope_table_scaled(10000.0, D // 2, 600, "linear", factor=2.0)).to(dev)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(TYPES[t]).to(dev) for _ in range(2))
    seqs = {}                     # name: pages, history of each layer's (k, v) as cached, in 64 bits
    read = lambda c, s: (_host(c) if s is None else
                         _host(c.view(torch.float8_e4m3fn).float()) * _host(s)[:, None])

    def tick(new):
        """new: {name: rows}; packs, appends and attends in every layer."""
        names = list(new)
        for n in names:
            s = seqs[n]
            want = -(-(s["len"] + new[n]) // P)
            s["pages"] += pool.alloc(want - len(s["pages"]))
            s["len"] += new[n]
        pk = binding.pack_tick([new[n] for n in names], [seqs[n]["len"] for n in names],
                               [seqs[n]["pages"] for n in names], P, N, window=W, sinks=S)
        pos = binding.tick_positions(pk["cu_seqlens_q"], pk["kv_lens"])
        T = len(pos)
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        for l in range(layers):
            qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * 2).to(TYPES[t]).to(dev)
            kc, vc, ks, vs = caches[2 * l], caches[2 * l + 1], scales[2 * l], scales[2 * l + 1]
            q = binding.norm_rope_kv_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], to(pos), table,
                                            to(pk["slot_mapping"]), kc, vc, q_weight=qw, k_weight=kw, interleaved=l == 1,
                                            k_scale=ks, v_scale=vs)
            out, lse = binding.window_attention(q, to(pk["cu_seqlens_q"]), to(pk["kv_lens"]), to(pk["page_tables"]), kc, vc,
                                                1 / math.sqrt(D), W, sinks=S, k_scale=ks, v_scale=vs)
            k, v, slots = read(kc, ks), read(vc, vs), pk["slot_mapping"]
            for i, b in enumerate(pk["order"]):
                s, n = seqs[names[b]], new[names[b]]
                a, e = pk["cu_seqlens_q"][i], pk["cu_seqlens_q"][i + 1]
                s["hist"][l] += [(k[x // P, x % P], v[x // P, x % P]) for x in slots[a:e]]
                kk, vv = (np.stack([h[j] for h in s["hist"][l]]) for j in (0, 1))
                wo, wl, mass, dot = O.attend(_host(q[a:e]), kk, vv, 1 / math.sqrt(D), W, S)
                ds = D * 2.0 ** -23 * dot + 2.0 ** -15
                tol = U[t] * np.abs(wo) + (UP[cache] + 2 * ds[..., None]) * mass + 2.0 ** -20
                assert (np.abs(_host(out[a:e]) - wo) <= tol).all()
                assert (np.abs(_host(lse[a:e]) - wl) <= ds + 2.0 ** -20 * (1 + np.abs(wl))).all()

    fresh = lambda: dict(pages=[], len=0, hist=[[] for _ in range(layers)])
    seqs.update(a=fresh(), b=fresh(), c=fresh())
    tick({"a": 70, "b": 3, "c": 33})
    names = iter("defghijk")
    for step in range(12):
        tick({n: 1 if rng.random() < 0.8 else int(rng.integers(2, 12)) for n in seqs})
        for s in seqs.values():
            s["pages"] = pool.trim(s["pages"], s["len"], W, S)
        if step % 3 == 1:
            parent = seqs[str(rng.choice(list(seqs)))]
            pages, copy = pool.fork(parent["pages"], parent["len"])
            if copy:
                src, dst, tokens = ([x] for x in copy)
                binding.copy_pages(caches, _i32(src, dev), _i32(dst, dev), _i32(tokens, dev))
            seqs[next(names)] = dict(pages=pages, len=parent["len"], hist=[list(h) for h in parent["hist"]])
        if step % 4 == 2:
            gone = str(rng.choice(list(seqs)))
            pool.release([x for x in seqs.pop(gone)["pages"] if x >= 0])
            src, dst, page_map = pool.compact()
            if len(src):
                binding.copy_pages(caches, _i32(src, dev), _i32(dst, dev))
            w = max(len(s["pages"]) for s in seqs.values())
            tables = np.full((len(seqs), w), -1, np.int32)
            for i, s in enumerate(seqs.values()):
                tables[i, :len(s["pages"])] = s["pages"]
            moved = binding.remap_pages(_i32(tables, dev), _i32(page_map, dev)).cpu().numpy()
            for i, s in enumerate(seqs.values()):
                s["pages"] = [int(x) for x in moved[i, :len(s["pages"])]]
            held = {x for s in seqs.values() for x in s["pages"] if x >= 0}
            assert held == set(range(len(held)))
    assert binding.device_status() == 0
    for s in seqs.values():
        pool.release([x for x in s["pages"] if x >= 0])
    assert pool.free_count() == N
