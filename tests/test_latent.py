"""Latent attention: the oracle against closed forms and against torch, the
calls' refusals on the host, and (GPU) every operator against the oracle in 64
bits, alone and as the run a serving tick makes of them.

Tolerances. u is half a step of the cache type (bf16 2^-8, f16 2^-11). A result
is rounded once (u |out|) and every softmax weight once before its product with
the values (u sum_j w_j |v_j|; f16 weights below 2^-14 are subnormal, off by up to
2^-25 of a weight scale that is at least 1, so 2^-25 max|v| a key). A score is an fp32 sum
of D products: off by at most D 2^-23 scale sum_d |q_d k_d| =: ds (2^-23: the
tensor core may truncate), which moves every weight by a factor exp(+-ds) before
and, through the sum, as much after: 2 ds sum_j w_j |v_j|. The output sums over L
keys in fp32 add at most (L + 64) 2^-23 of sum_j w_j |v_j|, and the exponential's and
the final scaling's errors, a few 2^-22 relative, are below 2^-20. lse moves by ds, by
the sum's own relative error (L + 64) 2^-23, and by 2^-20 plus two roundings of its size.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import latent as O
from oracle.rope import apply_rope
from paged_kv_attention_mapping_gb300 import binding

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SCALE = 1.0 / math.sqrt(192)


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
    return d


# ---------------------------------------------------------------------------
# oracle pins (CPU)

def test_oracle_attention_matches_torch():
    g = np.random.default_rng(0)
    n, L, H = 5, 11, 3
    q, rows = g.standard_normal((n, H, 320)), g.standard_normal((L, 320))
    mask = torch.ones(n, L, dtype=torch.bool).tril(L - n)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q).transpose(0, 1), t(rows).expand(H, L, 320), t(rows)[:, :256].expand(H, L, 256), mask, scale=0.1)
    out, lse, _ = O.attend_absorbed(q, rows, 0.1)
    assert np.abs(out - want.transpose(0, 1).numpy()).max() < 1e-12
    x = 0.1 * np.einsum("nhd,ld->nhl", q, rows)
    x[~np.broadcast_to(mask.numpy()[:, None], x.shape)] = -np.inf
    assert np.abs(lse - torch.logsumexp(t(x), -1).numpy()).max() < 1e-12


def test_oracle_expanded_equals_absorbed():
    """The two forms agree: with k_nope = c Wk and v = c Wv, attending the expanded
    keys equals attending the rows with q Wk^T and expanding the result."""
    g = np.random.default_rng(1)
    n, L, H, ld = 4, 9, 2, 32
    c, r = g.standard_normal((L, ld)), g.standard_normal((L, 64))
    wk, wv = g.standard_normal((H, ld, 128)) / 6, g.standard_normal((H, ld, 128)) / 6
    q = g.standard_normal((n, H, 192))
    kn, v = np.einsum("lc,hcd->lhd", c, wk), np.einsum("lc,hcd->lhd", c, wv)
    e, el, _ = O.attend_expanded(q, kn, v, r, SCALE)
    qa = np.concatenate([np.einsum("nhd,hcd->nhc", q[..., :128], wk), q[..., 128:]], -1)
    a, al, _ = O.attend_absorbed(qa, np.concatenate([c, r], -1), SCALE)
    assert np.abs(np.einsum("nhc,hcd->nhd", a, wv) - e).max() < 1e-12
    assert np.abs(al - el).max() < 1e-12


def test_oracle_one_key_and_rows_ahead():
    rows = np.random.default_rng(2).standard_normal((3, 96))
    q = np.random.default_rng(3).standard_normal((3, 1, 96))
    out, lse, _ = O.attend_absorbed(q, rows, 0.2)
    assert np.array_equal(out[0, 0], rows[0, :32])               # the first row sees one key
    assert abs(lse[0, 0] - 0.2 * q[0, 0] @ rows[0]) < 1e-14


def test_oracle_append_and_gather():
    cache = np.zeros((3, 2, 66))
    c, k = np.full((2, 2), 7.0), np.zeros((2, 64))
    k[:, 0] = 1.0
    got = O.append(cache, c, k, [0, 3], [5, -1], 100.0)
    assert list(got[2, 1, :3]) == [7.0, 7.0, 1.0] and np.count_nonzero(got) == 3
    assert np.array_equal(O.gather_sequence(got, [1, 2], 4)[3], got[2, 1])


# ---------------------------------------------------------------------------
# refusals (CPU: no pointer reaches a kernel)

FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)


def _desc(**kw):
    d = dict(num_pages=4, page_size=16, latent_dim=512, rope_dim=64, dtype=binding.PKV_BF16)
    d.update(kw)
    return binding.LatentDesc(**d)


BAD_DESCS = [(dict(dtype=binding.PKV_F32), -2), (dict(dtype=binding.PKV_FP8_E4M3), -2), (dict(dtype=9), -2),
             (dict(latent_dim=384), -3), (dict(rope_dim=32), -3), (dict(page_size=0), -3), (dict(num_pages=0), -3),
             (dict(num_pages=1 << 27, page_size=64), -3)]


def _append(lib, desc=None, c=FAKE, cs=512, ks=64, q=FAKE, qst=192, qsh=64, qo=FAKE, H=4, pos=FAKE, T=3, slots=FAKE,
            max_pos=8, cache=FAKE):
    d = desc or _desc()
    return lib.pkv_latent_append(c, cs, FAKE, ks, q, qst, qsh, qo, 192, 64, H, pos, FAKE, max_pos, slots, T, cache,
                                 ctypes.byref(d), None)


def _gather(lib, desc=None, B=1, total=4, width=1, out=FAKE, cu=FAKE):
    d = desc or _desc()
    return lib.pkv_latent_gather(FAKE, ctypes.byref(d), FAKE, width, cu, B, total, out, None)


def _attend(lib, desc=None, q=FAKE, B=1, T=2, H=16, W=4, max_kv=64, scale=0.1, out=FAKE, lse=None, ws=FAKE,
            ws_bytes=1 << 30):
    d = desc or _desc()
    return lib.pkv_latent_attention(q, FAKE, FAKE, FAKE, B, T, H, W, max_kv, FAKE, ctypes.byref(d), scale, out, lse,
                                    ws, ws_bytes, None)


def _prefill(lib, q=FAKE, kn=FAKE, kst=256, ksh=128, krs=64, B=1, Tq=2, Tk=4, H=2, dtype=binding.PKV_F16, scale=0.1,
             out=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return lib.pkv_latent_prefill(q, FAKE, kn, kst, ksh, FAKE, 256, 128, FAKE, krs, FAKE, B, Tq, Tk, H, dtype, scale,
                                  out, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", BAD_DESCS)
def test_bad_caches_are_refused(lib, kw, status):
    d = _desc(**kw)
    assert _append(lib, desc=d) == status
    assert _gather(lib, desc=d) == status
    assert _attend(lib, desc=d) == status
    assert lib.pkv_latent_attention_workspace_size(1, 1, 16, ctypes.byref(d)) == 0


def test_append_refusals(lib):
    assert _append(lib, T=-1) == -3 and _append(lib, max_pos=0) == -3
    assert _append(lib, cs=510) == -3 and _append(lib, ks=-8) == -3
    assert _append(lib, qst=100) == -3 and _append(lib, H=0) == -3
    assert _append(lib, c=None) == -1 and _append(lib, qo=None) == -1 and _append(lib, q=None) == -1
    assert _append(lib, pos=None) == -1 and _append(lib, slots=None) == -1 and _append(lib, cache=None) == -1
    assert _append(lib, c=ODD) == -7 and _append(lib, q=ODD) == -7 and _append(lib, slots=ctypes.c_void_p(4100)) == -7
    assert _append(lib, T=0) == 0


def test_gather_refusals(lib):
    assert _gather(lib, B=-1) == -3 and _gather(lib, total=-1) == -3 and _gather(lib, width=0) == -3
    assert _gather(lib, out=None) == -1 and _gather(lib, cu=None) == -1 and _gather(lib, out=ODD) == -7
    assert _gather(lib, total=0) == 0 and _gather(lib, B=0) == 0


def test_attention_refusals(lib):
    for kw in (dict(B=-1), dict(T=-1), dict(H=0), dict(H=4097), dict(max_kv=-1), dict(W=0), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 27, H=16),
               dict(W=1 << 28)):
        assert _attend(lib, **kw) == -3, kw
    assert _attend(lib, q=None) == -1 and _attend(lib, out=None) == -1 and _attend(lib, ws=None) == -1
    assert _attend(lib, q=ODD) == -7 and _attend(lib, out=ODD) == -7 and _attend(lib, lse=ODD) == -7
    assert _attend(lib, ws_bytes=16) == -6 and _attend(lib, ws=ctypes.c_void_p(4096 + 64)) == -6
    assert _attend(lib, T=0) == 0 and _attend(lib, B=0) == 0


def test_prefill_refusals(lib):
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(scale=0.0), dict(kst=100), dict(ksh=-8),
               dict(krs=4), dict(Tk=0), dict(Tq=1 << 30, H=4),
               dict(kst=0), dict(krs=0)):
        assert _prefill(lib, **kw) == -3, kw
    assert _prefill(lib, dtype=binding.PKV_F32) == -2 and _prefill(lib, dtype=binding.PKV_FP8_E4M3) == -2
    assert _prefill(lib, q=None) == -1 and _prefill(lib, kn=ODD) == -7
    assert _prefill(lib, ws_bytes=16) == -6
    assert _prefill(lib, Tq=0) == 0 and _prefill(lib, B=0) == 0


def test_workspace_sizes(lib):
    cache = torch.empty((4, 16, 576), dtype=torch.bfloat16)
    n = binding.latent_workspace_size(4, 10, 16, cache)
    assert n > 0 and n % 256 == 0
    n = binding.latent_prefill_workspace_size(4, 10, 16)
    assert n > 0 and n % 256 == 0
    with pytest.raises(binding.PagedKVError):
        binding.latent_workspace_size(4, 10, 0, cache)
    with pytest.raises(binding.PagedKVError):
        binding.latent_prefill_workspace_size(-1, 10, 16)


def test_a_workspace_for_a_large_call_serves_smaller_ones(lib):
    cache = torch.empty((4, 16, 576), dtype=torch.bfloat16)
    sizes = (1, 2, 17, 300, 4096, 8192)
    for B in (1, 64, 3000):
        for T in sizes:
            for H in (1, 5, 16, 128):
                for b, t, h in ((max(B // 2, 1), T, H), (B, max(T // 40, 1), H), (B, T, max(H // 5, 1)), (1, 1, 1)):
                    assert (binding.latent_prefill_workspace_size(b, t, h)
                            <= binding.latent_prefill_workspace_size(B, T, H)), (B, T, H, b, t, h)
                    assert (binding.latent_workspace_size(b, t, h, cache)
                            <= binding.latent_workspace_size(B, T, H, cache)), (B, T, H, b, t, h)


def test_binding_refuses_wrong_tensors(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    cache, q, tab = z(4, 16, 576), z(1, 8, 576), z(4, 32, 2, t=f32)
    cu, kv, pt = torch.tensor([0, 1], dtype=i32), z(1, t=i32), z(1, 1, t=i32)
    with pytest.raises(ValueError):                                        # host tensors
        binding.latent_attention(q, cu, kv, pt, cache, 0.1, 16)
    with pytest.raises(TypeError):
        binding.latent_attention(q, cu.long(), kv, pt, cache, 0.1, 16)
    with pytest.raises(ValueError):
        binding.latent_attention(q, cu, kv, pt, cache.transpose(0, 1), 0.1, 16)
    with pytest.raises(ValueError):
        binding.latent_gather(cache, pt, cu, 1)
    with pytest.raises(TypeError):
        binding.latent_gather(cache, pt.long(), cu, 1)
    with pytest.raises(ValueError):
        binding.latent_append(z(1, 512), z(1, 64), z(1, t=i32), tab, z(1, t=i64), cache)
    with pytest.raises(ValueError):
        binding.latent_prefill(z(1, 2, 192), cu, z(1, 2, 128), z(1, 2, 128), z(1, 64), cu, 0.1)
    with pytest.raises(TypeError):
        binding.latent_prefill(z(1, 2, 192), cu.long(), z(1, 2, 128), z(1, 2, 128), z(1, 64), cu, 0.1)


# ---------------------------------------------------------------------------
# GPU

def _cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _host(t):
    return t.double().cpu().numpy()


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _bounds(dtype, D, L, out, lse, spread, vmax):
    u = HALF_STEP[dtype]
    mass, dot = spread
    ds = D * 2.0 ** -23 * dot
    small = L * 2.0 ** -25 * vmax if dtype == "f16" else 0.0
    tol = u * np.abs(out) + (u + 2 * ds[..., None] + (L + 64) * 2.0 ** -23 + 2.0 ** -20) * mass + small
    return tol * (1 + u), ds + (L + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)


class Paged:
    """A tick over a latent cache: random rows in scattered pages, NaN in every
    slot that no sequence owns, -1 in unused table entries."""

    def __init__(self, dev, dtype, ld, H, P, q_lens, kv_lens, seed=0, pad_rows=0):
        g = np.random.default_rng(seed)
        self.dev, self.dtype, self.ld, self.H, self.P = dev, dtype, ld, H, P
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        need = [-(-L // P) for L in kv_lens]
        pages = sum(need) + 3
        perm = g.permutation(pages)
        self.table = np.full((len(need), max(need + [1]) + 1), -1, np.int32)
        cache = np.full((pages, P, ld + 64), np.nan, np.float32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            for j in range(kv_lens[b]):
                cache[self.table[b, j // P], j % P] = g.standard_normal(ld + 64)
        self.cache = torch.from_numpy(cache).to(dev, TYPES[dtype])
        self.total = int(sum(q_lens))
        self.q = torch.from_numpy(g.standard_normal((self.total + pad_rows, H, ld + 64)).astype(np.float32)).to(
            dev, TYPES[dtype])
        self.cu = _cum(q_lens)

    def call(self, **kw):
        return binding.latent_attention(self.q, _i32(self.cu, self.dev), _i32(self.kv_lens, self.dev),
                                        _i32(self.table, self.dev), self.cache, SCALE, max(self.kv_lens + [1]), **kw)

    def check(self, out, lse):
        out, lse, q, cache = _host(out), _host(lse), _host(self.q), _host(self.cache)
        for b, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0:
                continue
            rows = O.gather_sequence(cache, self.table[b], L)
            at = slice(int(self.cu[b]), int(self.cu[b]) + n)
            o, l, spread = O.attend_absorbed(q[at], rows, SCALE)
            tol, tol_lse = _bounds(self.dtype, self.ld + 64, L, o, l, spread, np.abs(rows).max())
            bad = np.abs(out[at] - o) > tol
            assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(out[at] - o).max())
            assert (np.abs(lse[at] - l) <= tol_lse).all(), (b, np.abs(lse[at] - l).max(), tol_lse.min())
            assert np.isfinite(out[at]).all()


ABSORBED = [
    # dtype, latent, heads, page, q_lens, kv_lens
    ("bf16", 512, 16, 64, [1], [1]),
    ("f16", 512, 16, 64, [1, 1, 1, 1], [63, 64, 65, 2]),
    ("bf16", 512, 128, 64, [1, 1, 1], [127, 128, 129]),
    ("bf16", 512, 128, 256, [1, 0, 1], [300, 77, 1000]),
    ("f16", 512, 1, 16, [1, 1], [33, 500]),
    ("bf16", 512, 3, 1, [2, 1], [70, 9]),
    ("bf16", 512, 20, 24, [5, 1, 3], [261, 24, 130]),
    ("f16", 512, 40, 48, [4, 2], [50, 513]),
    ("bf16", 512, 136, 100, [2, 1], [205, 99]),
    ("bf16", 512, 8, 128, [70, 1], [70, 5]),
    ("f16", 512, 16, 32, [33, 20], [161, 258]),
    ("bf16", 512, 64, 8, [3], [1000]),
    ("bf16", 512, 16, 3, [1], [400]),
    ("bf16", 512, 16, 64, [1], [20000]),
    ("f16", 512, 128, 64, [1], [5003]),
    ("bf16", 512, 32, 64, [5], [12 * 128 + 2]),
    ("bf16", 512, 16, 7, [9], [9]),
    ("bf16", 256, 16, 64, [1, 1], [1, 640]),
    ("f16", 256, 128, 16, [1, 2], [129, 400]),
    ("bf16", 256, 20, 24, [5, 1], [700, 25]),
    ("bf16", 256, 5, 100, [17], [3001]),
    ("bf16", 512, 16, 64, [1] * 90, [1 + 37 * k % 600 for k in range(90)]),
    ("f16", 256, 4, 64, [k % 4 for k in range(60)], [1 + 53 * k % 300 + k % 4 for k in range(60)]),
    # at most 16 rows a sequence on average, tiles of 16 rows
    ("bf16", 512, 8, 64, [2, 1, 1], [66, 64, 1]),
    ("f16", 512, 3, 16, [5, 4, 1], [33, 700, 32]),
    ("bf16", 512, 5, 100, [9, 0, 0, 0, 1], [9, 3, 1, 4, 31]),
    ("f16", 256, 16, 48, [1] * 7, [31, 32, 33, 95, 96, 97, 4000]),
    ("bf16", 256, 2, 1, [8, 7], [130, 65]),
    ("bf16", 512, 1, 32, [16], [16 * 64 + 9]),
    ("f16", 512, 16, 5, [1, 0], [7000, 12]),
    ("bf16", 512, 7, 256, [40] + [0] * 30 + [1], [3000] + [1] * 31),
    ("bf16", 512, 16, 64, [1] * 200, [1 + 97 * k % 500 for k in range(200)]),
    # short contexts: whole tiles, several a worker; the longest that are not cut, the shortest that are
    ("bf16", 512, 20, 64, [1] * 170, [1 + 41 * k % 300 for k in range(170)]),
    ("f16", 256, 40, 24, [k % 5 for k in range(100)], [5 + 37 * k % 400 for k in range(100)]),
    ("bf16", 256, 4, 64, [1] * 400, [1 + 11 * k % 64 for k in range(400)]),
    ("bf16", 512, 64, 64, [1] * 3, [640, 640, 5]), ("bf16", 512, 64, 64, [1] * 3, [641, 640, 5]),
    ("f16", 512, 8, 64, [1] * 2, [320, 7]), ("f16", 512, 8, 64, [1] * 2, [321, 7]),
    # rows by thread copies, more steps than slots, tails of every kind
    ("bf16", 512, 128, 16, [1, 1, 1], [1025, 640, 1000]),
    ("f16", 512, 33, 1, [1, 2], [777, 513]),
    ("bf16", 256, 130, 20, [1, 1], [1023, 1100]),
    ("f16", 256, 16, 16, [1, 1, 1], [1000, 65, 31]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ABSORBED, ids=lambda c: f"{c[0]}-{c[1]}-h{c[2]}-p{c[3]}-n{len(c[4])}-k{max(c[5])}")
def test_absorbed_matches_the_oracle(dev, case):
    t = Paged(dev, *case)
    out, lse = t.call()
    assert binding.device_status() == 0
    t.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("ld,heads,q_lens,kv_lens", [(256, 24, [1, 3], [40, 200]), (512, 24, [1, 3], [40, 200]),
                                                     (256, 4, [1, 2], [40, 200]), (512, 3, [2, 1, 1], [40, 3000, 9])])
def test_absorbed_leaves_padding_rows_and_unrequested_lse_alone(dev, ld, heads, q_lens, kv_lens):
    t = Paged(dev, "bf16", ld, heads, 16, q_lens, kv_lens, pad_rows=3)
    out = torch.full((t.total + 3, heads, ld), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((t.total + 3, heads), 5.0, device=dev)
    t.q[t.total:] = float("nan")
    t.call(out=out, lse=lse)
    assert binding.device_status() == 0
    assert (out[t.total:] == 5).all() and (lse[t.total:] == 5).all()
    t.check(out, lse)
    again, none = t.call(want_lse=False)
    assert none is None and torch.equal(again[:t.total], out[:t.total])


@pytest.mark.gpu
@pytest.mark.parametrize("ld,heads,seqs", [(512, 128, 300), (512, 40, 600), (256, 72, 500)])
def test_absorbed_many_segments_of_one_step(dev, ld, heads, seqs):
    """Workers with one segment of one step behind the other, where a row's sums are
    exchanged right before the next tile's maxima: every call gives the same bits, and the right ones."""
    t = Paged(dev, "bf16", ld, heads, 64, [1] * seqs, [1 + 7 * k % 128 for k in range(seqs)])
    first = t.call()
    for _ in range(20):
        again = t.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert binding.device_status() == 0
    t.check(*first)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld,page", [("bf16", 512, 16), ("f16", 512, 1), ("bf16", 256, 24)])
def test_absorbed_rows_behind_the_end_copied_by_threads(dev, dtype, ld, page):
    """Small pages, ends at every place of a step: the NaN rows behind an end are copied
    and then zeroed, whichever lane copied them."""
    kv = [1 + 3 * k for k in range(86)] + [1025 + 11 * k for k in range(12)]
    t = Paged(dev, dtype, ld, 64, page, [1] * len(kv), kv)
    first = t.call()
    for _ in range(10):
        again = t.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert binding.device_status() == 0
    t.check(*first)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [128, 12])
def test_absorbed_same_call_same_bits(dev, heads):
    t = Paged(dev, "bf16", 512, heads, 64, [1, 1, 2], [3000, 50, 700])
    first = t.call()
    for _ in range(3):
        again = t.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv", [(40, 90), (40, 9000), (4, 50), (4, 9000)])
def test_absorbed_nan_in_a_query_or_a_visible_key(dev, heads, kv):
    """NaN stays with the rows that it belongs to, in out and in lse."""
    t = Paged(dev, "bf16", 512, heads, 64, [1, 1, 1], [kv, 70, kv])
    good, good_lse = t.call()
    t.q[0, 1] = float("nan")
    key = kv - 3
    t.cache[int(t.table[2, key // 64]), key % 64, 5] = float("nan")
    out, lse = t.call()
    assert binding.device_status() == 0
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    assert out[2].isnan().all() and lse[2].isnan().all()
    for rows in ((0, slice(0, 1)), (0, slice(2, None)), (1, slice(None))):
        assert torch.equal(out[rows], good[rows]) and torch.equal(lse[rows], good_lse[rows])


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 4])
def test_absorbed_bad_data_skips_the_sequence(dev, heads):
    """A bad length or page skips that sequence's rows, a bad cu_seqlens_q every row."""
    t = Paged(dev, "bf16", 512, heads, 64, [1, 2, 1], [300, 4000, 100])
    good, good_lse = t.call()
    for what, bit in (("page", binding.DEV_BAD_PAGE), ("len", binding.DEV_BAD_LENGTHS), ("max", binding.DEV_BAD_LENGTHS)):
        table, kv = t.table.copy(), list(t.kv_lens)
        max_kv = max(kv)
        if what == "page":
            table[1, 40] = t.cache.shape[0]
        elif what == "len":
            kv[1] = 1
        else:
            max_kv = 3999
        out = torch.full_like(good, 9.0)
        lse = torch.full_like(good_lse, 9.0)
        binding.latent_attention(t.q, _i32(t.cu, dev), _i32(kv, dev), _i32(table, dev), t.cache, SCALE, max_kv,
                                 out=out, lse=lse)
        assert binding.device_status() == bit, what
        assert (out[1:3] == 9).all() and (lse[1:3] == 9).all(), what
        t2 = [(0, 1), (3, 4)]
        for a, b in t2:
            assert torch.isfinite(out[a:b]).all() and (out[a:b].float() - good[a:b].float()).abs().max() < 0.05, what
    for cu in ([0, 2, 1, 4], [1, 1, 3, 4], [0, 1, 3, 5]):
        out = torch.full_like(good, 9.0)
        binding.latent_attention(t.q, _i32(cu, dev), _i32(t.kv_lens, dev), _i32(t.table, dev), t.cache, SCALE, 4000,
                                 out=out)
        assert binding.device_status() == binding.DEV_BAD_LENGTHS, cu
        assert (out == 9).all(), cu


@pytest.mark.gpu
@pytest.mark.parametrize("heads,page", [(16, 64), (4, 64), (16, 8), (4, 8)])
def test_absorbed_short_contexts_bad_data(dev, heads, page):
    """The same where contexts are so short that no tile is cut."""
    t = Paged(dev, "bf16", 256, heads, page, [1, 2, 1], [60, 150, 100])
    good, good_lse = t.call()
    for what, bit in (("page", binding.DEV_BAD_PAGE), ("len", binding.DEV_BAD_LENGTHS)):
        table, kv = t.table.copy(), list(t.kv_lens)
        if what == "page":
            table[1, 1] = -1
        else:
            kv[1] = 151
        out, lse = torch.full_like(good, 9.0), torch.full_like(good_lse, 9.0)
        binding.latent_attention(t.q, _i32(t.cu, dev), _i32(kv, dev), _i32(table, dev), t.cache, SCALE, 150,
                                 out=out, lse=lse)
        assert binding.device_status() == bit, what
        assert (out[1:3] == 9).all() and (lse[1:3] == 9).all(), what
        assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3]), what


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 40])
def test_absorbed_pages_beyond_four_gigabytes(dev, heads):
    """Rows whose byte and element offsets pass 32 bits."""
    P, rows = 64, 4_200_000
    pages = rows // P
    cache = torch.empty((pages, P, 576), dtype=torch.bfloat16, device=dev)
    t = Paged(dev, "bf16", 512, heads, P, [1], [500])
    n = -(-500 // P)
    table = t.table.copy()
    for k in range(n):
        cache[pages - 1 - 3 * k] = t.cache[int(t.table[0, k])]
        table[0, k] = pages - 1 - 3 * k
    a = t.call()
    t.cache, t.table = cache, table
    b = t.call()
    assert binding.device_status() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    got = binding.latent_gather(cache, _i32(table, dev), _i32([0, 500], dev), 500)
    assert torch.equal(got, torch.cat([cache[int(p)] for p in table[0, :n]])[:500])


class Packed:
    """Packed chunks with expanded keys; NaN between and behind what belongs to them."""

    def __init__(self, dev, dtype, H, q_lens, kv_lens, seed=0, strided=True, pad=0):
        g = np.random.default_rng(seed)
        r = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(dev, TYPES[dtype])
        self.dev, self.dtype, self.H, self.q_lens, self.kv_lens = dev, dtype, H, list(q_lens), list(kv_lens)
        self.cu_q, self.cu_k = _cum(q_lens), _cum(kv_lens)
        self.Tq, self.Tk = int(self.cu_q[-1]) + pad, int(self.cu_k[-1]) + pad
        self.q = r(self.Tq, H, 192)
        if strided:
            up = r(self.Tk, H, 256)
            self.kn, self.v, self.kr = up[..., :128], up[..., 128:], r(self.Tk, 576)[:, 512:]
        else:
            self.kn, self.v, self.kr = r(self.Tk, H, 128), r(self.Tk, H, 128), r(self.Tk, 64)
        if pad:
            for x in (self.kn, self.v, self.kr):
                x[self.Tk - pad:] = float("nan")

    def call(self, **kw):
        return binding.latent_prefill(self.q, _i32(self.cu_q, self.dev), self.kn, self.v, self.kr,
                                      _i32(self.cu_k, self.dev), SCALE, **kw)

    def check(self, out, lse, only=None):
        out, lse, q, kn, v, kr = (_host(x) for x in (out, lse, self.q, self.kn, self.v, self.kr))
        for b, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0 or (only is not None and b not in only):
                continue
            a, k = slice(int(self.cu_q[b]), int(self.cu_q[b]) + n), slice(int(self.cu_k[b]), int(self.cu_k[b]) + L)
            o, l, spread = O.attend_expanded(q[a], kn[k], v[k], kr[k], SCALE)
            tol, tol_lse = _bounds(self.dtype, 192, L, o, l, spread, np.abs(v[k]).max())
            bad = np.abs(out[a] - o) > tol
            assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(out[a] - o).max())
            assert (np.abs(lse[a] - l) <= tol_lse).all(), (b, np.abs(lse[a] - l).max())


EXPANDED = [
    # dtype, heads, q_lens, kv_lens
    ("bf16", 1, [1], [1]),
    ("f16", 2, [1, 1], [1, 200]),
    ("bf16", 2, [127, 128, 129], [127, 128, 129]),
    ("f16", 1, [255, 256, 257], [255, 256, 257]),
    ("bf16", 3, [5, 0, 60], [300, 40, 61]),
    ("f16", 2, [300, 17], [700, 145]),
    ("bf16", 1, [600], [1111]),
    ("bf16", 5, [130, 1, 2], [258, 385, 128]),
    ("f16", 16, [33], [95]),
    ("bf16", 1, [k % 5 for k in range(40)], [k % 5 + 3 * k for k in range(40)]),
    # whole tiles of 512 rows, and what is left over (more than 256 rows, or fewer)
    ("bf16", 1, [511, 512, 513], [511, 600, 640]),
    ("f16", 2, [767, 768, 769], [767, 900, 769]),
    ("bf16", 1, [1200], [1333]),
    # enough tiles for every pair of CTAs: few rows of two heads go together
    ("bf16", 81, [100, 3], [200, 131]),
    ("f16", 80, [200, 600], [200, 700]),
    ("bf16", 161, [1, 129], [300, 129]),
    # few tiles and many keys: the keys are split, and some parts hold no key of some rows
    ("bf16", 1, [5], [5000]),
    ("f16", 3, [300, 20], [3000, 1500]),
    ("bf16", 2, [700], [2100]),
    ("bf16", 1, [2048], [2048]),
    ("f16", 1, [1300, 1, 40], [1300, 900, 1025]),
    ("bf16", 5, [256, 0, 257], [1153, 50, 1024]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("strided", [True, False])
@pytest.mark.parametrize("case", EXPANDED, ids=lambda c: f"{c[0]}-h{c[1]}-n{len(c[2])}-q{max(c[2])}-k{max(c[3])}")
def test_expanded_matches_the_oracle(dev, case, strided):
    t = Packed(dev, *case, strided=strided)
    out, lse = t.call()
    assert binding.device_status() == 0
    t.check(out, lse)


@pytest.mark.gpu
def test_expanded_takes_views(dev):
    """Keys and values laid out head by head, or one key and value for all heads."""
    t = Packed(dev, "bf16", 3, [40, 50, 300], [100, 50, 777], strided=False)
    out, lse = t.call()
    kn, v = t.kn, t.v
    t.kn, t.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (kn, v))
    again = t.call()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    t.kn, t.v = kn[:, :1].expand(-1, 3, -1), v[:, 1:2].expand(-1, 3, -1)
    got = t.call()
    assert binding.device_status() == 0
    t.check(*got)
    t.kn = kn[:1].expand(kn.shape[0], -1, -1)
    with pytest.raises(binding.PagedKVError):          # one key row for all tokens
        t.call()


@pytest.mark.gpu
def test_expanded_other_rows_never_reach_a_row(dev):
    """NaN in another sequence's keys and values, and behind the last one, stays there."""
    t = Packed(dev, "bf16", 2, [40, 50, 30], [100, 50, 77], pad=9)
    for x in (t.kn, t.v, t.kr):
        x[100:150] = float("nan")
    out = torch.full((t.Tq, 2, 128), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((t.Tq, 2), 5.0, device=dev)
    t.call(out=out, lse=lse)
    assert binding.device_status() == 0
    t.check(out, lse, only=(0, 2))
    assert (out[120:] == 5).all() and (lse[120:] == 5).all()
    assert torch.isnan(out[40:90]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [200, 6000])
def test_expanded_nan_in_a_query_or_a_visible_key(dev, kv):
    """NaN stays with the rows that it belongs to, in out and in lse."""
    t = Packed(dev, "bf16", 4, [3, 2], [kv, kv])
    good, good_lse = t.call()
    t.q[0, 1] = float("nan")
    t.kn[kv + 7, 2, 3] = float("nan")
    out, lse = t.call()
    assert binding.device_status() == 0
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    assert out[3:, 2].isnan().all() and lse[3:, 2].isnan().all()
    keep = torch.ones((5, 4), dtype=torch.bool, device=dev)
    keep[0, 1] = False
    keep[3:, 2] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])


@pytest.mark.gpu
def test_expanded_bad_lengths(dev):
    t = Packed(dev, "bf16", 2, [40, 50, 30], [100, 50, 77])
    good, _ = t.call()
    out = torch.full_like(good, 9.0)
    binding.latent_prefill(t.q, _i32(t.cu_q, dev), t.kn, t.v, t.kr, _i32([0, 100, 149, 227], dev), SCALE, out=out)
    assert binding.device_status() == binding.DEV_BAD_LENGTHS
    assert (out[40:90] == 9).all() and torch.equal(out[:40], good[:40]) and torch.isfinite(out[90:]).all()
    for cq, ck in (([0, 40, 30, 120], t.cu_k), (t.cu_q, [0, 100, 90, 227]), ([0, 40, 90, 121], t.cu_k),
                   (t.cu_q, [0, 100, 150, 228]), ([1, 40, 90, 120], t.cu_k), (t.cu_q, [2, 100, 150, 227])):
        out = torch.full_like(good, 9.0)
        binding.latent_prefill(t.q, _i32(cq, dev), t.kn, t.v, t.kr, _i32(ck, dev), SCALE, out=out)
        assert binding.device_status() == binding.DEV_BAD_LENGTHS, (cq, ck)
        assert (out == 9).all(), (cq, ck)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld,T,H,P", [("bf16", 512, 1, 1, 1), ("f16", 512, 33, 16, 16), ("bf16", 256, 70, 3, 24),
                                            ("f16", 256, 9, 128, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_append_matches_the_oracle(dev, dtype, ld, T, H, P, in_place):
    """Rows land in their slots and nowhere else; rotated values are within half
    a step of the exact rotation (fp32 angles and products add 2^-22 of the pair)."""
    g = np.random.default_rng(T)
    r = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(dev, TYPES[dtype])
    pages = -(-2 * T // P) + 1
    cache = r(pages, P, ld + 64)
    slots = g.permutation(pages * P)[:T].astype(np.int64)
    slots[::7] = -1
    pos = g.integers(0, 5000, T).astype(np.int32)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 5000)).to(dev)
    c, kr, wide = r(T, ld), r(T, ld + 64)[:, ld:], r(T, H, 192)
    q = wide[..., 128:]
    before = wide.clone()
    want = O.append(_host(cache), _host(c), _host(kr), pos, slots, 10000.0)
    want_q = apply_rope(_host(q), pos, 10000.0)
    big = r(T, H, ld + 64)
    kept = big.clone()
    q_out = q if in_place else big[..., ld:]
    got = binding.latent_append(c, kr, torch.from_numpy(pos).to(dev), table, torch.from_numpy(slots).to(dev), cache,
                                q_rope=q, q_out=q_out)
    assert binding.device_status() == 0 and got is q_out
    u = HALF_STEP[dtype]
    pair = lambda x: np.abs(x[..., :32]) + np.abs(x[..., 32:])
    near = lambda a, b: (np.abs(a - b) <= u * np.abs(b) + 2.0 ** -22 * np.concatenate([pair(b)] * 2, -1) + 2.0 ** -25).all()
    assert np.array_equal(_host(cache)[..., :ld], want[..., :ld])
    assert near(_host(cache)[..., ld:], want[..., ld:]) and near(_host(q_out), want_q)
    if in_place:
        assert torch.equal(wide[..., :128], before[..., :128])
    else:
        assert torch.equal(wide, before) and torch.equal(big[..., :ld], kept[..., :ld])


@pytest.mark.gpu
def test_append_without_queries_and_bad_tokens(dev):
    cache = torch.zeros((4, 8, 320), dtype=torch.float16, device=dev)
    c, kr = torch.ones((3, 256), dtype=torch.float16, device=dev), torch.ones((3, 64), dtype=torch.float16, device=dev)
    q = torch.full((3, 2, 64), 3.0, dtype=torch.float16, device=dev)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 16)).to(dev)
    i64 = lambda *a: torch.tensor(a, dtype=torch.int64, device=dev)
    assert binding.latent_append(c, kr, _i32([0, 0, 0], dev), table, i64(31, -1, 0), cache) is None
    assert binding.device_status() == 0
    rows = cache.view(32, 320)
    assert (rows[[0, 31]] == 1).all() and rows.count_nonzero() == 640
    out = torch.full_like(q, 7.0)
    cache.zero_()
    binding.latent_append(c, kr, _i32([16, 0, -1], dev), table, i64(1, 32, 2), cache, q_rope=q, q_out=out)
    assert binding.device_status() == binding.DEV_BAD_SLOT | binding.DEV_BAD_POSITION
    assert cache.count_nonzero() == 0 and (out[[0, 2]] == 7).all() and (out[1] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld,P,lens", [("bf16", 512, 1, [1]), ("f16", 512, 64, [64, 0, 65, 1000, 0]),
                                             ("bf16", 256, 24, [0, 23, 24, 25, 500]), ("f16", 256, 100, [7] * 70)])
def test_gather_is_bit_exact(dev, dtype, ld, P, lens):
    t = Paged(dev, dtype, ld, 1, P, [0] * len(lens), lens)
    cu = _cum(lens)
    n = int(cu[-1])
    out = torch.full((n + 5, ld + 64), 4.0, dtype=TYPES[dtype], device=dev)
    binding.latent_gather(t.cache, _i32(t.table, dev), _i32(cu, dev), n + 5, out=out)
    assert binding.device_status() == 0
    cache = _host(t.cache)
    want = np.concatenate([O.gather_sequence(cache, t.table[b], L) for b, L in enumerate(lens)])
    assert np.array_equal(_host(out[:n]), want) and (out[n:] == 4).all()


@pytest.mark.gpu
def test_gather_bad_data(dev):
    t = Paged(dev, "bf16", 256, 1, 8, [0, 0], [20, 20])
    good = binding.latent_gather(t.cache, _i32(t.table, dev), _i32([0, 20, 40], dev), 40)
    table = t.table.copy()
    table[0, 1] = -1
    out = torch.full_like(good, 4.0)
    binding.latent_gather(t.cache, _i32(table, dev), _i32([0, 20, 40], dev), 40, out=out)
    assert binding.device_status() == binding.DEV_BAD_PAGE
    assert (out[8:16] == 4).all() and torch.equal(out[:8], good[:8]) and torch.equal(out[16:], good[16:])
    for cu in ([0, 30, 20], [1, 20, 40], [0, 20, 41]):
        out = torch.full_like(good, 4.0)
        binding.latent_gather(t.cache, _i32(t.table, dev), _i32(cu, dev), 40, out=out)
        assert binding.device_status() == binding.DEV_BAD_LENGTHS and (out == 4).all(), cu
    out = torch.full((60, 320), 4.0, dtype=torch.bfloat16, device=dev)     # 40 rows from a table of 4 pages of 8
    binding.latent_gather(t.cache, _i32(t.table, dev), _i32([0, 40, 60], dev), 60, out=out)
    assert binding.device_status() == binding.DEV_BAD_LENGTHS
    assert (out[:40] == 4).all() and torch.equal(out[40:], good[20:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld,H,P", [("bf16", 512, 16, 64), ("f16", 256, 5, 24)])
def test_a_tick_through_both_forms(dev, dtype, ld, H, P):
    """A tick as a server runs it: new tokens appended (keys and queries rotated),
    a chunk through gather, up-projection and the expanded form, a decode row
    through the absorbed form, both against one computation in 64 bits."""
    g = np.random.default_rng(7)
    r = lambda *s, k=1.0: torch.from_numpy((k * g.standard_normal(s)).astype(np.float32)).to(dev, TYPES[dtype])
    kv, ql = [90, 200], [1, 70]                          # packed: the decode row first
    need = [-(-L // P) for L in kv]
    perm = g.permutation(sum(need) + 2)
    pages = [list(map(int, perm[:need[0]])), list(map(int, perm[need[0]:sum(need)]))]
    pk = binding.pack_tick(ql, kv, pages, P, sum(need) + 2)
    T = sum(ql)
    cache = r(sum(need) + 2, P, ld + 64)
    c, kr, q = r(T, ld), r(T, 64), r(T, H, 192)
    wk, wv = r(H, ld, 128, k=ld ** -0.5), r(H, ld, 128, k=ld ** -0.5)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 256)).to(dev)
    pos = binding.tick_positions(pk["cu_seqlens_q"], pk["kv_lens"])
    rows64 = O.append(_host(cache), _host(c), _host(kr), pos, pk["slot_mapping"], 10000.0)
    q64 = _host(q)
    q64[..., 128:] = apply_rope(q64[..., 128:], pos, 10000.0)

    binding.latent_append(c, kr, _i32(pos, dev), table, torch.from_numpy(pk["slot_mapping"]).to(dev), cache,
                          q_rope=q[..., 128:], q_out=q[..., 128:])
    # the chunk: gather, up-project, expanded attention
    rows = binding.latent_gather(cache, _i32(pk["page_tables"][1:], dev), _i32([0, kv[1]], dev), kv[1])
    up = torch.einsum("lc,hcd->lhd", rows[:, :ld], torch.cat([wk, wv], -1))
    e, _ = binding.latent_prefill(q[1:].contiguous(), _i32([0, ql[1]], dev), up[..., :128], up[..., 128:],
                                  rows[:, ld:], _i32([0, kv[1]], dev), SCALE)
    # the decode row: absorb, attend the pages, project the values
    qa = torch.cat([torch.einsum("nhd,hcd->nhc", q[:1, :, :128], wk), q[:1, :, 128:]], -1).contiguous()
    a, _ = binding.latent_attention(qa, _i32([0, 1], dev), _i32(kv[:1], dev), _i32(pk["page_tables"][:1], dev), cache,
                                    SCALE, kv[0])
    a = torch.einsum("nhc,hcd->nhd", a, wv)
    assert binding.device_status() == 0
    wk64, wv64 = _host(wk), _host(wv)
    got = np.concatenate([_host(a), _host(e)])
    for b, at in ((0, slice(0, 1)), (1, slice(1, T))):
        full = O.gather_sequence(rows64, pk["page_tables"][b], kv[b])
        kn, v = (np.einsum("lc,hcd->lhd", full[:, :ld], w) for w in (wk64, wv64))
        want, _, (mass, dot) = O.attend_expanded(q64[at], kn, v, full[:, ld:], SCALE)
        # Scores: the queries' and keys' rotary parts, the up-projected keys (or the
        # absorbed queries) are each rounded to u, so a score is off by 2 u of its
        # absolute dot product (in the absorbed form of the wider one, which the
        # up-projection of |q| and |c| bounds); values and outputs: three more roundings.
        wide = np.einsum("nhd,hcd->nhc", np.abs(q64[at][..., :128]), np.abs(wk64))
        dot = np.maximum(dot, SCALE * np.einsum("nhc,c->nh", wide, np.abs(full[:, :ld]).max(0)))
        u = HALF_STEP[dtype]
        vmass = np.einsum("c,hcd->hd", np.abs(full[:, :ld]).max(0), np.abs(wv64))
        assert (np.abs(got[at] - want) <= u * (4 * dot[..., None] * mass + 3 * vmass)).all(), b


def _rel(got, want):
    return np.linalg.norm(np.asarray(got, np.float64) - want) / np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld,H,P", [("bf16", 512, 16, 64), ("f16", 256, 5, 24), ("bf16", 256, 128, 16)])
def test_every_stage_of_a_tick_on_what_it_read(dev, dtype, ld, H, P):
    """Append, gather, both attention forms, each against 64 bits on the tensors that it
    read, so that the bounds of one call apply; and both forms of the same rows against one another.

    The forms differ by roundings of half a step at most, uniform in +-u: root mean square
    u / sqrt(3) each, of the keys or the absorbed queries (through the scores, whose
    products then weigh 0.8 and less), the values, the weights, and the results before and after the
    value projection. Eight of them make 8 ** 0.5 u / 3 ** 0.5 = 1.6 u of relative error in the
    2-norm; 4 u leaves a factor of 2.5. Results of a wrong page, position or head are off by more than 0.2."""
    g = np.random.default_rng(11)
    r = lambda *s, k=1.0: torch.from_numpy((k * g.standard_normal(s)).astype(np.float32)).to(dev, TYPES[dtype])
    kv, ql = [90, 137, 200], [1, 2, 70]
    need = [-(-L // P) for L in kv]
    perm = list(map(int, g.permutation(sum(need) + 2)))
    ends = np.cumsum([0] + need)
    pages = [perm[ends[b]:ends[b + 1]] for b in range(3)]
    pk = binding.pack_tick(ql, kv, pages, P, sum(need) + 2)
    T, cu, tables = sum(ql), pk["cu_seqlens_q"], pk["page_tables"]
    assert list(pk["kv_lens"]) == kv
    cache = r(sum(need) + 2, P, ld + 64)
    c, kr, q = r(T, ld), r(T, 64), r(T, H, 192)
    wk, wv = r(H, ld, 128, k=ld ** -0.5), r(H, ld, 128, k=ld ** -0.5)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 256)).to(dev)
    pos = binding.tick_positions(cu, pk["kv_lens"])
    before, q_before = _host(cache), _host(q)
    binding.latent_append(c, kr, _i32(pos, dev), table, torch.from_numpy(pk["slot_mapping"]).to(dev), cache,
                          q_rope=q[..., 128:], q_out=q[..., 128:])
    u = HALF_STEP[dtype]
    want = O.append(before, _host(c), _host(kr), pos, pk["slot_mapping"], 10000.0)
    after = _host(cache)
    assert np.array_equal(after[..., :ld], want[..., :ld])
    turned = want[..., ld:].reshape(-1, 64)
    pair = lambda x: np.concatenate([np.abs(x[..., :32]) + np.abs(x[..., 32:])] * 2, -1)
    near = lambda a, b: (np.abs(a - b) <= u * np.abs(b) + 2.0 ** -22 * pair(b) + 2.0 ** -25).all()
    assert near(after[..., ld:].reshape(-1, 64), turned)
    turned_q = apply_rope(q_before[..., 128:], pos, 10000.0)
    assert near(_host(q)[..., 128:], turned_q) and np.array_equal(_host(q)[..., :128], q_before[..., :128])
    assert not near(_host(q)[..., 128:], q_before[..., 128:])

    total = sum(kv)
    cu_k = _cum(kv)
    rows = binding.latent_gather(cache, _i32(tables, dev), _i32(cu_k, dev), total)
    packed = np.concatenate([O.gather_sequence(after, tables[b], kv[b]) for b in range(3)])
    assert np.array_equal(_host(rows), packed)

    up = torch.einsum("lc,hcd->lhd", rows[:, :ld], torch.cat([wk, wv], -1))
    e, e_lse = binding.latent_prefill(q, _i32(cu, dev), up[..., :128], up[..., 128:], rows[:, ld:], _i32(cu_k, dev), SCALE)
    qa = torch.cat([torch.einsum("nhd,hcd->nhc", q[..., :128], wk), q[..., 128:]], -1).contiguous()
    a, a_lse = binding.latent_attention(qa, _i32(cu, dev), _i32(kv, dev), _i32(tables, dev), cache, SCALE, max(kv))
    assert binding.device_status() == 0
    q64, up64, qa64 = _host(q), _host(up), _host(qa)
    for b in range(3):
        at, k = slice(int(cu[b]), int(cu[b + 1])), slice(int(cu_k[b]), int(cu_k[b + 1]))
        own = packed[k]
        for got, got_lse, (o, l, spread), D, v in (
                (e, e_lse, O.attend_expanded(q64[at], up64[k, :, :128], up64[k, :, 128:], own[:, ld:], SCALE), 192, up64[k]),
                (a, a_lse, O.attend_absorbed(qa64[at], own, SCALE), ld + 64, own)):
            tol, tol_lse = _bounds(dtype, D, kv[b], o, l, spread, np.abs(v).max())
            assert (np.abs(_host(got)[at] - o) <= tol).all() and (np.abs(_host(got_lse)[at] - l) <= tol_lse).all(), b
            assert not (np.abs(o) <= tol).mean() > 0.5, b                    # zeros would not pass
        projected = _host(torch.einsum("nhc,hcd->nhd", a[at], wv))
        assert _rel(projected, _host(e)[at]) < 4 * u, (b, _rel(projected, _host(e)[at]) / u)
        # what a wrong page, an unturned query or a head out of place would give is far off
        other = packed[slice(int(cu_k[(b + 1) % 3]), int(cu_k[(b + 1) % 3 + 1]))][:kv[b]]
        wrong = np.concatenate([other, own[len(other):]])
        assert _rel(_host(a)[at], O.attend_absorbed(qa64[at], wrong, SCALE)[0]) > 0.2
        assert _rel(_host(a)[at], O.attend_absorbed(qa64[at][:, ::-1], own, SCALE)[0]) > 0.2


def _sink(t, kv, weight):
    """Keys of the row's own sequence that share `weight` of a first key that has nearly all
    of the softmax: 2^weight each. Returns the query and key entry that does it: q k = that score."""
    score = -weight * math.log(2.0) / SCALE
    return 16.0, score / 16.0


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv", [(40, 40000), (8, 40000), (40, 500), (8, 300)])
def test_absorbed_small_f16_weights_are_not_lost(dev, heads, kv):
    """A first key with nearly all of the weight, and the values in the others'. A weight's
    rounding is half a step where it is normal, and 2^-25 of a unit that is 2^-7 of
    the row's weight scale or less where it is not: 2^-32 max|v| a key."""
    t = Paged(dev, "f16", 256, heads, 64, [1], [kv])
    qv, kx = _sink(t, kv, -25.2)
    t.q.zero_()
    t.q[..., -1] = qv
    rows = t.cache.view(-1, 320)
    at = torch.from_numpy((t.table[0, np.arange(kv) // 64].astype(np.int64) * 64 + np.arange(kv) % 64)).to(dev)
    rows[at, -64:] = 0
    rows[at[0]] = 0
    rows[at[0], -1] = kx
    rows[at[1:], :256] = rows[at[1:], :256].abs()
    out, lse = t.call()
    assert binding.device_status() == 0
    own = O.gather_sequence(_host(t.cache), t.table[0], kv)
    o, l, (mass, dot) = O.attend_absorbed(_host(t.q), own, SCALE)
    u = HALF_STEP["f16"]
    ds = 320 * 2.0 ** -23 * dot[..., None]
    tol = u * np.abs(o) + (u + 2 * ds + (kv + 64) * 2.0 ** -23 + 2.0 ** -20) * mass + kv * 2.0 ** -32 * np.abs(own).max()
    tol = tol * (1 + u) + 2.0 ** -25                  # (results this small are subnormal themselves)
    assert (np.abs(_host(out) - o) <= tol).all(), (np.abs(_host(out) - o).max(), tol.min(), np.abs(o).max())
    assert np.abs(_host(lse) - l).max() <= ds.max() + (kv + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(l).max()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,q_len,kv", [(1, 3, 40000), (2, 300, 900), (90, 257, 700)])
def test_expanded_small_f16_weights_are_not_lost(dev, heads, q_len, kv):
    """As test_absorbed_small_f16_weights_are_not_lost."""
    t = Packed(dev, "f16", heads, [q_len], [kv], strided=False)
    qv, kx = _sink(t, kv, -25.2)
    t.q.zero_()
    t.q[..., -1] = qv
    t.kr.zero_()
    t.kr[0, -1] = kx
    t.v[0] = 0
    t.v.abs_()
    out, lse = t.call()
    assert binding.device_status() == 0
    o, l, (mass, dot) = O.attend_expanded(_host(t.q), _host(t.kn), _host(t.v), _host(t.kr), SCALE)
    u = HALF_STEP["f16"]
    ds = 192 * 2.0 ** -23 * dot[..., None]
    tol = (u * np.abs(o) + (u + 2 * ds + (kv + 64) * 2.0 ** -23 + 2.0 ** -20) * mass
           + kv * 2.0 ** -32 * float(t.v.abs().max())) * (1 + u) + 2.0 ** -25
    assert (np.abs(_host(out) - o) <= tol).all(), (np.abs(_host(out) - o).max(), tol.min(), np.abs(o).max())
    assert np.abs(_host(lse) - l).max() <= ds.max() + (kv + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(l).max()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv", [(40, 1), (40, 300), (40, 9000), (4, 1), (4, 50), (4, 9000)])
def test_absorbed_rows_whose_scores_are_all_minus_infinity(dev, heads, kv):
    """As the formula has it: the softmax of such a row is NaN, its log sum -inf; cut tiles or not."""
    t = Paged(dev, "bf16", 256, heads, 64, [1, 1], [kv, kv])
    t.q[..., -1] = 1.0
    good = t.call()
    at = t.table[0, np.arange(kv) // 64].astype(np.int64) * 64 + np.arange(kv) % 64
    t.cache.view(-1, 320)[torch.from_numpy(at).to(dev), -1] = -math.inf
    out, lse = t.call()
    assert binding.device_status() == 0
    assert out[0].isnan().all() and (lse[0] == -math.inf).all()
    assert torch.equal(out[1], good[0][1]) and torch.equal(lse[1], good[1][1])


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv", [(2, 4), (2, 300), (3, 6000), (90, 300)])
def test_expanded_rows_whose_scores_are_all_minus_infinity(dev, heads, kv):
    """As test_absorbed_rows_whose_scores_are_all_minus_infinity."""
    t = Packed(dev, "bf16", heads, [3, 2], [kv, kv])
    t.q[..., -1] = 1.0
    good = t.call()
    t.kr[:kv, -1] = -math.inf
    out, lse = t.call()
    assert binding.device_status() == 0
    assert out[:3].isnan().all() and (lse[:3] == -math.inf).all()
    assert torch.equal(out[3:], good[0][3:]) and torch.equal(lse[3:], good[1][3:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H", [("bf16", 2), ("f16", 1)])
def test_expanded_more_sequences_than_the_plan_sorts(dev, dtype, H):
    """2100 sequences of 0-3 rows, empty ones between them, one long chunk and one sequence
    with fewer keys than rows behind the first thousand."""
    q_lens = [k % 4 for k in range(2100)]
    kv_lens = [q + 7 * k % 30 for k, q in enumerate(q_lens)]
    q_lens[1500], kv_lens[1500] = 300, 700
    q_lens[1201], kv_lens[1201] = 3, 2
    t = Packed(dev, dtype, H, q_lens, kv_lens)
    out, lse = torch.full((t.Tq, H, 128), 9.0, dtype=TYPES[dtype], device=dev), torch.full((t.Tq, H), 9.0, device=dev)
    t.call(out=out, lse=lse)
    assert binding.device_status() == binding.DEV_BAD_LENGTHS
    rows = slice(int(t.cu_q[1201]), int(t.cu_q[1202]))
    assert (out[rows] == 9).all() and (lse[rows] == 9).all()
    t.check(out, lse, only=set(range(2100)) - {1201})


@pytest.mark.gpu
def test_graphs_replay_with_new_lengths_and_side_by_side(dev):
    """One captured decode tick serves new lengths and tables; two captured graphs
    with a workspace each give their results when replayed on two streams at once."""
    big = Paged(dev, "bf16", 512, 16, 64, [1, 1, 1], [900, 2000, 333])
    other = Paged(dev, "bf16", 512, 128, 64, [1, 1], [1500, 4000], seed=5)
    chunk = Packed(dev, "bf16", 4, [200, 30], [300, 200], seed=6)

    def captured(fn):
        fn()
        torch.cuda.synchronize()
        s, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            got = fn()
        return gr, got, s

    kv, tab, cu = _i32(big.kv_lens, dev), _i32(big.table, dev), _i32(big.cu, dev)
    ws = binding.alloc_latent_workspace(3, 3, 16, big.cache)
    out, lse = torch.empty((3, 16, 512), dtype=torch.bfloat16, device=dev), torch.empty((3, 16), device=dev)
    g1, _, s1 = captured(lambda: binding.latent_attention(big.q, cu, kv, tab, big.cache, SCALE, 4096, out=out, lse=lse,
                                                          workspace=ws))
    o_cu, o_kv, o_tab = _i32(other.cu, dev), _i32(other.kv_lens, dev), _i32(other.table, dev)
    g2, got2, s2 = captured(lambda: binding.latent_attention(other.q, o_cu, o_kv, o_tab, other.cache, SCALE, 4096))
    c_q, c_k = _i32(chunk.cu_q, dev), _i32(chunk.cu_k, dev)
    g3, got3, s3 = captured(lambda: binding.latent_prefill(chunk.q, c_q, chunk.kn, chunk.v, chunk.kr, c_k, SCALE))
    for lens in ([900, 2000, 333], [1, 64, 65], [899, 1999, 2]):
        kv.copy_(_i32(lens, dev))
        out.fill_(9)
        torch.cuda.synchronize()
        for _ in range(3):
            for gr, s in ((g1, s1), (g2, s2), (g3, s3)):
                with torch.cuda.stream(s):
                    gr.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        big.kv_lens = lens
        big.check(out, lse)
    other.check(*got2)
    chunk.check(*got3)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [40, 4])
def test_outputs_aligned_to_sixteen_bytes_only(dev, heads):
    def shifted(like):
        flat = torch.full((like.numel() + 8,), 9.0, dtype=like.dtype, device=dev)
        return flat, flat[8:].view(like.shape)
    for t in (Paged(dev, "bf16", 512, heads, 64, [1, 2], [300, 70]), Packed(dev, "bf16", heads, [300, 40], [400, 40])):
        good, good_lse = t.call()
        flat, out = shifted(good)
        assert out.data_ptr() % 32 == 16
        _, lse = t.call(out=out)
        assert torch.equal(out, good) and torch.equal(lse, good_lse) and (flat[:8] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,q_lens,kv_lens", [(4, [20, 0, 300, 1], [20, 7, 300, 90]), (3, [257], [5000]),
                                                  (16, [70, 5], [4000, 6000]), (2, [513, 40], [513, 2600])])
def test_expanded_calls_with_and_without_a_plan_agree(dev, heads, q_lens, kv_lens):
    """Small calls find their tiles by themselves; a call with more sequences than the GPU
    has pairs of CTAs takes the planning kernel. Same tiles, same bits; bad lengths are
    skipped by both."""
    t = Packed(dev, "bf16", heads, q_lens, kv_lens)
    few, few_lse = t.call()
    t.check(few, few_lse)
    t.cu_q = np.concatenate([t.cu_q, np.full(80, t.cu_q[-1], np.int32)])
    t.cu_k = np.concatenate([t.cu_k, np.full(80, t.cu_k[-1], np.int32)])
    many, many_lse = t.call()
    assert binding.device_status() == 0
    assert torch.equal(few, many) and torch.equal(few_lse, many_lse)
    good_k = t.cu_k
    for empties in (80, 0):
        t.cu_q, t.cu_k = t.cu_q[:len(q_lens) + 1 + empties], good_k[:len(q_lens) + 1 + empties].copy()
        t.cu_k[1] = q_lens[0] - 1            # fewer keys than rows: its rows are skipped
        out = torch.full_like(few, 9.0)
        t.call(out=out)
        assert binding.device_status() == binding.DEV_BAD_LENGTHS
        assert (out[:q_lens[0]] == 9).all() and torch.isfinite(out).all() and (out[q_lens[0]:] != 9).any(-1).all()
        t.cu_k[-1] = t.Tk + 1                # ends behind the keys: every row is skipped
        out.fill_(9.0)
        t.call(out=out)
        assert binding.device_status() == binding.DEV_BAD_LENGTHS
        assert (out == 9).all()


@pytest.mark.gpu
def test_eager_calls_on_two_streams_at_once(dev):
    ticks = [Paged(dev, "bf16", 512, 16, 64, [1, 1], [3000, 20], seed=1),
             Paged(dev, "f16", 512, 64, 16, [1, 2], [700, 2500], seed=2)]
    chunks = [Packed(dev, "bf16", 3, [70, 300], [90, 800], seed=k) for k in (3, 4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for t, c in zip(ticks, chunks):
            s = torch.cuda.Stream()
            got.append((t, t.call(stream=s)))
            got.append((c, c.call(stream=s)))
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    for t, (out, lse) in got:
        t.check(out, lse)


@pytest.mark.gpu
def test_no_rows_and_no_sequences(dev):
    t = Paged(dev, "bf16", 256, 4, 16, [0, 0], [5, 0])
    out, lse = t.call()
    assert out.shape == (0, 4, 256) and lse.shape == (0, 4)
    q, cu = torch.zeros((0, 2, 192), dtype=torch.bfloat16, device=dev), _i32([0, 0], dev)
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device=dev)
    out, lse = binding.latent_prefill(q, cu, k, k, k[:, 0, :64], cu, SCALE)
    assert out.shape == (0, 2, 128)
    none = lambda *shape, t=torch.bfloat16: torch.zeros(shape, dtype=t, device=dev)
    binding.latent_append(none(0, 256), none(0, 64), none(0, t=torch.int32), none(4, 32, 2, t=torch.float32),
                          none(0, t=torch.int64), t.cache)
    assert binding.device_status() == 0


@pytest.mark.gpu
def test_calls_on_a_stream_argument(dev):
    t = Paged(dev, "bf16", 512, 16, 64, [1], [700])
    c = Packed(dev, "f16", 2, [50], [90])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = t.call(stream=s)
    b = c.call(stream=s)
    s.synchronize()
    t.check(*a)
    c.check(*b)


@pytest.mark.gpu
@pytest.mark.parametrize("ld", [256, 512])
def test_absorbed_at_the_ends_of_the_ranges(dev, ld):
    """A pool of one slot; 4096 heads; thousands of sequences, most of them without rows."""
    for heads in (1, 4, 40):
        t = Paged(dev, "bf16", ld, heads, 1, [1], [1])
        t.cache, t.table = t.cache[int(t.table[0, 0]):][:1].contiguous(), np.zeros((1, 1), np.int32)
        out, lse = t.call()
        assert binding.device_status() == 0
        t.check(out, lse)
    t = Paged(dev, "f16", ld, 4096, 16, [2, 1], [70, 9])
    t.check(*t.call())
    lens = [1 + 5 * k % 90 for k in range(5000)]
    for heads, every in ((40, 7), (4, 3)):
        q_lens = [int(k % every == 0) for k in range(5000)]
        t = Paged(dev, "bf16", ld, heads, 16, q_lens, lens)
        t.check(*t.call())
    assert binding.device_status() == 0


@pytest.mark.gpu
def test_expanded_at_the_ends_of_the_ranges(dev):
    for heads, q_lens, kv_lens in ((4096, [3, 1], [40, 200]), (1, [1], [1]), (4095, [1], [130])):
        t = Packed(dev, "bf16", heads, q_lens, kv_lens)
        t.check(*t.call())
    assert binding.device_status() == 0


@pytest.mark.gpu
def test_one_workspace_for_calls_of_every_size(dev):
    """Allocated for a large call that splits nothing, used by calls that do, and by both absorbed kernels."""
    ws = torch.empty(binding.latent_prefill_workspace_size(100, 8192, 128), dtype=torch.uint8, device=dev)
    for case in (("bf16", 1, [5], [5000]), ("f16", 3, [300, 20], [3000, 1500]), ("bf16", 90, [100, 30], [400, 300])):
        t = Packed(dev, *case)
        t.check(*t.call(workspace=ws))
    ws = None
    for heads, q_lens, kv_lens in ((128, [1, 2], [3000, 700]), (4, [1, 2], [5000, 70]), (40, [1, 1], [90, 60])):
        t = Paged(dev, "bf16", 512, heads, 64, q_lens, kv_lens)
        if ws is None:
            ws = binding.alloc_latent_workspace(200, 200, 128, t.cache)
        t.check(*t.call(workspace=ws))
    assert binding.device_status() == 0
