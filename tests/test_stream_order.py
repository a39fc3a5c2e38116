"""Stream order: what a call reads may come from the kernel right before it, lengths
and tables included, also when that kernel lets its successors start early."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from paged_kv_attention_mapping_gb300 import binding, build

from test_latent import SCALE, TYPES, Packed, Paged, _i32, dev, lib  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
DELAY_US = 40


@pytest.fixture(scope="module")
def late_write(dev, tmp_path_factory):
    """late_write(dst, src): dst becomes src some time after the kernels behind it may start."""
    so = str(tmp_path_factory.mktemp("late") / "late_writer.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_writer.cu")
    subprocess.run([build.nvcc(), build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", src, "-o", so], check=True)
    fn = ctypes.CDLL(so).late_write
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p]

    def write(dst, src):
        assert dst.nbytes == src.nbytes and dst.nbytes % 4 == 0 and dst.is_contiguous() and src.is_contiguous()
        assert fn(src.data_ptr(), dst.data_ptr(), dst.nbytes // 4, DELAY_US, torch.cuda.current_stream().cuda_stream) == 0

    return write


ABSORBED = [
    # dtype, latent, heads, page, q_lens, kv_lens, lengths before, max_kv_len
    ("bf16", 512, 64, 64, [1, 1, 1], [3000, 700, 41], [1, 2, 3], 3000),             # 128-row tiles, cut
    ("f16", 256, 40, 24, [2, 1], [1500, 90], [2, 1], 1500),
    ("bf16", 512, 64, 64, [1] * 5, [100, 64, 65, 300, 2], [1] * 5, 300),            # whole tiles
    ("bf16", 512, 8, 64, [1, 2, 1], [5000, 66, 700], [1, 2, 3], 5000),              # 16-row tiles, cut
    ("f16", 512, 4, 16, [1] * 6, [60, 50, 40, 30, 20, 10], [1] * 6, 64),            # and whole
]


@pytest.mark.parametrize("case", ABSORBED, ids=lambda c: f"{c[0]}-{c[1]}-h{c[2]}-k{max(c[5])}")
def test_absorbed_lengths_from_the_kernel_before(dev, late_write, case):
    *shape, stale, max_kv = case
    t = Paged(dev, *shape)
    cu, new, tab = _i32(t.cu, dev), _i32(t.kv_lens, dev), _i32(t.table, dev)
    old = _i32(stale, dev)
    ws = binding.alloc_latent_workspace(len(t.kv_lens), t.total, t.H, t.cache)
    for _ in range(3):
        kv = old.clone()
        out, lse = torch.empty((t.total, t.H, t.ld), dtype=t.q.dtype, device=dev), torch.empty((t.total, t.H), device=dev)
        torch.cuda.synchronize()
        late_write(kv, new)
        binding.latent_attention(t.q, cu, kv, tab, t.cache, SCALE, max_kv, out=out, lse=lse, workspace=ws)
        assert binding.device_status() == 0
        t.check(out, lse)


def test_absorbed_rows_and_tables_from_the_kernel_before(dev, late_write):
    """cu_seqlens_q, page tables, queries and cache rows: each arrives late once."""
    for heads in (64, 4):
        t = Paged(dev, "bf16", 512, heads, 16, [1, 3, 2], [900, 300, 77])
        cu, kv, tab = _i32(t.cu, dev), _i32(t.kv_lens, dev), _i32(t.table, dev)
        one = _i32([0, 6, 6, 6], dev)
        for late, stale in ((cu, one), (tab, torch.zeros_like(tab)), (t.q, torch.zeros_like(t.q)),
                            (t.cache, torch.zeros_like(t.cache))):
            good = late.clone()
            late.copy_(stale)
            torch.cuda.synchronize()
            late_write(late, good)
            out, lse = binding.latent_attention(t.q, cu, kv, tab, t.cache, SCALE, 900)
            assert binding.device_status() == 0
            t.check(out, lse)


EXPANDED = [
    # dtype, heads, q_lens, kv_lens, empty sequences behind them
    ("bf16", 3, [40, 300, 1], [90, 777, 200], 0),      # every pair of CTAs finds its tile
    ("f16", 2, [70, 5], [4000, 6000], 0),              # the same, keys split
    ("bf16", 3, [40, 300, 1], [90, 777, 200], 80),     # planned
    ("bf16", 2, [70, 5], [4000, 6000], 80),            # planned and split
    ("f16", 90, [100, 30], [400, 300], 0),
]


@pytest.mark.parametrize("case", EXPANDED, ids=lambda c: f"{c[0]}-h{c[1]}-k{max(c[3])}-e{c[4]}")
@pytest.mark.parametrize("which", ["q", "k"])
def test_expanded_lengths_from_the_kernel_before(dev, late_write, case, which):
    dtype, heads, q_lens, kv_lens, empty = case
    t = Packed(dev, dtype, heads, q_lens, kv_lens)
    more = lambda cu: _i32(np.concatenate([cu, np.full(empty, cu[-1])]), dev)
    cu = {"q": more(t.cu_q), "k": more(t.cu_k)}
    good = cu[which].clone()
    n = len(q_lens)
    for _ in range(3):
        if which == "q":
            cu["q"].copy_(more(np.arange(n + 1)))                  # one row a sequence
        else:
            cu["k"].copy_(more(t.cu_q))                            # the chunks' own keys only
        torch.cuda.synchronize()
        late_write(cu[which], good)
        out, lse = binding.latent_prefill(t.q, cu["q"], t.kn, t.v, t.kr, cu["k"], SCALE)
        assert binding.device_status() == 0
        t.check(out, lse)


def test_append_and_gather_from_the_kernel_before(dev, late_write):
    t = Paged(dev, "bf16", 256, 1, 16, [0, 0], [100, 30])
    cu, tab = _i32([0, 100, 130], dev), _i32(t.table, dev)
    want = binding.latent_gather(t.cache, tab, cu, 130)
    for late, stale in ((cu, _i32([0, 1, 2], dev)), (tab, torch.zeros_like(tab)), (t.cache, torch.zeros_like(t.cache))):
        good = late.clone()
        late.copy_(stale)
        torch.cuda.synchronize()
        late_write(late, good)
        assert torch.equal(binding.latent_gather(t.cache, tab, cu, 130), want)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 64)).to(dev)
    c, kr = want[:9, :256].contiguous(), want[:9, 256:].contiguous()
    pos, slots = _i32(range(9), dev), torch.arange(3, 12, dtype=torch.int64, device=dev)
    cache = torch.zeros_like(t.cache)
    binding.latent_append(c, kr, pos, table, slots, cache)
    for late in (pos, slots, c, kr):
        good, got = late.clone(), torch.zeros_like(cache)
        late.zero_()
        torch.cuda.synchronize()
        late_write(late, good)
        binding.latent_append(c, kr, pos, table, slots, got)
        assert torch.equal(got, cache)
    assert binding.device_status() == 0


@pytest.mark.parametrize("dtype,ld,H,P", [("bf16", 512, 32, 64), ("f16", 256, 4, 24)])
def test_a_captured_tick_that_counts_on(dev, dtype, ld, H, P):
    """One graph of a decode tick whose lengths, positions, slots and cu_seqlens are computed
    on the device right before the calls that read them: append, absorbed attention,
    gather, up-projection, expanded attention. Each replay is one token further; both
    forms are checked against 64 bits on what they read."""
    start, steps = [P - 2, 130, 700], 4
    B = len(start)
    t = Paged(dev, dtype, ld, H, P, [1] * B, [n + steps for n in start])
    r = lambda *s, k=1.0: (k * torch.randn(s, generator=g)).to(TYPES[dtype]).to(dev)
    g = torch.Generator().manual_seed(3)
    kv, tab, cu_q = _i32(start, dev), _i32(t.table, dev), _i32(t.cu, dev)
    c, kr, q = r(B, ld), r(B, 64), r(B, H, ld + 64)
    w = r(H, ld, 256, k=ld ** -0.5)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 1024)).to(dev)
    total = sum(start) + B * steps
    rows = torch.zeros((total, ld + 64), dtype=TYPES[dtype], device=dev)
    ws = binding.alloc_latent_workspace(B, B, H, t.cache)
    got = {}

    def tick():
        kv.add_(1)
        pos = kv - 1
        slots = torch.gather(tab, 1, (pos // P).long()[:, None])[:, 0].long() * P + pos % P
        q_now = q.clone()
        binding.latent_append(c, kr, pos, table, slots, t.cache, q_rope=q[..., ld:], q_out=q_now[..., ld:])
        got["absorbed"] = binding.latent_attention(q_now, cu_q, kv, tab, t.cache, SCALE, 1024, workspace=ws)
        cu_k = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        cu_k[1:] = torch.cumsum(kv, 0)
        binding.latent_gather(t.cache, tab, cu_k, total, out=rows)
        up = torch.einsum("lc,hcd->lhd", rows[:, :ld], w)
        qe = q_now[..., -192:].contiguous()
        got["expanded"] = binding.latent_prefill(qe, cu_q, up[..., :128], up[..., 128:], rows[:, ld:], cu_k, SCALE)
        got["in"] = q_now, qe, up

    tick()                                   # (also warms the projection's library call up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tick()
    for step in range(2, steps + 1):         # (the capture itself ran nothing)
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        lens = [n + step for n in start]
        assert kv.tolist() == lens
        q_now, qe, up = got["in"]
        t.q, t.kv_lens = q_now, lens
        t.check(*got["absorbed"])
        e = Packed.__new__(Packed)
        e.dtype, e.H, e.q_lens, e.kv_lens = dtype, H, [1] * B, lens
        e.cu_q, e.cu_k = t.cu, np.concatenate([[0], np.cumsum(lens)])
        e.q, e.kn, e.v, e.kr = qe, up[..., :128], up[..., 128:], rows[:, ld:]
        e.check(*got["expanded"])


def _decode_tick(dev, dtype, Hq, Hkv, d, P, q_lens, kv_lens, seed=0):
    """Tensors of a paged K/V tick: q, caches, cu_seqlens_q, kv_lens, page tables."""
    g = torch.Generator(device=dev).manual_seed(seed)
    need = [-(-L // P) for L in kv_lens]
    pages = sum(need) + 1
    perm = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    table, at = np.zeros((len(need), max(need)), np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    r = lambda *s: torch.randn(s, generator=g, device=dev).to(TYPES[dtype])
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    return (r(int(cu[-1]), Hq, d), _i32(cu, dev), _i32(kv_lens, dev), _i32(table, dev), r(pages, P, Hkv, d),
            r(pages, P, Hkv, d))


PAGED = [
    # dtype, query heads, KV heads, head_dim, page, q_lens, kv_lens
    ("bf16", 32, 8, 128, 64, [1] * 6, [40, 900, 5000, 3, 77, 2100]),
    ("bf16", 16, 4, 128, 16, [1] * 4 + [300, 40], [40, 900, 30, 70, 400, 40]),
    ("f16", 8, 2, 64, 16, [1] * 700 + [9], [1 + 13 * k % 200 for k in range(700)] + [90]),
    ("bf16", 4, 4, 64, 8, [64] * 300, [64 + k for k in range(300)]),               # more tiles than are ranked
    ("bf16", 4, 4, 64, 8, [1] * 6200, [1 + k % 9 for k in range(6200)]),           # lengths not kept in shared memory
    ("bf16", 8, 2, 256, 16, [1, 2, 1], [40, 600, 9]),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"{c[0]}-h{c[1]}-d{c[3]}-n{len(c[5])}-k{max(c[6])}")
def test_paged_lengths_from_the_kernel_before(dev, late_write, case):
    dtype, Hq, Hkv, d, P, q_lens, kv_lens = case
    q, cu, kv, tab, kc, vc = _decode_tick(dev, *case)
    max_kv = max(kv_lens)
    out, lse = binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, max_kv)
    torch.cuda.synchronize()
    n = len(q_lens)
    ends = np.minimum(np.arange(n + 1), int(cu[-1]))
    ends[-1] = int(cu[-1])
    # lengths before: no sequence longer than its rows; all rows in one sequence; lengths that are refused
    for late, stale in ((kv, _i32(q_lens, dev)), (cu, _i32(ends, dev)), (kv, torch.full_like(kv, -5)),
                        (cu, torch.full_like(cu, 1 << 30))):
        good = late.clone()
        late.copy_(stale)
        torch.cuda.synchronize()
        late_write(late, good)
        again = binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, max_kv)
        assert binding.device_status() == 0
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("heads,kv_lens", [(64, [100, 64, 65, 300, 2]), (4, [60, 50, 40, 30, 20, 10])])
def test_one_workspace_for_latent_and_paged_calls(dev, heads, kv_lens):
    """Calls behind one another on a stream may share their workspace, and memory that a call
    read may be the next one's workspace."""
    t = Paged(dev, "bf16", 512, heads, 64, [1] * len(kv_lens), kv_lens)
    want = t.call()
    q, cu, kv, tab, kc, vc = _decode_tick(dev, "bf16", 16, 4, 128, 16, [1] * 4 + [300, 40], [40, 900, 30, 70, 400, 40])
    paged = binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900)
    chunk = Packed(dev, "bf16", 3, [40, 300], [400, 900])
    expanded = chunk.call()
    size = max(binding.workspace_size(6, 344, 16, kc, 900), t.q.nbytes,
               binding.latent_workspace_size(len(kv_lens), t.total, heads, t.cache),
               binding.latent_prefill_workspace_size(2, 340, 3))
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    args = _i32(t.cu, dev), _i32(t.kv_lens, dev), _i32(t.table, dev), t.cache, SCALE, max(kv_lens)
    k = chunk.cu_q, chunk.cu_k
    k = [_i32(x, dev) for x in k]
    q_in_ws = ws[:t.q.nbytes].view(torch.bfloat16).view(t.q.shape)
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append(binding.latent_attention(t.q, *args, workspace=ws) + want)
        got.append(binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900, workspace=ws) + paged)
        got.append(binding.latent_prefill(chunk.q, k[0], chunk.kn, chunk.v, chunk.kr, k[1], SCALE, workspace=ws)
                   + expanded)
        got.append(binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900, workspace=ws) + paged)
        q_in_ws.copy_(t.q)                   # the queries lie where the next call's plan goes
        got.append(binding.latent_attention(q_in_ws, *args) + want)
        got.append(binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900, workspace=ws) + paged)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    for i, (out, lse, good, good_lse) in enumerate(got):
        assert torch.equal(out, good) and torch.equal(lse, good_lse), i


def test_appended_rows_may_lie_in_the_next_workspace(dev):
    q, cu, kv, tab, kc, vc = _decode_tick(dev, "bf16", 16, 4, 128, 16, [1] * 4, [40, 900, 30, 70])
    T = 6000
    pool = torch.zeros((T // 16, 16, 4, 128), dtype=torch.bfloat16, device=dev)
    pool_v = torch.zeros_like(pool)
    rows = torch.randn((T, 4, 128), device=dev).to(torch.bfloat16)
    slots = torch.arange(T, dtype=torch.int64, device=dev)
    latents = rows.view(T, 512)
    latent_pool = torch.zeros((T // 16, 16, 576), dtype=torch.bfloat16, device=dev)
    table = torch.from_numpy(binding.rope_table(10000.0, 64, 16)).to(dev)
    pos, kr = torch.zeros(T, dtype=torch.int32, device=dev), rows[:, 0, :64]
    want = binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900)
    ws = torch.empty(max(rows.nbytes, binding.workspace_size(4, 4, 16, kc, 900)), dtype=torch.uint8, device=dev)
    src = ws[:rows.nbytes].view(torch.bfloat16).view(rows.shape)
    for latent in (False, True):
        src.copy_(rows)
        if latent:
            binding.latent_append(src.view(T, 512), kr, pos, table, slots, latent_pool)
        else:
            binding.kv_append(src, rows, slots, pool, pool_v)
        got = binding.paged_attention(q, cu, kv, tab, kc, vc, 0.1, 900, workspace=ws)
        assert binding.device_status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(pool.view(T, 4, 128), rows) and torch.equal(latent_pool.view(T, 576)[:, :512], latents)
