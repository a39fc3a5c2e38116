"""Layers with a window: stream order (inputs from the kernel right before a call, also when it lets
its successors start early; what comes behind a call must not reach what it still reads),
outputs aligned to 16 bytes only, the ends of the ranges."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from paged_kv_attention_mapping_gb300 import binding, build

from test_window import Problem, _append, _append_inputs, _attend, _check_append, _cum, _i32, dev, lib  # noqa: F401

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


# type, cache, Hq, Hkv, D, page, window, sinks, q_lens, kv_lens: single rows; rows beside chunks; chunks alone
SHAPES = [("bf16", "bf16", 8, 2, 64, 16, 50, 3, [1, 1, 1, 1], [300, 40, 1, 77]),
          ("f16", "f16", 8, 1, 128, 64, 600, 3, [1], [3000]),
          ("bf16", "bf16", 8, 2, 128, 64, 50, 3, [1, 120, 1, 30], [300, 150, 90, 400]),
          ("bf16", "e4m3", 8, 2, 128, 16, 50, 0, [1, 120, 1, 30], [300, 150, 90, 400]),
          ("f16", "f16", 6, 2, 64, 32, 90, 0, [300, 260], [300, 600]),
          ("f32", "f32", 4, 2, 64, 16, 20, 1, [1, 3], [100, 40])]


def _call(p, t, **kw):
    return binding.window_attention(t["q"], t["cu"], t["kv"], t["tab"], t["k"], t["v"], p.scale, p.W, sinks=p.S,
                                    k_scale=p.ks, v_scale=p.vs, **kw)


def _tensors(p, dev):
    return dict(q=p.q.clone(), cu=_i32(_cum(p.q_lens), dev), kv=_i32(p.kv_lens, dev), tab=_i32(p.tables, dev),
                k=p.kc.clone(), v=p.vc.clone())


@pytest.mark.gpu
@pytest.mark.parametrize("late", ["q", "cu", "kv", "tab", "k", "v"])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[0]}-{c[1]}-n{len(c[8])}-q{max(c[8])}")
def test_inputs_from_the_kernel_before(dev, late_write, case, late):
    p = Problem(dev, *case)
    t = _tensors(p, dev)
    good = t[late].clone()
    stale = {"cu": _i32(np.minimum(np.arange(len(p.q_lens) + 1), sum(p.q_lens)), dev),
             "kv": _i32(np.maximum(p.q_lens, 1), dev)}.get(late, torch.zeros_like(good))
    for _ in range(3):
        t[late].copy_(stale)
        _call(p, t)                      # (lines of the stale values may stay in the SMs' caches)
        torch.cuda.synchronize()
        binding.device_status()
        late_write(t[late], good)
        out, lse = _call(p, t)
        assert binding.device_status() == 0
        p.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHAPES[2:4], ids=lambda c: f"{c[0]}-{c[1]}")
def test_what_comes_behind_a_call_waits_for_all_of_it(dev, case):
    # long chunks and short rows: the row kernel is through long before the chunks are
    t, cache, Hq, Hkv, D, P, _, _, _, _ = case
    p = Problem(dev, t, cache, 32, 8, D, 64, 700, 3, [1, 1500, 1, 1400], [300, 1500, 90, 2500])
    x = _tensors(p, dev)
    want, wl = _call(p, x)
    T = 3000
    a = _append_inputs(dev, t, cache, T, 32, 8, D, 64, 64)
    slots = torch.arange(T, device=dev, dtype=torch.int64) % (p.N * 64)
    keep = {n: x[n].clone() for n in ("k", "v", "q")}
    q0 = x["q"][:T].clone() if x["q"].shape[0] >= T else None
    for _ in range(5):
        out, lse = _call(p, x)
        # the next layer's append over the slots just read, and over the queries
        binding.norm_rope_kv_append(a["q"], a["k"], a["v"], a["pos"], a["cs"], slots, x["k"], x["v"], k_scale=a["ks"],
                                    v_scale=a["vs"])
        src, dst = _i32([0], dev), _i32([p.N - 1], dev)
        binding.copy_pages([x["k"], x["v"]], src, dst)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        for n in keep:
            x[n].copy_(keep[n])
    assert binding.device_status() == 0 and (q0 is None or torch.equal(q0, keep["q"][:T]))


@pytest.mark.gpu
def test_append_and_pages_from_the_kernel_before(dev, late_write):
    x = _append_inputs(dev, "bf16", "bf16", 40, 8, 2, 64, 16, 32)
    x0 = {k: None if v is None else v.clone() for k, v in x.items()}
    for late in ("pos", "slots", "q", "k", "v", "cs", "qw"):
        good = x0[late].clone()
        x[late].zero_()
        x["kc"].copy_(x0["kc"])
        x["vc"].copy_(x0["vc"])
        torch.cuda.synchronize()
        late_write(x[late], good)
        got = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                          q_weight=x["qw"], k_weight=x["kw"], eps=1e-5)
        assert binding.device_status() == 0
        _check_append(x, x0, got, "bf16", "bf16", False, "qk", 1e-5)
    c = torch.arange(8 * 16 * 64, device=dev, dtype=torch.int32).view(8, 16, 64)
    want = c.clone()
    want[5] = want[2]
    for late, stale in (("src", [1]), ("dst", [4]), ("cache", None)):
        t = dict(src=_i32([2], dev), dst=_i32([5], dev), cache=c.clone())
        good = t[late].clone()
        t[late].copy_(torch.zeros_like(good) if stale is None else _i32(stale, dev))
        torch.cuda.synchronize()
        late_write(t[late], good)
        binding.copy_pages([t["cache"]], t["src"], t["dst"])
        assert torch.equal(t["cache"], want), late
    t, m = _i32([0, 3, -1], dev), _i32([3, 1, 2, 0], dev)
    good = m.clone()
    m.zero_()
    torch.cuda.synchronize()
    late_write(m, good)
    assert binding.remap_pages(t, m).tolist() == [3, 0, -1] and binding.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[0]}-{c[1]}-n{len(c[8])}-q{max(c[8])}")
def test_tensors_aligned_to_sixteen_bytes_only(dev, case):
    p = Problem(dev, *case)
    t = _tensors(p, dev)
    want, wl = _call(p, t)

    def moved(x):
        n = 16 // x.element_size()
        big = torch.zeros(x.numel() + n, dtype=x.dtype, device=dev)
        y = big[n:].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        return y

    for name in ("q", "k", "v"):
        t[name] = moved(t[name])
    out = moved(torch.full_like(p.q, 7.0))
    got, lse = _call(p, t, out=out)
    assert got is out and torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.gpu
@pytest.mark.parametrize("T,q_lens", [(3, [1, 1, 1]), (60, [1, 59])])
def test_many_heads(dev, T, q_lens):
    p = Problem(dev, "bf16", "bf16", 4096, 512, 64, 16, 30, 2, q_lens, [100, 59, 7][:len(q_lens)])
    out, lse = p.run()
    assert binding.device_status() == 0
    wo, wl, to, tl = p.want(0)
    assert (np.abs(out[:1].double().cpu().numpy() - wo) <= to).all()
    p.check(out, lse, [0])


@pytest.mark.gpu
@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("t,D", [("bf16", 128), ("f32", 64)])
def test_positions_near_the_end_of_their_range(dev, q, t, D):
    # a context of nearly 2^31 keys, all but the window's pages freed
    P, W = 1 << 16, 200
    width = (1 << 15) - 1
    L = width * P - 5
    p = Problem(dev, t, t, 8, 2, D, P, W, 0, [q], [300])
    tab = np.full((1, width), -1, np.int32)
    last = p.tables[0, 0]
    tab[0, -1] = last
    # the keys that Problem made at 300 - q - W + 1 .. 299 move to the end of the context
    n = W + q - 1
    kc, vc = p.kc.clone(), p.vc.clone()
    kc[last], vc[last] = math.nan, math.nan
    at = (L - 1) % P
    kc[last, at - n + 1:at + 1], vc[last, at - n + 1:at + 1] = p.kc[last, 300 - n:300], p.vc[last, 300 - n:300]
    out, lse = binding.window_attention(p.q, _i32([0, q], dev), _i32([L], dev), _i32(tab, dev), kc, vc, p.scale, W)
    assert binding.device_status() == 0
    p.check(out, lse)


def test_contexts_beyond_the_range_are_refused(lib):
    from test_window import _desc
    assert _attend(lib, desc=_desc(N=4, P=1 << 16), W=1 << 15) == -3
    assert _attend(lib, desc=_desc(N=4, P=1 << 16), W=(1 << 15) - 1, T=0) == 0


@pytest.mark.gpu
def test_two_threads_call_at_once(dev):
    import threading
    probs = [Problem(dev, *SHAPES[2], seed=3), Problem(dev, *SHAPES[4], seed=4), Problem(dev, *SHAPES[0], seed=5)]
    wants = [p.run() for p in probs]
    torch.cuda.synchronize()
    wrong = []

    def work(p, want):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = p.run()
                s.synchronize()
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    wrong.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(probs, wants)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong and binding.device_status() == 0


# ---------------------------------------------------------------------------
# windows and sinks beyond 32 bits mean what 2^31 - 1 does; negative ones are refused

BEYOND = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63]


@pytest.mark.parametrize("n", BEYOND)
def test_counts_beyond_32_bits_on_the_host(lib, n):
    args = ([1, 2], [9, 40], [[3, 0, 5], list(range(10))], 4, 10)
    for kw in (dict(window=n), dict(window=3, sinks=n)):
        with pytest.raises(binding.PagedKVError):       # every page is seen
            binding.pack_tick([1], [9], [[-1, 0, 5]], 4, 10, **kw)
        for a, b in zip(binding.pack_tick(*args, **kw), binding.pack_tick(*args)):
            assert np.array_equal(a, b)
        pool = binding.PagePool(10, 4)
        pages = [int(x) for x in pool.alloc(10)]
        assert pool.trim(pages, 40, **kw) == pages and pool.free_count() == 0
    for kw in (dict(window=-n), dict(window=-n + 5), dict(window=3, sinks=-n), dict(window=3, sinks=-n + 5)):
        with pytest.raises(binding.PagedKVError):
            binding.pack_tick(*args, **kw)
        with pytest.raises(binding.PagedKVError):
            pool.trim(pages, 40, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("n", BEYOND)
@pytest.mark.parametrize("case", [SHAPES[0], SHAPES[2], SHAPES[5]], ids=lambda c: f"{c[0]}-q{max(c[8])}")
def test_counts_beyond_32_bits(dev, case, n):
    p = Problem(dev, *case[:6], 2 ** 31 - 1, 0, *case[8:])
    want = p.run()
    p.check(*want)
    for p.W, p.S in ((n, 0), (1, n), (n, n)):
        got = p.run()
        p.W, p.S = 2 ** 31 - 1, 0       # (the same keys are seen)
        p.check(*got)
    for p.W, p.S in ((-n, 0), (-n + 5, 0), (1, -n), (1, -n + 5)):
        with pytest.raises(binding.PagedKVError):
            p.run()
    assert binding.device_status() == 0
