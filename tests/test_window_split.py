"""Layers with a window: which rows of a call go to which kernel, and how each numbers its work. Every
row is written once, whatever the mix of sequences, and a cu_seqlens_q that breaks its rules
reaches nothing outside the call's rows."""
import numpy as np
import pytest
import torch

from paged_kv_attention_mapping_gb300 import binding

from test_window import Problem, _cum, _i32, dev, lib  # noqa: F401

TOP = 2 ** 31 - 8


# Differences of neighbours that are small counts in 32 bits only, between whole sequences.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,D", [("bf16", "bf16", 128), ("f16", "e4m3", 128), ("f32", "f32", 64)])
@pytest.mark.parametrize("q", [1, 4, 120])
def test_offsets_whose_difference_wraps(dev, t, cache, D, q):
    n = [q, 1, 1, 1, q, 130]
    p = Problem(dev, t, cache, 8, 2, D, 64, 60, 3, n, [200, 150, 300, 220, 260, 400])
    cu = _cum(n)
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
    for mid in ([TOP, -TOP, cu[4]], [TOP, -2 ** 31, cu[4]], [2 ** 31 - 1, -2 ** 31, cu[4]], [-2 ** 31, TOP, -TOP]):
        bad = np.array([0, cu[1], *mid, cu[5], cu[6]], np.int64).astype(np.int32)
        binding.window_attention(p.q, _i32(bad, dev), _i32(p.kv_lens, dev), _i32(p.tables, dev), p.kc, p.vc, p.scale, p.W,
                                 sinks=p.S, k_scale=p.ks, v_scale=p.vs, out=out, lse=lse)
        assert binding.device_status() & binding.DEV_BAD_LENGTHS
    again = p.run()                      # the device goes on, and nothing of the bad calls is left
    assert binding.device_status() == 0
    p.check(*again)


# Counts of rows at and next to 16, 32 and 48 columns, in calls of few and of many tiles.
@pytest.mark.gpu
@pytest.mark.parametrize("copies,Hkv", [(1, 2), (4, 8)])
@pytest.mark.parametrize("t,cache,D,G", [("bf16", "bf16", 128, 1), ("f16", "f16", 128, 3), ("bf16", "bf16", 128, 8),
                                         ("bf16", "bf16", 128, 16), ("f16", "f16", 64, 4), ("bf16", "bf16", 64, 16),
                                         ("bf16", "e4m3", 128, 2), ("f16", "e4m3", 128, 5), ("bf16", "e4m3", 128, 16)])
def test_rows_at_the_edges_of_the_rule(dev, t, cache, D, G, copies, Hkv):
    q = [x for c in (16, 32, 48) for x in (c // G, c // G + 1)] * copies
    kv = [x + (0, 37, 150)[i % 3] for i, x in enumerate(q)]
    p = Problem(dev, t, cache, G * Hkv, Hkv, D, 64, 50, 3, q, [max(x, 1) for x in kv], seed=G)
    out, lse = p.run(out=torch.full_like(p.q, float("nan")))
    assert binding.device_status() == 0
    p.check(out, lse, range(0, len(q), copies))
    assert not out.isnan().any() and not lse.isnan().any()


# More sequences than lanes: a lane counts the tiles of several, and looks one up in rounds of 32.
@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 1024, 1100])
def test_tiles_of_many_sequences(dev, cache, n):
    r = np.random.default_rng(n)
    q = [int(x) for x in r.choice([0, 0, 1, 7, 20, 49, 90], n)]
    q[-1] = 300                          # several tiles, the last ones of the call
    kv = [x + 1 + int(r.integers(0, 40)) for x in q]
    p = Problem(dev, "bf16", cache, 4, 2, 128, 16, 30, 2, q, kv, seed=n)
    out, lse = p.run(out=torch.full_like(p.q, float("nan")))
    assert binding.device_status() == 0
    assert not out.isnan().any() and not lse.isnan().any()
    p.check(out, lse, sorted({0, n // 2, n - 2, n - 1} | set(range(0, n, max(1, n // 12)))))
