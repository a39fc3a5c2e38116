"""Layers with a window: hand-offs between work tiles, pages that only some tiles of a call need, the
choice of kernels in mixed and padded calls, what may follow a call, and forks of trimmed sequences."""
import numpy as np
import pytest
import torch

from paged_kv_attention_mapping_gb300 import binding

from test_window import Problem, _append_inputs, _cum, _i32, dev, lib  # noqa: F401


# Work tiles of one step each, of one query tile and of two: a tile's queries are loaded and (bf16 over
# e4m3) brought to f16 while the warps of the tile before it are still at theirs.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "bf16")])
def test_many_short_work_tiles(dev, t, cache):
    r = np.random.default_rng(7)
    n = 700
    q = [int(x) for x in r.choice([13, 20, 31, 32, 33, 50, 64], n)]
    kv = [x + int(r.integers(0, 40)) for x in q]
    p = Problem(dev, t, cache, 8, 2, 128, 16, 20, 0, q, kv, seed=7)
    out, lse = p.run(out=torch.full_like(p.q, float("nan")))
    assert binding.device_status() == 0
    p.check(out, lse, range(0, n, 23))
    assert not out.isnan().any() and not lse.isnan().any()
    for _ in range(20):
        again = p.run()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert binding.device_status() == 0
