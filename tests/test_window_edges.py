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


# A page outside the pool. Which rows need it goes by the window alone; rows fewer than 256 / group positions
# from one of those may be left out with it, all others are as if the page were good.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,G,P,W", [("bf16", "bf16", 4, 32, 20), ("f16", "f16", 4, 8, 20), ("bf16", "bf16", 1, 64, 50),
                                           ("bf16", "e4m3", 4, 32, 20), ("f16", "e4m3", 7, 16, 90),
                                           ("bf16", "bf16", 16, 32, 9)])
def test_a_bad_page_leaves_out_the_same_rows_every_time(dev, t, cache, G, P, W):
    n, D = 700, 128
    p = Problem(dev, t, cache, 2 * G, 2, D, P, W, 0, [n], [n])
    good, glse = p.run()
    p.check(good, glse)
    pos = np.arange(n)
    for page in (1, 3, n // P // 2, n // P):
        tables = p.tables.copy()
        tables[0, page] = p.N + 3
        needs = (pos >= page * P) & (pos - W < (page + 1) * P - 1)
        far = (np.abs(pos[:, None] - pos[needs]) >= 256 // G).all(1)
        left = None
        for _ in range(20):
            out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
            binding.window_attention(p.q, _i32([0, n], dev), _i32([n], dev), _i32(tables, dev), p.kc, p.vc, p.scale, W,
                                     k_scale=p.ks, v_scale=p.vs, out=out, lse=lse)
            assert binding.device_status() == binding.DEV_BAD_PAGE
            skipped = (out == 7).flatten(1).all(1).cpu().numpy()
            assert skipped[needs].all() and not skipped[far].any()
            # a row is left out whole or is what it would be
            kept = torch.from_numpy(~skipped).to(dev)
            assert (lse[~kept] == 7).all() and torch.equal(out[kept], good[kept]) and torch.equal(lse[kept], glse[kept])
            assert left is None or np.array_equal(left, skipped)
            left = skipped


# The page is that of the second query tile alone: the first (positions 0 .. 31) sees page 0 only.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,n", [("bf16", "bf16", 64), ("f16", "e4m3", 64), ("bf16", "e4m3", 47), ("f16", "f16", 200)])
def test_a_bad_page_of_the_second_query_tile(dev, t, cache, n):
    p = Problem(dev, t, cache, 8, 2, 128, 32, 1000, 0, [n], [n])
    good, _ = p.run()
    tables = p.tables.copy()
    tables[0, 1] = -1
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
    binding.window_attention(p.q, _i32([0, n], dev), _i32([n], dev), _i32(tables, dev), p.kc, p.vc, p.scale, p.W,
                             k_scale=p.ks, v_scale=p.vs, out=out, lse=lse)
    assert binding.device_status() == binding.DEV_BAD_PAGE
    assert torch.equal(out[:32], good[:32]) and (out[32:] == 7).all() and (lse[32:] == 7).all()


def _kernels(p):
    """The kernels that a call runs, after checking its results."""
    binding.set_kernel_timing(True)
    try:
        binding.kernel_times()
        out, lse = p.run()
        torch.cuda.synchronize()
        names = set(binding.kernel_times())
    finally:
        binding.set_kernel_timing(False)
    assert binding.device_status() == 0
    p.check(out, lse, sorted({0, len(p.q_lens) // 2, len(p.q_lens) - 1}))
    return names


# Short sequences become work tiles only where those are few and their windows short.
@pytest.mark.gpu
@pytest.mark.parametrize("G,W,q_lens,kv_lens,rows", [
    (4, 8000, [1, 600], [9000, 600], True),            # a long window in one CTA a head
    (4, 8000, [1, 511], [3000, 511], True),
    (2, 700, [1, 700], [2000, 700], True),             # 5 work tiles, one of them the short sequence's
    (1, 100, [1] * 32 + [8416], [150] * 32 + [8416], True),   # as many tiles again
    (4, 100, [1, 1100], [150, 1100], False),           # one tile a head beside 17
    (4, 8000, [600], [600], False),                    # nothing beside it
    (7, 300, [400, 700], [400, 900], False),
    (7, 3000, [400, 700], [3500, 900], True)])
def test_when_short_sequences_are_left_to_the_tiles(dev, G, W, q_lens, kv_lens, rows):
    p = Problem(dev, "bf16", "bf16", G, 1, 128, 64, W, 0, q_lens, kv_lens)
    assert _kernels(p) == ({"window_tiles", "window_rows"} if rows else {"window_tiles"})
