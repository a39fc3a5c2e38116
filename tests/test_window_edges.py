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


# Calls with no more rows than places for sequences, most of them idle: chunks in them share their keys too.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,Hq,Hkv,D,P,W,S", [
    ("bf16", "bf16", 8, 2, 128, 64, 90, 3), ("f16", "f16", 3, 3, 64, 16, 40, 0), ("bf16", "bf16", 10, 2, 128, 16, 50, 1),
    ("bf16", "bf16", 8, 1, 64, 8, 30, 0), ("f16", "f16", 16, 1, 128, 32, 20, 0), ("bf16", "bf16", 4, 4, 256, 24, 60, 9),
    ("bf16", "e4m3", 6, 2, 128, 16, 70, 2), ("f32", "f32", 4, 2, 64, 16, 30, 2)])
@pytest.mark.parametrize("q", [[0, 33, 0, 1, 7], [1, 1, 0, 16, 2, 0, 90], [130]])
def test_chunks_in_padded_calls(dev, t, cache, Hq, Hkv, D, P, W, S, q):
    rows = sum(q)
    q = q + [0] * (rows - len(q) + 2)
    kv = [x + (0, 5, 200)[i % 3] for i, x in enumerate(q)]
    p = Problem(dev, t, cache, Hq, Hkv, D, P, W, S, q, kv, pad=2)
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device=dev)
    p.run(out=out, lse=lse)
    assert binding.device_status() == 0 and p.q.shape[0] <= len(q)
    p.check(out, lse)
    assert (out[rows:] == 7).all() and (lse[rows:] == 7).all()


@pytest.mark.gpu
def test_a_chunk_in_a_padded_call_reads_its_keys_once_for_several_rows(dev):
    n, L = 400, 2400
    p = Problem(dev, "bf16", "bf16", 4, 4, 128, 64, 2000, 0, [n] + [0] * n, [L] + [1] * n)
    tables = np.full((n, p.tables.shape[1]), -1, np.int32)
    tables[:] = p.tables[0]
    kv = np.arange(L - n + 1, L + 1)
    calls = [([0, n] + [n] * n, p.kv_lens, p.tables), (list(range(n + 1)), kv, tables)]   # one chunk; single rows of the same keys
    times, outs = [], []
    for cu, kv, tab in calls:
        args = (p.q, _i32(cu, dev), _i32(kv, dev), _i32(tab, dev), p.kc, p.vc, p.scale, p.W)
        outs.append(binding.window_attention(*args)[0])
        best = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(5):
                binding.window_attention(*args)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        times.append(min(best))
    assert binding.device_status() == 0
    # 8 rows of a piece share each key: an eighth of the reads and products, and less than two thirds of the time
    assert times[0] < 0.67 * times[1], times


# Squares beyond the fp32 range: zeros, also where a weight or the rotation would carry the values beyond it.
@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,cache,D,rot", [("bf16", "bf16", 128, 64), ("f32", "f32", 64, 64), ("bf16", "e4m3", 256, 256)])
def test_append_of_heads_whose_squares_pass_the_range(dev, t, cache, D, rot, interleaved):
    x = _append_inputs(dev, t, cache, 20, 4, 2, D, 16, rot)
    q0 = x["q"].clone()
    x["q"][:, 1::2] = torch.where(q0[:, 1::2] < 0, -3e38, 3e38).to(q0.dtype)
    x["k"][:, 1] = x["q"][:, 1]
    x["qw"].fill_(2.0)
    x["kw"].fill_(-2.0)
    q = binding.norm_rope_kv_append(x["q"], x["k"], x["v"], x["pos"], x["cs"], x["slots"], x["kc"], x["vc"],
                                    q_weight=x["qw"], k_weight=x["kw"], eps=1e-6, interleaved=interleaved, k_scale=x["ks"],
                                    v_scale=x["vs"])
    assert binding.device_status() == 0
    assert (q[:, 1::2] == 0).all() and q[:, 0::2].isfinite().all() and (q[:, 0::2] != 0).flatten(1).any(1).all()
    k = x["kc"].flatten(0, 1)[x["slots"][x["slots"] >= 0]][:, 1]
    assert ((k & 0x7f if cache == "e4m3" else k) == 0).all()


# A slot named twice: every value is one of the tokens', other slots are not touched.
@pytest.mark.gpu
@pytest.mark.parametrize("t,cache", [("bf16", "bf16"), ("f32", "f32"), ("f16", "e4m3")])
def test_append_of_a_slot_named_twice(dev, t, cache):
    x = _append_inputs(dev, t, cache, 64, 32, 16, 128, 16, 64)
    k0, v0 = x["kc"].clone(), x["vc"].clone()
    args = (x["q"], x["k"], x["v"], x["pos"], x["cs"])
    kw = dict(q_weight=x["qw"], k_weight=x["kw"], k_scale=x["ks"], v_scale=x["vs"])
    apart = torch.arange(64, device=dev)
    kc, vc = torch.zeros_like(k0), torch.zeros_like(v0)
    want_q = binding.norm_rope_kv_append(*args, apart, kc, vc, **kw)
    slots = torch.full((64,), 19, dtype=torch.int64, device=dev)
    q = binding.norm_rope_kv_append(*args, slots, x["kc"], x["vc"], **kw)
    assert binding.device_status() == 0 and torch.equal(q, want_q)
    for got, each, before in ((x["kc"], kc, k0), (x["vc"], vc, v0)):
        got, each, before = (c.flatten(0, 1) for c in (got, each, before))
        assert (got[19] == each[:64]).any(0).all()
        rest = torch.arange(got.shape[0], device=dev) != 19
        assert torch.equal(got[rest], before[rest])


# --- what may follow a call: kernels that start early and write over what the call reads

# rows beside chunks (the row kernel is through long before the chunks are), chunks alone, single rows alone
FOLLOWED = [("bf16", "bf16", [1, 1500, 1, 1400], [300, 1500, 90, 2500]), ("bf16", "e4m3", [1, 1500, 1, 1400], [300, 1500, 90, 2500]),
            ("f16", "f16", [2900], [4000]), ("bf16", "bf16", [1] * 100, [3000] * 100)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,cache,q,kv", FOLLOWED, ids=["mixed", "mixed-e4m3", "chunk", "rows"])
def test_queries_and_tables_written_right_behind_a_call(dev, t, cache, q, kv):
    p = Problem(dev, t, cache, 32, 8, 128, 64, 700, 3, q, kv)
    want, wl = p.run()
    T = p.q.shape[0]
    a = _append_inputs(dev, t, cache, T, 32, 8, 128, 64, 64)
    q0, cu, lens, tab0 = p.q.clone(), _i32(_cum(q), dev), _i32(kv, dev), _i32(p.tables, dev)
    moved = _i32((np.arange(p.N) + 1) % p.N, dev)
    for first in ("queries", "tables") * 3:
        x, tab = q0.clone(), tab0.clone()
        torch.cuda.synchronize()
        out, lse = binding.window_attention(x, cu, lens, tab, p.kc, p.vc, p.scale, p.W, sinks=p.S, k_scale=p.ks,
                                            v_scale=p.vs)

        def append():    # the next layer's queries go where this call's are (its keys elsewhere)
            binding.norm_rope_kv_append(a["q"], a["k"], a["v"], a["pos"], a["cs"], a["slots"], a["kc"], a["vc"],
                                        k_scale=a["ks"], v_scale=a["vs"], q_out=x)

        def remap():
            binding.remap_pages(tab, moved)

        for f in (append, remap) if first == "queries" else (remap, append):
            f()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        # (both were written over while or after the call read them)
        assert (x != q0).flatten(1).any(1).all() and (tab != tab0)[tab0 >= 0].all()
    assert binding.device_status() == 0


# --- forks of sequences whose pages behind a window have been let go (CPU)

def test_a_fork_below_the_length_of_the_trim_is_refused(lib):
    pool = binding.PagePool(60, 4)
    parent = pool.trim(pool.alloc(25), 100, 40, 0)         # the next row sees keys 61 .. 100
    assert parent[:15] == [-1] * 15 and min(parent[15:]) >= 0
    held = [pool.refcount(i) for i in range(60)]
    with pytest.raises(binding.PagedKVError):              # its next row would see keys 31 .. 70
        pool.fork(parent, 70, 40)
    assert [pool.refcount(i) for i in range(60)] == held and pool.free_count() == 50
    assert pool.fork(parent, 70)[0][:15] == [-1] * 15      # (without a window nothing is known of what is seen)
    child, copy = pool.fork(parent, 100, 40)
    assert child == parent and copy is None
    child, copy = pool.fork(parent, 99, 38)                # 62 .. 99
    assert child[:24] == parent[:24] and copy == (parent[24], child[24], 3)
    with pytest.raises(binding.PagedKVError):              # the sinks' page is gone
        pool.fork(parent, 100, 40, sinks=1)


@pytest.mark.parametrize("P", [1, 4, 7])
@pytest.mark.parametrize("W,S", [(1, 0), (5, 0), (5, 3), (16, 4), (100, 0), (2 ** 40, 0), (3, 2 ** 40)])
def test_a_fork_takes_what_its_rows_need(lib, P, W, S):
    L = 41
    for kv in range(L + 1):
        for gone in range(-(-L // P)):
            pool = binding.PagePool(64, P)
            pages = pool.alloc(-(-L // P))
            pool.release([pages[gone]])
            pages[gone] = -1
            first, end = gone * P, gone * P + P
            used, partly = first < kv, first < kv < end    # a partly filled page is copied, whatever is seen of it
            seen = first < S or end > kv - W + 1
            if used and (partly or seen):
                with pytest.raises(binding.PagedKVError):
                    pool.fork(pages, kv, W, S)
            else:
                child, _ = pool.fork(pages, kv, W, S)
                assert child[:kv // P] == list(pages[:kv // P])
    for w, s in ((0, 0), (-1, 0), (1, -1), (-2 ** 40, 0), (1, -2 ** 40)):
        with pytest.raises(binding.PagedKVError):
            binding.PagePool(4, P).fork([], 0, w, s)
