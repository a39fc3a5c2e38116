"""The operators of a serving tick's windowed layers, and the cases they are measured on.

Keys and values lie in pages, caches [num_pages, page_size, kv_heads, head_dim].

  append   the tick's new tokens: queries and keys are normed per head (root mean
           square, a weight per channel), the first `rot` values of each head are
           rotated by its position (pairs half a rotation width apart, or
           neighbours), keys and values go into their slots (in the cache's type, or
           as e4m3 codes of x / scale), queries into a tensor of their own
  window   attention of packed rows over the pages, where a row at position p sees
           the keys p - window + 1 .. p and the first `sinks` keys
  copy     pages of several caches copied to other pages (whole, or their first
           tokens), and page tables rewritten for pages that have moved

Where `own` is false `run` computes them from elementary torch operations in 32
bits; where it is true it calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
MAX_POS = 16384


def listed():
    return [
        # one decode tick's new tokens: a launch and little else
        dict(name="append_decode", op="append", dtype="bf16", cache="bf16", T=64, Hq=32, Hkv=8, D=128, P=256, rot=128,
             pairs="half", table="plain"),
        # a tick of decode rows and two chunks
        dict(name="append_tick", op="append", dtype="bf16", cache="bf16", T=4192, Hq=32, Hkv=8, D=128, P=256, rot=128,
             pairs="half", table="plain"),
        # a long prompt into an e4m3 cache, half of each head rotated in neighbouring pairs, angles of a stretched context
        dict(name="append_codes", op="append", dtype="f16", cache="e4m3", T=8191, Hq=32, Hkv=4, D=128, P=16, rot=64,
             pairs="neighbours", table="ramp"),
        # a short prompt of a small model in fp32
        dict(name="append_f32", op="append", dtype="f32", cache="f32", T=255, Hq=8, Hkv=2, D=64, P=16, rot=32,
             pairs="half", table="linear"),
        # a decode batch with a narrow window: latency
        dict(name="window_decode_narrow", op="window", dtype="f16", cache="f16", B=64, q_lo=1, q_hi=1, kv_lo=100, kv_hi=2048, chunks=0,
             Hq=32, Hkv=4, D=64, P=16, window=128, sinks=4, lens=1),
        # a full decode batch with a wide window: reading keys and values
        dict(name="window_decode_wide", op="window", dtype="bf16", cache="bf16", B=128, q_lo=1, q_hi=1, kv_lo=512, kv_hi=8192, chunks=0,
             Hq=32, Hkv=8, D=128, P=256, window=4096, sinks=4, lens=2),
        # a few long contexts over an e4m3 cache, drafted tokens checked together
        dict(name="window_drafts_codes", op="window", dtype="bf16", cache="e4m3", B=6, q_lo=2, q_hi=5, kv_lo=5000, kv_hi=30000, chunks=0,
             Hq=40, Hkv=8, D=128, P=64, window=8000, sinks=16, lens=3),
        # a tick of decode rows and two chunks, one of them after a cached prefix
        dict(name="window_tick", op="window", dtype="bf16", cache="bf16", B=96, q_lo=1, q_hi=1, kv_lo=256, kv_hi=4096, chunks=2,
             new_lo=2048, new_hi=2048, pre_lo=0, pre_hi=2000, Hq=32, Hkv=8, D=128, P=256, window=1024, sinks=4, lens=4),
        # prompts of ragged lengths, a narrow window, an odd group of query heads
        dict(name="window_prompts", op="window", dtype="bf16", cache="bf16", B=0, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, chunks=7,
             new_lo=300, new_hi=2500, pre_lo=0, pre_hi=0, Hq=28, Hkv=4, D=128, P=16, window=512, sinks=0, lens=5),
        # one long prompt
        dict(name="window_long", op="window", dtype="f16", cache="f16", B=0, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, chunks=1,
             new_lo=16384, new_hi=16384, pre_lo=0, pre_hi=0, Hq=32, Hkv=8, D=128, P=256, window=2048, sinks=64, lens=6),
        # sequences forked: the partly filled last page of each, in every layer
        dict(name="copy_forks", op="copy", cache="f16", layers=22, N=96, P=16, Hkv=4, D=64, n=24, part=True, tables=0),
        # a pool compacted: whole pages moved in every layer and the tables rewritten
        dict(name="copy_compact", op="copy", cache="bf16", layers=8, N=320, P=256, Hkv=8, D=128, n=112, part=False, tables=128),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, evenly spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "append", "window", "window", "window", "copy"])
    lens = rng.randrange(1 << 30)
    D = rng.choice([64, 64, 128, 128, 128, 256])
    P = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return dict(op=op, dtype=dtype, cache=rng.choice([dtype, dtype, "e4m3"]), T=_log(rng, 1, 8192 if D < 256 else 3000),
                    Hq=Hq, Hkv=Hkv, D=D, P=P, rot=rng.choice([D, D, D // 2, 16, 48]), pairs=rng.choice(["half", "neighbours"]),
                    table=rng.choice(["plain", "linear", "ramp"]))
    if op == "copy":
        P = rng.choice([8, 16, 24, 64, 100, 256])
        return dict(op=op, cache=rng.choice(["bf16", "f32", "e4m3"]), layers=rng.randint(1, 24), N=2 * (256 // P + 20) + 3,
                    P=P, Hkv=rng.choice([1, 2, 4]), D=rng.choice([64, 128]), n=rng.randint(1, 256 // P + 20),
                    part=rng.random() < 0.5, tables=rng.choice([0, 3, 200]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    cache = dtype if dtype == "f32" else rng.choice([dtype, dtype, "e4m3"])
    c = dict(op=op, dtype=dtype, cache=cache, B=0, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, chunks=0, new_lo=1, new_hi=1, pre_lo=0, pre_hi=0, Hq=Hq, Hkv=Hkv, D=D,
             P=P, window=_log(rng, 1, 5000), sinks=rng.choice([0, 0, 1, 4, 64, 130]), lens=lens)
    kind = rng.choice(["decode", "decode", "tick", "prompts"])
    if kind != "prompts":
        q_hi = rng.choice([1, 1, 1, 3, 8])
        kv_hi = max(q_hi, _log(rng, 1, 8192))
        c.update(B=_log(rng, 1, 96), q_lo=1, q_hi=q_hi, kv_lo=max(q_hi, kv_hi // 8), kv_hi=kv_hi)
    if kind != "decode":
        q_hi = _log(rng, 9, 2048 if dtype != "f32" else 300)
        pre = rng.choice([0, rng.randint(1, 3000)])
        c.update(chunks=rng.randint(1, 4), new_lo=max(1, q_hi // 3), new_hi=q_hi, pre_lo=pre // 3, pre_hi=pre)
    return c


def _lengths(case):
    """Query and key lengths of the sequences, from the case alone."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["chunks"])]
    return q + new, kv + [n + r.randint(case["pre_lo"], case["pre_hi"]) for n in new]


def _cumulative(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _angles(rot, kind):
    """Angle of each pair at position 1, in 64 bits, and the factor on cos and sin: the usual ones, all divided by 4, or
    a ramp over the pairs from the usual angle to a quarter of it, whose products get a factor."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / rot)
    if kind == "plain":
        return f, 1.0
    if kind == "linear":
        return f / 4.0, 1.0
    share = ((i - rot / 16) / (rot / 4)).clamp(0.0, 1.0)
    return f * (1 - share) + f / 4.0 * share, 0.1 * math.log(4.0) + 1.0


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    ct = TYPES[case["cache"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    def filled(*shape):
        return normal(*shape).to(torch.bfloat16 if case["cache"] == "e4m3" else ct).to(ct)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    s = {"op": case["op"], "case": case}
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    if case["op"] == "copy":
        N, n = case["N"], case["n"]
        perm = torch.randperm(N, generator=g, device=dev).to(torch.int32)
        pool = filled(2 * case["layers"], N, P, Hkv, D)                     # keys and values of every layer
        s.update(pool=pool, caches=list(pool.unbind()), src=perm[:n].contiguous(), dst=perm[n:2 * n].contiguous(),
                 tokens=None, tables=None)
        if case["part"]:
            s["tokens"] = torch.randint(1, P + 1, (n,), generator=g, device=dev, dtype=torch.int32)
        if case["tables"]:
            s["map"] = torch.arange(N, device=dev, dtype=torch.int32).index_copy(0, s["src"].long(), s["dst"])
            s["tables"] = torch.randint(-1, N, (case["tables"], 33), generator=g, device=dev, dtype=torch.int32)
        return s
    t, Hq = TYPES[case["dtype"]], case["Hq"]
    e4m3 = case["cache"] == "e4m3"
    # scales of an e4m3 cache: the largest code stands for about 4 standard deviations
    s.update(k_scale=None, v_scale=None)
    if e4m3:
        s.update(k_scale=torch.rand(Hkv, generator=g, device=dev) * 0.004 + 0.008,
                 v_scale=torch.rand(Hkv, generator=g, device=dev) * 0.004 + 0.008)
    if case["op"] == "append":
        T = case["T"]
        pages = -(-T // P) + 2
        s["slots"] = torch.randperm(pages * P, generator=g, device=dev)[:T].contiguous()
        s["positions"] = torch.randint(0, MAX_POS, (T,), generator=g, device=dev, dtype=torch.int32)
        f, factor = _angles(case["rot"], case["table"])
        a = torch.arange(MAX_POS, dtype=torch.float64, device=dev)[:, None] * f
        s["table"] = (torch.stack([a.cos(), a.sin()], -1) * factor).float()
        s["k_cache"], s["v_cache"] = filled(pages, P, Hkv, D), filled(pages, P, Hkv, D)
        qkv = normal(T, Hq + 2 * Hkv, D, std=2.0).to(t)                     # the projection's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_weight"], s["k_weight"] = (1 + normal(D, std=0.1)).to(t), (1 + normal(D, std=0.1)).to(t)
        s.update(eps=1e-6, q_out=torch.empty(T, Hq, D, dtype=t, device=dev))
        return s
    q_lens, kv_lens = _lengths(case)
    need = [-(-n // P) for n in kv_lens]
    pages = sum(need) + sum(need) // 4 + 1
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    width = max(need)
    first = torch.tensor(_cumulative(need)[:-1], device=dev)[:, None] + torch.arange(width, device=dev)
    used = torch.arange(width, device=dev) < torch.tensor(need, device=dev)[:, None]
    s["page_tables"] = torch.where(used, perm[first.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    cu = _cumulative(q_lens)
    s.update(cu=ints(cu), kv_lens=ints(kv_lens), q=normal(cu[-1], Hq, D).to(t))
    if e4m3:
        s["k_cache"], s["v_cache"] = ((normal(pages, P, Hkv, D) * 100).to(ct) for _ in range(2))
    else:
        s["k_cache"], s["v_cache"] = filled(pages, P, Hkv, D), filled(pages, P, Hkv, D)
    s.update(scale=1.0 / math.sqrt(D), out=torch.empty(cu[-1], Hq, D, dtype=t, device=dev),
             lse=torch.empty(cu[-1], Hq, dtype=torch.float32, device=dev))
    # the plain form's rows in blocks of one sequence: the first row of each, its rows, sequence and position
    s["blocks"] = [(rows, ints([(cu[b] + i, min(rows, q_lens[b] - i), b, kv_lens[b] - q_lens[b] + i)
                                for b in some for i in range(0, q_lens[b], rows)]))
                   for rows, some in ((case["q_hi"], range(case["B"])), (256, range(case["B"], len(q_lens)))) if some]
    return s


# ---------------------------------------------------------------------------
# plain forms

def _turn(x, cs, half):
    """The pairs of the first values of each head rotated; x fp32 [T, H, D], cs [T, 1, rot / 2, 2]."""
    rot = 2 * cs.shape[-2]
    y = x[..., :rot]
    a, b = (y[..., :rot // 2], y[..., rot // 2:]) if half else (y[..., 0::2], y[..., 1::2])
    c, s = cs[..., 0], cs[..., 1]
    y = torch.cat([a * c - b * s, b * c + a * s], -1) if half else torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _normed(x, w, eps):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _store(x, cache, slots, scale):
    """Values into their slots, as the cache holds them."""
    if scale is None:
        cache.view(-1, *cache.shape[2:])[slots] = x.to(cache.dtype)
    else:
        codes = (x.float() / scale[:, None]).clamp(-448.0, 448.0).to(cache.dtype)
        cache.view(-1, *cache.shape[2:]).view(torch.uint8)[slots] = codes.view(torch.uint8)


def _append(s):
    half = s["case"]["pairs"] == "half"
    cs = s["table"][s["positions"].long()][:, None]
    s["q_out"].copy_(_turn(_normed(s["q"], s["q_weight"], s["eps"]), cs, half))
    k = _turn(_normed(s["k"], s["k_weight"], s["eps"]), cs, half)
    _store(k, s["k_cache"], s["slots"], s["k_scale"])
    _store(s["v"], s["v_cache"], s["slots"], s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": s["q_out"]}


def _blocks(s, rows, what):
    """Rows in blocks of `rows` of one sequence, all blocks at once."""
    c = s["case"]
    W, S, P, Hkv = c["window"], c["sinks"], c["P"], c["Hkv"]
    first, n, b, p0 = what.long().unbind(1)
    i = torch.arange(rows, device="cuda")
    there = i < n[:, None]                                                                   # [blocks, rows]
    at = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    last = p0 + n - 1
    w = min(W + rows - 1, s["page_tables"].shape[1] * P)
    begin = (p0 - W + 1).clamp(min=0)
    sink = torch.arange(min(S, s["page_tables"].shape[1] * P), device="cuda").expand(len(b), -1)
    keys = torch.cat([torch.where(sink < begin[:, None], sink, 1 << 30), begin[:, None] + torch.arange(w, device="cuda")], 1)
    seen = keys <= last[:, None]
    k_at = torch.where(seen, keys, 0)
    page = s["page_tables"][b[:, None], k_at // P].long()
    slot = torch.where(seen, page, 0) * P + k_at % P
    q = s["q"][at].float()                                                                   # [blocks, rows, Hq, D]
    k, v = (x.view(-1, *x.shape[2:]).view(torch.uint8 if s["k_scale"] is not None else x.dtype)[slot].view(x.dtype).float()
            for x in (s["k_cache"], s["v_cache"]))                                           # [blocks, keys, Hkv, D]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    v = v.masked_fill(~seen[..., None, None], 0.0)
    B, _, Hq, D = q.shape
    q = q.view(B, rows, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, Hkv, Hq // Hkv, rows, -1)
    p = (p0[:, None] + i)[..., None]
    hidden = ~((keys[:, None] <= p) & ((keys[:, None] > p - W) | (keys[:, None] < S)))       # [blocks, rows, keys]
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v.transpose(1, 2)).view(B, Hkv, Hq // Hkv, rows, D) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)
    s["out"][at[there]] = o[there].to(s["out"].dtype)
    s["lse"][at[there]] = lse[there]


def _window(s):
    [_blocks(s, rows, what) for rows, what in s["blocks"]]
    return {"out": s["out"], "lse": s["lse"]}


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    pool = s["pool"].view(torch.uint8) if s["case"]["cache"] == "e4m3" else s["pool"]
    new = pool[:, src]
    if s["tokens"] is not None:
        keep = torch.arange(pool.shape[2], device="cuda") < s["tokens"][:, None]
        new = torch.where(keep[..., None, None], new, pool[:, dst])
    pool[:, dst] = new
    if s["tables"] is None:
        return {"pool": s["pool"]}
    t = s["tables"]
    t.copy_(torch.where(t >= 0, s["map"][t.long().clamp(min=0)], t))
    return {"pool": s["pool"], "tables": t}


# ---------------------------------------------------------------------------

def _library(s):
    from paged_kv_attention_mapping_gb300 import binding
    if s["op"] == "append":
        binding.norm_rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["k_cache"], s["v_cache"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                    interleaved=s["case"]["pairs"] != "half", k_scale=s["k_scale"], v_scale=s["v_scale"],
                                    q_out=s["q_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": s["q_out"]}
    if s["op"] == "window":
        out, lse = binding.window_attention(s["q"], s["cu"], s["kv_lens"], s["page_tables"], s["k_cache"], s["v_cache"],
                                            s["scale"], s["case"]["window"], sinks=s["case"]["sinks"], k_scale=s["k_scale"],
                                            v_scale=s["v_scale"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    binding.copy_pages(s["caches"], s["src"], s["dst"], tokens=s["tokens"])
    if s["tables"] is None:
        return {"pool": s["pool"]}
    return {"pool": s["pool"], "tables": binding.remap_pages(s["tables"], s["map"])}


def run(state):
    if own:
        return _library(state)
    return {"append": _append, "window": _window, "copy": _copy}[state["op"]](state)


def _seen(n, L, W, S):
    """Pairs of rows and keys, and the keys that some row sees, of n rows at the end of L keys."""
    def pairs(m):   # over rows at positions 0 .. m - 1
        full = min(m, W)
        inside = full * (full + 1) // 2 + (m - full) * W
        beyond = max(0, m - W)                  # rows with keys before their window: min(S, p - W + 1) of them are sinks
        ramp = min(beyond, S)
        return inside + ramp * (ramp + 1) // 2 + (beyond - ramp) * S
    begin = max(0, L - n - W + 1)
    return pairs(L) - pairs(L - n), L - begin + min(S, begin)


def work(case):
    e, Hkv, D = BYTES[case["cache"]], case["Hkv"], case["D"]
    if case["op"] == "copy":
        # half of a page on average where it is partly filled
        slots = case["n"] * case["P"] // (2 if case["part"] else 1)
        return {"bytes": 2 * slots * Hkv * D * e * 2 * case["layers"] + 8 * case["n"] + 8 * 33 * case["tables"], "flops": 0}
    t, Hq = BYTES[case["dtype"]], case["Hq"]
    if case["op"] == "append":
        T, rot = case["T"], case["rot"]
        rows = MAX_POS * (1 - (1 - 1 / MAX_POS) ** T)      # rows of the table that T positions meet
        return {"bytes": int(T * ((2 * Hq + 2 * Hkv) * D * t + 2 * Hkv * D * e + 12) + rows * rot * 4),
                "flops": T * (Hq + Hkv) * (4 * D + 3 * rot)}
    q_lens, kv_lens = _lengths(case)
    seen = [_seen(n, L, case["window"], case["sinks"]) for n, L in zip(q_lens, kv_lens)]
    return {"bytes": sum(k for _, k in seen) * 2 * Hkv * D * e + sum(q_lens) * Hq * (2 * D * t + 4),
            "flops": 4 * D * Hq * sum(p for p, _ in seen)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        at = torch.arange(case["P"], device="cuda")
        keep = at < (s["tokens"][:, None] if case["part"] else case["P"])
        keep = keep.expand(case["n"], -1)
        to, of = ((s[x].long()[:, None] * case["P"] + at)[keep] for x in ("dst", "src"))
        rows = s["pool"].float().flatten(1, 2)
        pool = rows.index_copy(1, to, rows[:, of]).view(s["pool"].shape)
        if s["tables"] is None:
            return {"pool": pool}
        moved = {int(a): int(b) for a, b in zip(s["src"].tolist(), s["dst"].tolist())}
        new = [[moved.get(x, x) for x in row] for row in s["tables"].tolist()]
        return {"pool": pool, "tables": torch.tensor(new, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        f, factor = _angles(case["rot"], case["table"])
        a = s["positions"].double()[:, None, None] * f
        by = torch.polar(torch.full_like(a, factor), a)
        r = case["rot"]

        def rotated(x, w):
            x = x.double()
            x = x / (x.square().sum(-1, keepdim=True) / case["D"] + s["eps"]).sqrt() * w.double()
            pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["pairs"] == "half" \
                else x[..., :r].unflatten(-1, (r // 2, 2))
            z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * by
            y = torch.stack([z.real, z.imag], -1)
            y = y.transpose(-1, -2) if case["pairs"] == "half" else y
            return torch.cat([y.flatten(-2), x[..., r:]], -1)

        def cached(cache, new, scale):
            rows = cache.float().double().flatten(0, 1)
            if scale is not None:
                new = (new / scale.double()[:, None]).clamp(-448, 448)
            return rows.index_copy(0, s["slots"], new).view(cache.shape)

        return {"k_cache": cached(s["k_cache"], rotated(s["k"], s["k_weight"]), s["k_scale"]),
                "v_cache": cached(s["v_cache"], s["v"].double(), s["v_scale"]), "q": rotated(s["q"], s["q_weight"])}
    q_lens, kv_lens = _lengths(case)
    W, S, P, Hkv = case["window"], case["sinks"], case["P"], case["Hkv"]
    outs, lses, row = [], [], 0
    for b, (n, L) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_tables"][b, :-(-L // P)].long()
        k, v = ((x[pages] if x.dtype != torch.float8_e4m3fn else x.view(torch.uint8)[pages].view(x.dtype)).float().double()
                for x in (s["k_cache"], s["v_cache"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        k, v = (x.flatten(0, 1)[:L].transpose(0, 1)[:, None] for x in (k, v))                # [Hkv, 1, L, D]
        for i in range(0, n, 512):
            m = min(512, n - i)
            p = torch.arange(L - n + i, L - n + i + m, device="cuda")[:, None]
            lo = max(0, L - n + i - W + 1)
            j = torch.cat([torch.arange(min(S, lo), device="cuda"), torch.arange(lo, L - n + i + m, device="cuda")])
            q = s["q"][row + i:row + i + m].double().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3)
            x = s["scale"] * (q @ k[:, :, j].transpose(-1, -2))                              # [Hkv, g, rows, keys]
            x = x.masked_fill((j > p) | ((j <= p - W) & (j >= S)), -math.inf)
            lse = torch.logsumexp(x, -1)
            o = torch.exp(x - lse[..., None]) @ v[:, :, j]
            outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
            lses.append(lse.permute(2, 0, 1).flatten(1, 2))
        row += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
