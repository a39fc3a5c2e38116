"""The latent-attention operators and the cases they are measured on.

A latent cache keeps, for each token, one vector shared by all heads: a latent
part of `ld` values and a rotary key part of `rd` = 64 values, in pages
[num_pages, page_size, ld + rd]. Four operators work on it:

  append   new tokens' latents and rotated keys go into their slots, the rotary
           parts of the tick's queries are rotated
  gather   the cached rows of every sequence, through its page table, into one
           packed tensor (what the up-projection of the expanded form reads)
  absorbed attention of packed query rows (ld + rd wide, the key projection
           already multiplied in) over the pages; scores over ld + rd values,
           output the weighted sum of the latent parts
  expanded causal attention of chunks over up-projected keys and values: a
           128-wide key part and a 128-wide value per head, and the 64-wide
           rotary key that all heads share

Where `own` is false `run` computes them from elementary torch operations in
32 bits; where it is true it calls the library.
"""
import math
import random

import torch

own = False

RD = 64      # rotary part of a key
NOPE = 128   # expanded form: key values of a head beside the rotary part
DV = 128     # expanded form: values of a head
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode tick's new tokens, all heads on one GPU: a launch and little else
        dict(name="append_decode", op="append", dtype="bf16", T=128, H=128, P=64, ld=512, lens=1),
        # a prefill tick's tokens, the heads of one of eight shards
        dict(name="append_chunk", op="append", dtype="f16", T=8192, H=16, P=256, ld=512, lens=2),
        # short cached prefixes on small pages, before their expansion
        dict(name="gather_short", op="gather", dtype="bf16", B=6, kv_lo=1, kv_hi=700, P=16, ld=512, lens=3),
        # long cached prefixes: reading and writing at full rate
        dict(name="gather_long", op="gather", dtype="bf16", B=12, kv_lo=4096, kv_hi=16384, P=64, ld=512, lens=4),
        # one user, a short context: latency
        dict(name="absorbed_single", op="absorbed", dtype="bf16", B=1, H=16, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=1000,
             P=64, ld=512, lens=5),
        # a full decode batch with all heads
        dict(name="absorbed_decode", op="absorbed", dtype="bf16", B=128, H=128, q_lo=1, q_hi=1, kv_lo=512,
             kv_hi=8192, P=64, ld=512, lens=6),
        # a full decode batch with the heads of one of eight shards, large pages
        dict(name="absorbed_shard", op="absorbed", dtype="f16", B=96, H=16, q_lo=1, q_hi=1, kv_lo=64, kv_hi=16384,
             P=256, ld=512, lens=7),
        # few sequences with very long contexts: the keys are split over the whole GPU
        dict(name="absorbed_long", op="absorbed", dtype="bf16", B=2, H=128, q_lo=1, q_hi=1, kv_lo=65536,
             kv_hi=131072, P=64, ld=512, lens=8),
        # drafted tokens checked together, an odd head count, pages that end inside a tile, a narrow latent
        dict(name="absorbed_drafts", op="absorbed", dtype="bf16", B=40, H=20, q_lo=1, q_hi=5, kv_lo=5, kv_hi=3000,
             P=24, ld=256, lens=9),
        # a few short prompts
        dict(name="expanded_short", op="expanded", dtype="f16", B=3, H=16, q_lo=20, q_hi=300, pre_lo=0, pre_hi=0,
             lens=10),
        # chunks of several prompts, each after a cached prefix
        dict(name="expanded_prefix", op="expanded", dtype="bf16", B=8, H=32, q_lo=100, q_hi=700, pre_lo=0,
             pre_hi=4000, lens=11),
        # one long prompt, all heads
        dict(name="expanded_full", op="expanded", dtype="bf16", B=1, H=128, q_lo=4096, q_hi=4096, pre_lo=0,
             pre_hi=0, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, evenly spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "gather", "absorbed", "absorbed", "expanded"])
    dtype = rng.choice(["bf16", "f16"])
    lens = rng.randrange(1 << 30)
    P = rng.choice([8, 16, 20, 24, 32, 48, 64, 100, 128, 256])
    ld = rng.choice([256, 512, 512])
    if op == "append":
        return dict(op=op, dtype=dtype, T=_log(rng, 1, 8192), H=rng.randint(1, 16), P=P, ld=ld, lens=lens)
    if op == "gather":
        hi = _log(rng, 10, 16384)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, max(1, min(64, 120000 // hi))), kv_lo=rng.randint(0, hi // 2),
                    kv_hi=hi, P=P, ld=ld, lens=lens)
    if op == "absorbed":
        B, hi = _log(rng, 1, 128), _log(rng, 8, 8192)
        q_hi = rng.choice([1, 1, 1, 2, 4, 7])
        return dict(op=op, dtype=dtype, B=B, H=rng.choice([1, 4, 8, 16, 20, 32, 40, 64, 96, 128]) // (2 if q_hi > 2 else 1) or 1,
                    q_lo=1, q_hi=q_hi, kv_lo=min(hi, max(q_hi, hi // 8)), kv_hi=max(hi, q_hi), P=P, ld=ld, lens=lens)
    q_hi = _log(rng, 1, 2048)
    pre = rng.choice([0, 0, rng.randint(1, 2048)])
    room = 128 * 4096 * 4096 // (4 * q_hi * (q_hi + pre))
    H = rng.choice([1, 3, 8, 16, 32, 64])
    B = _log(rng, 1, max(1, min(16, room // H, 16000 // (q_hi + pre))))
    return dict(op=op, dtype=dtype, B=B, H=H, q_lo=max(1, q_hi // 4), q_hi=q_hi, pre_lo=0, pre_hi=pre, lens=lens)


def _lengths(case):
    """Query and key lengths of the sequences, from the case alone."""
    r = random.Random(case["lens"])
    n = range(case["B"])
    if case["op"] == "gather":
        kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in n]
        if not any(kv):
            kv[0] = case["kv_hi"]
        return [0] * case["B"], kv
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in n]
    if case["op"] == "expanded":
        return q, [a + r.randint(case["pre_lo"], case["pre_hi"]) for a in q]
    return q, [max(a, r.randint(case["kv_lo"], case["kv_hi"])) for a in q]


def _cumulative(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _rope_table(positions, dim):
    """cos and sin of p * base^(-2 i / dim), in 64 bits until the last step: [positions, dim / 2, 2]."""
    f = 10000.0 ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(t)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    s = {"op": case["op"]}
    if case["op"] == "append":
        T, H, P, ld = case["T"], case["H"], case["P"], case["ld"]
        pages = -(-T // P) * 2 + 1
        perm = torch.randperm(pages * P, generator=g, device=dev)
        s["slots"] = perm[:T].contiguous()                                  # int64
        s["positions"] = torch.randint(0, 16384, (T,), generator=g, device=dev, dtype=torch.int32)
        s["table"] = _rope_table(16384, RD)
        s["cache"] = normal(pages, P, ld + RD)
        s["c_kv"] = normal(T, ld)                                           # the normalised latent
        s["k_rope"] = normal(T, ld + RD)[:, ld:]                            # the tail of the down-projection
        s["q_rope"] = normal(T, H, NOPE + RD)[..., NOPE:]                   # the tail of each query head
        s["q_out"] = normal(T, H, ld + RD)[..., ld:]                        # where the absorbed query keeps it
        return s
    q_lens, kv_lens = _lengths(case)
    B, cu_q, cu_k = case["B"], _cumulative(q_lens), _cumulative(kv_lens)
    s.update(q_max=max(q_lens), kv_max=max(kv_lens), total_q=cu_q[-1], total_k=cu_k[-1], cu_q=ints(cu_q),
             cu_k=ints(cu_k), kv_lens=ints(kv_lens))
    if case["op"] == "expanded":
        H = case["H"]
        up = normal(s["total_k"], H, NOPE + DV)                             # the up-projection's output
        s.update(q=normal(s["total_q"], H, NOPE + RD), k_nope=up[..., :NOPE], v=up[..., NOPE:],
                 k_rope=normal(s["total_k"], 512 + RD)[:, 512:],            # the tail of the gathered rows
                 scale=1.0 / math.sqrt(NOPE + RD))
        s.update(out=torch.empty(s["total_q"], H, DV, dtype=t, device=dev),
                 lse=torch.empty(s["total_q"], H, dtype=torch.float32, device=dev))
        if own:
            from paged_kv_attention_mapping_gb300 import binding
            s["workspace"] = binding.alloc_latent_prefill_workspace(B, s["q"])
        return s
    P, ld = case["P"], case["ld"]
    need = [-(-n // P) for n in kv_lens]
    pages = sum(need) + sum(need) // 4 + 1
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    width = max(need)
    first = torch.tensor(_cumulative(need)[:-1], device=dev)[:, None] + torch.arange(width, device=dev)
    used = torch.arange(width, device=dev) < torch.tensor(need, device=dev)[:, None]
    s["page_tables"] = torch.where(used, perm[first.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    s["cache"] = normal(pages, P, ld + RD)
    if case["op"] == "gather":
        s["out"] = torch.empty(s["total_k"], ld + RD, dtype=t, device=dev)
        return s
    s.update(q=normal(s["total_q"], case["H"], ld + RD), scale=1.0 / math.sqrt(NOPE + RD), ld=ld)
    s.update(out=torch.empty(s["total_q"], case["H"], ld, dtype=t, device=dev),
             lse=torch.empty(s["total_q"], case["H"], dtype=torch.float32, device=dev))
    if own:
        from paged_kv_attention_mapping_gb300 import binding
        s["workspace"] = binding.alloc_latent_workspace(B, s["total_q"], case["H"], s["cache"])
    return s


# ---------------------------------------------------------------------------
# plain forms

def _rotate(x, cs):
    a, b = x.float().split(RD // 2, -1)
    c, s = cs[..., 0], cs[..., 1]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


def _append(s):
    cs = s["table"][s["positions"].long()]
    rows = s["cache"].view(-1, s["cache"].shape[-1])
    rows[s["slots"]] = torch.cat([s["c_kv"], _rotate(s["k_rope"], cs)], -1)
    s["q_out"].copy_(_rotate(s["q_rope"], cs[:, None]))
    return {"cache": s["cache"], "q": s["q_out"]}


def _cached_rows(s, b, pos):
    """Row numbers in the pool of positions `pos` of sequences `b`."""
    P = s["cache"].shape[1]
    return s["page_tables"][b, pos // P].long() * P + pos % P


def _gather(s):
    at = torch.arange(s["total_k"], device="cuda")
    b = torch.searchsorted(s["cu_k"][1:].long(), at, right=True)
    rows = _cached_rows(s, b, at - s["cu_k"].long()[b])
    return s["cache"].view(-1, s["cache"].shape[-1])[rows]


def _padded(cu, total, width):
    """[B, width] numbers of the packed rows of each sequence, and which of them exist."""
    n = torch.arange(width, device="cuda")
    return (cu[:-1, None] + n).clamp(max=total - 1).long(), n < (cu[1:] - cu[:-1])[:, None]


def _softmax(scores, s):
    """Causal softmax over padded scores [B, H, q, k]: weights, and the logarithm of each row's sum."""
    i, j = torch.arange(s["q_max"], device="cuda"), torch.arange(s["kv_max"], device="cuda")
    ahead = (s["kv_lens"] - (s["cu_q"][1:] - s["cu_q"][:-1]))[:, None, None] + i[:, None]   # a row's own position
    scores.masked_fill_((j > ahead)[:, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    w = scores.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    return w, total, (top + total.log()).squeeze(-1)


def _absorbed(s):
    rows_q, there_q = _padded(s["cu_q"], s["total_q"], s["q_max"])
    B, H, ld = rows_q.shape[0], s["q"].shape[1], s["ld"]
    j = torch.arange(s["kv_max"], device="cuda")
    there = j < s["kv_lens"][:, None]
    at = torch.where(there, _cached_rows(s, torch.arange(B, device="cuda")[:, None], j[None]), 0)
    kv = s["cache"].view(-1, s["cache"].shape[-1])[at].float()                              # [B, k, ld + rd]
    kv.masked_fill_(~there[..., None], 0.0)
    q = s["q"][rows_q].float().flatten(1, 2)                                                # [B, q H, ld + rd]
    scores = torch.matmul(q, kv.transpose(1, 2)).mul_(s["scale"]).view(B, s["q_max"], H, -1).transpose(1, 2)
    w, total, lse = _softmax(scores, s)
    o = torch.matmul(w.transpose(1, 2).flatten(1, 2), kv[..., :ld]).view(B, s["q_max"], H, ld)
    o = o / total.transpose(1, 2)
    return {"out": o[there_q].to(s["q"].dtype), "lse": lse.transpose(1, 2)[there_q]}


def _expanded(s):
    rows_q, there_q = _padded(s["cu_q"], s["total_q"], s["q_max"])
    rows_k, there_k = _padded(s["cu_k"], s["total_k"], s["kv_max"])
    q = s["q"][rows_q].transpose(1, 2).float()                                              # [B, H, q, 192]
    k = s["k_nope"][rows_k].permute(0, 2, 3, 1).float()                                     # [B, H, 128, k]
    kr = s["k_rope"][rows_k].transpose(1, 2)[:, None].float()                               # [B, 1, 64, k]
    scores = torch.matmul(q[..., :NOPE], k).add_(torch.matmul(q[..., NOPE:], kr)).mul_(s["scale"])
    w, total, lse = _softmax(scores, s)
    v = s["v"][rows_k].float().masked_fill_(~there_k[..., None, None], 0.0).transpose(1, 2)
    o = (torch.matmul(w, v) / total).transpose(1, 2)
    return {"out": o[there_q].to(s["q"].dtype), "lse": lse.transpose(1, 2)[there_q]}


# ---------------------------------------------------------------------------

def _library(s):
    from paged_kv_attention_mapping_gb300 import binding
    if s["op"] == "append":
        binding.latent_append(s["c_kv"], s["k_rope"], s["positions"], s["table"], s["slots"], s["cache"],
                              q_rope=s["q_rope"], q_out=s["q_out"])
        return {"cache": s["cache"], "q": s["q_out"]}
    if s["op"] == "gather":
        return binding.latent_gather(s["cache"], s["page_tables"], s["cu_k"], s["total_k"], out=s["out"])
    if s["op"] == "absorbed":
        out, lse = binding.latent_attention(s["q"], s["cu_q"], s["kv_lens"], s["page_tables"], s["cache"],
                                            s["scale"], s["kv_max"], out=s["out"], lse=s["lse"],
                                            workspace=s["workspace"])
    else:
        out, lse = binding.latent_prefill(s["q"], s["cu_q"], s["k_nope"], s["v"], s["k_rope"], s["cu_k"], s["scale"],
                                          out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _library(state)
    return {"append": _append, "gather": _gather, "absorbed": _absorbed, "expanded": _expanded}[state["op"]](state)


def work(case):
    if case["op"] == "append":
        T, H, ld = case["T"], case["H"], case["ld"]
        # latent and key read and written, the queries' rotary parts read and written, slot, position, angles
        return {"bytes": T * (4 * (ld + RD) + 4 * H * RD + 12 + 4 * RD), "flops": T * (H + 1) * 3 * RD}
    q_lens, kv_lens = _lengths(case)
    if case["op"] == "gather":
        return {"bytes": sum(kv_lens) * 4 * (case["ld"] + RD) + sum(4 * -(-n // case["P"]) for n in kv_lens), "flops": 0}
    H, rows = case["H"], sum(q_lens)
    pairs = sum(q * (L - q) + q * (q + 1) // 2 for q, L in zip(q_lens, kv_lens))
    if case["op"] == "absorbed":
        ld = case["ld"]
        return {"bytes": 2 * sum(kv_lens) * (ld + RD) + rows * H * (2 * (2 * ld + RD) + 4),
                "flops": 2 * pairs * H * (2 * ld + RD)}
    return {"bytes": 2 * sum(kv_lens) * (H * (NOPE + DV) + RD) + rows * H * (2 * (NOPE + RD + DV) + 4),
            "flops": 2 * pairs * H * (NOPE + RD + DV)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence

def _attend(q, k, v, scale):
    """q [H, n, d], k [H or 1, L, d], v [H or 1, L, e]: row i sees keys 0 .. L - n + i."""
    n, L = q.shape[1], k.shape[1]
    x = scale * (q @ k.transpose(1, 2))
    hidden = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)
    x = x.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(x, -1)
    return (torch.exp(x - lse[..., None]) @ v).transpose(0, 1), lse.transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        p = s["positions"].double()[:, None]
        a = p * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                          -torch.arange(0, RD, 2, dtype=torch.float64, device="cuda") / RD)
        turn = torch.polar(torch.ones_like(a), a)

        def rotated(x, by):
            z = torch.complex(x[..., :RD // 2].double(), x[..., RD // 2:].double()) * by
            return torch.cat([z.real, z.imag], -1)

        cache = s["cache"].double().flatten(0, 1)
        cache.index_copy_(0, s["slots"], torch.cat([s["c_kv"].double(), rotated(s["k_rope"], turn)], 1))
        return {"cache": cache.view(s["cache"].shape), "q": rotated(s["q_rope"], turn[:, None])}
    q_lens, kv_lens = _lengths(case)
    cu_q, cu_k = _cumulative(q_lens), _cumulative(kv_lens)
    outs, lses = [], []
    for b in range(case["B"]):
        L = kv_lens[b]
        if case["op"] != "expanded":
            table = s["page_tables"][b, :-(-L // case["P"])].long()
            rows = s["cache"][table].flatten(0, 1)[:L].double()
        if case["op"] == "gather":
            outs.append(rows)
            continue
        q = s["q"][cu_q[b]:cu_q[b + 1]].double().transpose(0, 1)
        if case["op"] == "absorbed":
            o, l = _attend(q, rows[None], rows[None, :, :case["ld"]], s["scale"])
        else:
            at = slice(cu_k[b], cu_k[b + 1])
            kr = s["k_rope"][at, None].double().expand(-1, case["H"], -1)
            k = torch.cat([s["k_nope"][at].double(), kr], -1).transpose(0, 1)
            o, l = _attend(q, k, s["v"][at].double().transpose(0, 1), s["scale"])
        outs.append(o)
        lses.append(l)
    return torch.cat(outs) if case["op"] == "gather" else {"out": torch.cat(outs), "lse": torch.cat(lses)}
