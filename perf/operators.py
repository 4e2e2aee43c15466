"""Measured cases of the serving operators that stand next to the delta rule.

Five kinds of call, each with its plain torch form (``own`` false) and the library call (``own``
true): the short causal convolution and the selective scan (prompts and single tokens), the
cache plan (block tables and slots from request lengths), the append that quantises into the
8-bit cache, and the attention that reads it.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # the convolution in front of a delta-rule layer: five prompts of 4001 tokens in all, rows of
        # the packed width 8192 (16 query, 16 key and 32 value heads of 128)
        dict(name="conv-prompt", op="conv", B=5, low=27, high=1573, C=8192, W=4, dtype="bf16", bias=False, silu=True,
             extra=0),
        # the same layer at a decode step of 64 requests, q | k | v of 32 heads each
        dict(name="conv-step", op="conv", B=64, low=1, high=1, C=12288, W=4, dtype="bf16", bias=True, silu=True,
             extra=64),
        # a prompt through a selective-scan layer as wide as 32 heads of 128
        dict(name="scan-prompt", op="scan", B=1, low=4000, high=4000, C=4096, N=16, G=1, dtype="bf16", gate=True),
        # few channels and a long prompt among short ones: parallel only along the tokens
        dict(name="scan-long", op="scan", B=3, low=1, high=16411, C=1000, N=16, G=1, dtype="f32", gate=False),
        # a decode step of 64 requests through the same layer
        dict(name="scan-step", op="scan", B=64, low=1, high=1, C=4096, N=16, G=1, dtype="bf16", gate=True),
        # a decode step's tables: one new token for each of 250 requests
        dict(name="plan-step", op="plan", B=250, width=256, page=64, old=16000, new_low=1, new_high=1, pad=6),
        # prompts that arrive next to running requests: 1 to 4000 new tokens each
        dict(name="plan-prompt", op="plan", B=33, width=128, page=32, old=100, new_low=1, new_high=4000, pad=0),
        # one token a request into caches of 8 key-value heads
        dict(name="append-step", op="append", B=64, low=1, high=1, old=4000, Hkv=8, D=128, page=64, dtype="bf16"),
        # prompts that begin inside a page
        dict(name="append-prompt", op="append", B=4, low=27, high=1973, old=100, Hkv=8, D=128, page=64, dtype="bf16"),
        # a decode step of 64 requests with 100 to 8000 cached tokens, four query heads to a key-value head
        dict(name="attend-step", op="attend", B=64, q_low=1, q_high=1, kv_low=100, kv_high=8000, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16"),
        # one request with a long cache
        dict(name="attend-long", op="attend", B=1, q_low=1, q_high=1, kv_low=131071, kv_high=131071, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16"),
        # chunks of prompts over what is cached of them already
        dict(name="attend-prompt", op="attend", B=3, q_low=500, q_high=2011, kv_low=2500, kv_high=4000, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw(rng):
    op = rng.choice(["conv", "scan", "plan", "append", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        step = rng.random() < 0.3
        high = 1 if step else _log_int(rng, 2, 4000)
        return dict(op=op, B=_log_int(rng, 1, 256), low=1 if step else rng.randint(0, high), high=high,
                    C=8 * _log_int(rng, 8, 1536), W=rng.choice([2, 3, 4, 4]), dtype=dtype, bias=rng.random() < 0.5,
                    silu=rng.random() < 0.8, extra=8 * rng.randint(0, 9))
    if op == "scan":
        step = rng.random() < 0.3
        high = 1 if step else _log_int(rng, 2, 16411)
        G = rng.choice([1, 1, 2, 4])
        return dict(op=op, B=_log_int(rng, 1, 64), low=1 if step else rng.randint(0, high), high=high,
                    C=8 * G * _log_int(rng, 8, 512 // G), N=rng.choice([16, 16, 32, 64, 128]), G=G, dtype=dtype,
                    gate=rng.random() < 0.6)
    if op == "plan":
        high = rng.choice([1, 1, 3, 50, 1000, 4000])
        return dict(op=op, B=_log_int(rng, 1, 1000), width=1024, page=rng.choice([16, 32, 64, 128]),
                    old=_log_int(rng, 1, 8000), new_low=rng.randint(0, high), new_high=high, pad=rng.randint(0, 40))
    if op == "append":
        high = rng.choice([1, 1, 4, _log_int(rng, 2, 4000)])
        return dict(op=op, B=_log_int(rng, 1, 256), low=rng.randint(0, high), high=high, old=_log_int(rng, 1, 2000),
                    Hkv=rng.choice([1, 2, 4, 8, 32]), D=rng.choice([32, 64, 128, 128]),
                    page=rng.choice([16, 32, 64, 128]), dtype=dtype)
    kind = rng.choice(["step", "step", "few", "prompt"])
    Hkv = rng.choice([1, 2, 4, 8])
    q_high = 1 if kind == "step" else rng.randint(2, 8) if kind == "few" else _log_int(rng, 9, 2000)
    kv_high = q_high + _log_int(rng, 1, 131072 if kind == "step" else 16411 if kind == "few" else 2000)
    return dict(op=op, B=_log_int(rng, 1, 128 if kind != "prompt" else 6), q_low=rng.randint(1, q_high), q_high=q_high,
                kv_low=rng.randint(q_high, kv_high), kv_high=kv_high, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 16]), Hkv=Hkv,
                D=rng.choice([32, 64, 128, 128]), page=rng.choice([16, 32, 64, 128]), dtype=dtype)


def _cost(c):
    """(bytes the plain form holds at its widest, its work): what a drawn case is bounded by."""
    w = work(c)
    if c["op"] == "conv":
        wide = sum(_lengths(c["B"], c["low"], c["high"])) * c["C"] * c["W"] * 4
    elif c["op"] == "scan":
        wide = sum(_lengths(c["B"], c["low"], c["high"])) * c["C"] * c["N"] * 4
    elif c["op"] == "append":
        wide = _pool(c) * c["Hkv"] * c["page"] * c["D"] * 4
    elif c["op"] == "attend":
        wide = c["B"] * c["kv_high"] * max(c["Hkv"] * c["D"], c["Hq"] * c["q_high"]) * 4
    else:
        wide = 16 * sum(_lengths(c["B"], c["new_low"], c["new_high"]))
    return wide, max(w["bytes"], w["flops"] / 50)


def draw(rng):
    tops = {}
    for c in listed():
        wide, cost = _cost(c)
        top = tops.setdefault(c["op"], [0, 0])
        top[0], top[1] = max(top[0], wide), max(top[1], cost)
    while True:
        c = _draw(rng)
        if c["op"] == "plan":
            fits = c["old"] + c["new_high"] <= c["width"] * c["page"]
        elif c["op"] == "append":
            fits = c["high"] > 0
        elif c["op"] in ("conv", "scan"):
            fits = c["high"] > 0
        else:
            fits = True
        wide, cost = _cost(c)
        if fits and wide <= tops[c["op"]][0] and cost <= tops[c["op"]][1]:
            return c


# ------------------------------------------------------------------------------------ inputs

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(count, low, high):
    """`count` lengths from `low` to `high`, spread evenly and in a mixed order; one alone has `high`."""
    if count == 1:
        return [high]
    spread = [high - (high - low) * i // (count - 1) for i in range(count)]
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, count) == 1)
    return [spread[(i * step) % count] for i in range(count)]


def _offsets(lengths, dev="cuda"):
    return torch.cumsum(torch.tensor([0] + list(lengths)), 0).to(torch.int32).to(dev)


def _ceil(a, b):
    return -(-a // b)


def _old_lengths(c):
    """Cached tokens of each request before the call, for the append: up to `old`, some at a page's end."""
    return _lengths(c["B"], 0, c["old"])


def _pool(c):
    """Pages of the pool of an append case."""
    total = sum(_ceil(a + b, c["page"]) for a, b in zip(_old_lengths(c), _lengths(c["B"], c["low"], c["high"])))
    return total + 3


def _tables(lengths, page, gen):
    """A block table for requests of these lengths over a shuffled pool, and the pool's size."""
    counts = [_ceil(n, page) for n in lengths]
    width = max(1, max(counts))
    pool = sum(counts) + 3
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    first = _offsets(counts)[:-1].long()
    col = torch.arange(width, device="cuda")
    have = torch.tensor(counts, device="cuda")
    at = (first[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < have[:, None], perm[at], torch.full_like(perm[at], -1)), pool


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = dict(c=c)
    if c["op"] in ("conv", "scan"):
        B, C, dt = c["B"], c["C"], DTYPES[c["dtype"]]
        lens = _lengths(B, c["low"], c["high"])
        n = sum(lens)
        s["dense"] = c["low"] == c["high"]        # equal lengths: a dense batch, no offsets
        s["step"] = c["low"] == c["high"] == 1
        s["longest"] = max(lens)
        s["cu"] = _offsets(lens)
        if c["op"] == "conv":
            # a slice of a wider projection row
            s["x"] = randn(n, C + c["extra"]).to(dt)[:, c["extra"]:]
            s["weight"] = randn(C, c["W"]) / math.sqrt(c["W"])
            s["bias"] = randn(C) * 0.1 if c["bias"] else None
            s["state"] = randn(B, c["W"] - 1, C).to(dt)
            return s
        N, G = c["N"], c["G"]
        s["x"] = randn(n, C).to(dt)
        # steps of 0.001 to 0.1 around the bias, as such layers start from
        s["dt"] = (randn(n, C) * 0.5).to(dt)
        step = torch.exp(rand(C) * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)).repeat(C, 1) + randn(C, N) * 0.1
        s["Bm"], s["Cm"] = randn(n, G, N).to(dt), randn(n, G, N).to(dt)
        s["D"] = randn(C)
        s["z"] = randn(n, C).to(dt) if c["gate"] else None
        s["state"] = randn(B, C, N) * 0.1
        return s
    page = c["page"]
    if c["op"] == "plan":
        B, width = c["B"], c["width"]
        new = _lengths(B, c["new_low"], c["new_high"])
        old = list(reversed(_lengths(B, 0, c["old"])))
        held = [_ceil(n, page) for n in old]
        pool = sum(held) + sum(_ceil(a + b, page) for a, b in zip(old, new)) + 5
        perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        first = _offsets(held)[:-1].long()
        col = torch.arange(width, device="cuda")
        at = (first[:, None] + col).clamp(max=pool - 1)
        have = torch.tensor(held, device="cuda")
        s["table"] = torch.where(col < have[:, None], perm[at], torch.full_like(perm[at], -1))
        s["seq_lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        left = pool - sum(held)
        s["free_pages"] = torch.cat([perm[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32, device="cuda")])
        s["free_count"] = torch.tensor([left], dtype=torch.int32, device="cuda")
        s["total"] = sum(new) + c["pad"]
        return s
    Hkv, D, dt = c["Hkv"], c["D"], DTYPES[c["dtype"]]
    if c["op"] == "append":
        old, new = _old_lengths(c), _lengths(c["B"], c["low"], c["high"])
        n = sum(new)
        table, pool = _tables([a + b for a, b in zip(old, new)], page, gen)
        cu = _offsets(new).long()
        tok = torch.arange(n, device="cuda")
        req = torch.searchsorted(cu, tok, right=True) - 1
        pos = torch.tensor(old, device="cuda")[req] + tok - cu[req]
        s["slots"] = table[req, pos // page].long() * page + pos % page
        s["k"], s["v"] = randn(n, Hkv, D).to(dt), (randn(n, Hkv, D) * 0.5).to(dt)
    else:
        q_lens = _lengths(c["B"], c["q_low"], c["q_high"])
        kv_lens = _lengths(c["B"], c["kv_low"], c["kv_high"])
        table, pool = _tables(kv_lens, page, gen)
        s["table"] = table
        s["cu"], s["kv_lens"] = _offsets(q_lens), torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        s["q"] = (randn(sum(q_lens), c["Hq"], D) * 1.5).to(dt)
    for name, spread in (("k", 0.03), ("v", 0.015)):
        s[name + "_cache"] = torch.round(randn(pool, Hkv, page, D) * 38).clamp_(-127, 127).to(torch.int8)
        s[name + "_scale"] = spread * (0.5 + rand(pool, Hkv))
    return s


# ------------------------------------------------------------------------------------ the passes


def run(s):
    op = s["c"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "plan": _own_plan, "append": _own_append, "attend": _own_attend}[op](s)
    return {"conv": _plain_conv, "scan": _plain_scan, "plan": _plain_plan, "append": _plain_append,
            "attend": _plain_attend}[op](s)


def _batched(s, t):
    """A packed tensor as the dense batch [B, T, ...] of an equal-length case."""
    return t.unflatten(0, (s["c"]["B"], -1)) if t is not None else None


def _own_conv(s):
    import gated_delta_rule_channelwise_gb300 as cg
    kw = dict(bias=s["bias"], silu=s["c"]["silu"])
    if s["step"]:
        o = cg.conv_decode(s["x"], s["weight"], s["state"], **kw)
    elif s["dense"]:
        o = cg.conv_prefill(_batched(s, s["x"]), s["weight"], s["state"], **kw).flatten(0, 1)
    else:
        o = cg.conv_prefill(s["x"], s["weight"], s["state"], cu_seqlens=s["cu"], **kw)
    return dict(o=o, state=s["state"])


def _own_scan(s):
    import gated_delta_rule_channelwise_gb300 as cg
    kw = dict(D=s["D"], dt_bias=s["dt_bias"])
    if s["step"]:
        o = cg.scan_decode(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], z=s["z"], **kw)
    elif s["dense"]:
        x, dt, Bm, Cm, z = (_batched(s, s[k]) for k in ("x", "dt", "Bm", "Cm", "z"))
        o = cg.scan_prefill(x, dt, s["A_log"], Bm, Cm, s["state"], z=z, **kw).flatten(0, 1)
    else:
        o = cg.scan_prefill(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], z=s["z"], cu_seqlens=s["cu"], **kw)
    return dict(o=o, state=s["state"])


def _own_plan(s):
    import gated_delta_rule_channelwise_gb300 as cg
    p = cg.cache_plan(s["table"], s["seq_lens"], s["new_lens"], s["free_pages"], s["free_count"], s["total"], s["c"]["page"])
    return dict(table=s["table"], kv_lens=p.kv_lens, cu=p.cu_seqlens, free_count=p.free_count, slots=p.slots,
                requests=p.requests, positions=p.positions)


def _own_append(s):
    import gated_delta_rule_channelwise_gb300 as cg
    cg.cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_attend(s):
    import gated_delta_rule_channelwise_gb300 as cg
    c = s["c"]
    return cg.cache_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_lens"],
                           s["cu"], max_q=c["q_high"], max_kv=c["kv_high"])


def _places(cu, n):
    """Sequence and place in it of each of n packed tokens."""
    tok = torch.arange(n, device=cu.device)
    seq = torch.searchsorted(cu.long(), tok, right=True) - 1
    return tok, seq, tok - cu.long()[seq]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(s):
    c, x, state = s["c"], s["x"], s["state"]
    B, C, W, n = c["B"], c["C"], c["W"], s["x"].shape[0]
    rows = torch.cat([state.reshape(B * (W - 1), C), x]).float()
    tok, seq, pos = _places(s["cu"], n)
    back = torch.arange(W, device=x.device) - (W - 1)
    at = pos[:, None] + back
    at = torch.where(at >= 0, B * (W - 1) + tok[:, None] + back, seq[:, None] * (W - 1) + W - 1 + at)
    o = (rows[at] * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        o = o + s["bias"]
    if c["silu"]:
        o = _silu(o)
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    last = lens[:, None] + back[1:] - 1
    first = s["cu"][:-1].long()
    number = torch.arange(B, device=x.device)
    last = torch.where(last >= 0, B * (W - 1) + first[:, None] + last, number[:, None] * (W - 1) + W - 1 + last)
    state.copy_(rows[last])
    return dict(o=o.to(x.dtype), state=state)


def _plain_scan(s):
    c, state = s["c"], s["state"]
    C, N, G, n = c["C"], c["N"], c["G"], s["x"].shape[0]
    x, Bm, Cm = s["x"].float(), s["Bm"].float(), s["Cm"].float()
    t = s["dt"].float() + s["dt_bias"]
    t = torch.where(t > 20, t, torch.log1p(torch.exp(t.clamp(max=20))))
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    _, seq, pos = _places(s["cu"], n)
    a = torch.exp(t[:, :, None] * -torch.exp(s["A_log"]))
    b = ((t * x).unflatten(1, (G, -1))[..., None] * Bm[:, :, None]).flatten(1, 2)
    begins = (pos == 0)[:, None, None]
    b = torch.addcmul(b, a * begins, state[seq])
    a = torch.where(begins, torch.zeros_like(a), a)
    # pairs (a, b) of h -> a h + b, joined over 1, 2, 4, ... tokens
    shift = 1
    while shift < s["longest"]:
        b = torch.cat([b[:shift], torch.addcmul(b[shift:], a[shift:], b[:-shift])])
        a = torch.cat([a[:shift], a[shift:] * a[:-shift]])
        shift *= 2
    o = (b.unflatten(1, (G, -1)) * Cm[:, :, None]).sum(-1).flatten(1) + s["D"] * x
    if s["z"] is not None:
        o = o * _silu(s["z"].float())
    ends = (s["cu"][1:].long() - 1).clamp(min=0)
    state.copy_(torch.where((lens > 0)[:, None, None], b[ends], state))
    return dict(o=o.to(s["x"].dtype), state=state)


def _plain_plan(s):
    page, total = s["c"]["page"], s["total"]
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    held, need = -(-old // page), -(-(old + new) // page)
    cu = torch.cat([old.new_zeros(1), torch.cumsum(new, 0)])
    taken = torch.cumsum(need - held, 0) - (need - held)
    left = s["free_count"].long()
    col = torch.arange(s["table"].shape[1], device=old.device)
    fresh = (col >= held[:, None]) & (col < need[:, None])
    at = left - 1 - (taken[:, None] + col - held[:, None])
    at = at.clamp(0, s["free_pages"].shape[0] - 1)
    s["table"].copy_(torch.where(fresh, s["free_pages"][at], s["table"]))
    tok = torch.arange(total, device=old.device)
    req = torch.searchsorted(cu, tok, right=True) - 1
    inside = tok < cu[-1]
    safe = req.clamp(max=old.shape[0] - 1)
    pos = old[safe] + tok - cu[safe]
    pos = torch.where(inside, pos, torch.zeros_like(pos))
    slots = s["table"][safe, pos // page].long() * page + pos % page
    none = torch.full_like(tok, -1)
    return dict(table=s["table"], kv_lens=(old + new).int(), cu=cu.int(), free_count=(left - (need - held).sum()).int(),
                slots=torch.where(inside, slots, none), requests=torch.where(inside, req, none).int(),
                positions=torch.where(inside, pos, none).int())


def _plain_append(s):
    page, slots = s["c"]["page"], s["slots"]
    n, Hkv, D = s["k"].shape
    pool = s["k_cache"].shape[0]
    pages, offs = slots // page, slots % page
    # the lowest offset that is written in each page: what lies below it is there already
    low = torch.full((pool,), page, device=slots.device).scatter_reduce(0, pages, offs, "amin")
    some = pages if n < pool else torch.arange(pool, device=slots.device)    # where anything can change
    out = {}
    for name in ("k", "v"):
        x, cache, scale = s[name].float(), s[name + "_cache"], s[name + "_scale"]
        top = torch.zeros(pool, Hkv, device=x.device).index_reduce(0, pages, x.abs().amax(-1), "amax")
        had = torch.where((low > 0)[:, None], scale, torch.zeros_like(scale))
        grown = torch.maximum(had, top * (1.0 / 127.0))
        safe = torch.where(grown > 0, grown, torch.ones_like(grown))
        before = cache[some].float()
        kept = torch.round(before * scale[some][..., None, None] / safe[some][..., None, None])
        below = (torch.arange(page, device=x.device) < low[some][:, None]) & (low[some] < page)[:, None]
        changed = below[:, None] & (grown > had)[some][:, :, None]
        cache[some] = torch.where(changed[..., None], kept, before).to(torch.int8)
        cache[pages, :, offs] = torch.round(x / safe[pages][..., None]).to(torch.int8)
        scale.copy_(grown)
        out[name], out[name + "_scale"] = cache, scale
    return out


def _plain_attend(s):
    c, q = s["c"], s["q"]
    B, D, page, Hkv = c["B"], c["D"], c["page"], c["Hkv"]
    n, G = q.shape[0], c["Hq"] // c["Hkv"]
    q_lens = (s["cu"][1:] - s["cu"][:-1]).long()
    kv = s["kv_lens"].long()
    at = s["table"].clamp(min=0).long()

    def gathered(cache, scale):                    # [B, Hkv, tokens, D]
        x = cache[at].float() * scale[at][..., None, None]
        return x.transpose(1, 2).flatten(2, 3)

    _, req, place = _places(s["cu"], n)
    rows = torch.zeros(B, c["q_high"], Hkv, G, D, device=q.device)
    rows[req, place] = q.float().unflatten(1, (Hkv, G))
    rows = rows.permute(0, 2, 3, 1, 4).flatten(2, 3)                               # [B, Hkv, G * q, D]
    scores = rows @ gathered(s["k_cache"], s["k_scale"]).transpose(2, 3)           # [B, Hkv, G * q, tokens]
    scores = (scores / math.sqrt(D)).unflatten(2, (G, -1))
    last = (kv - q_lens)[:, None] + torch.arange(c["q_high"], device=q.device)     # [B, q]
    seen = torch.arange(scores.shape[-1], device=q.device) <= last[..., None]
    seen = (seen & (torch.arange(scores.shape[-1], device=q.device) < kv[:, None])[:, None])[:, None, None]
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = p.flatten(2, 3) @ gathered(s["v_cache"], s["v_scale"])
    o = o.unflatten(2, (G, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)               # [B, q, Hq, D]
    return o[req, place].to(q.dtype)


# ------------------------------------------------------------------------------------ 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "plan": lambda s: None, "append": _exact_append,
            "attend": _exact_attend}[c["op"]](s)


def _spans(s):
    cu = s["cu"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_conv(s):
    W, w = s["c"]["W"], s["weight"].double()
    o, state = [], []
    for b, (i, j) in enumerate(_spans(s)):
        u = torch.cat([s["state"][b], s["x"][i:j]]).double()
        y = sum(w[:, k] * u[k:k + j - i] for k in range(W))
        y = y + s["bias"].double() if s["bias"] is not None else y
        o.append(y * torch.sigmoid(y) if s["c"]["silu"] else y)
        state.append(u[u.shape[0] - (W - 1):])
    return dict(o=torch.cat(o), state=torch.stack(state))


def _exact_scan(s):
    c = s["c"]
    spans = _spans(s)
    order = sorted(range(len(spans)), key=lambda b: spans[b][0] - spans[b][1])     # the longest first
    first = torch.tensor([spans[b][0] for b in order], device="cuda")
    lens = [spans[b][1] - spans[b][0] for b in order]
    A = -torch.exp(s["A_log"].double())
    t = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double())
    x, per = s["x"].double(), c["C"] // c["G"]
    Bm, Cm = s["Bm"].double(), s["Cm"].double()
    h = s["state"][order].double()
    o = torch.empty_like(x)
    live = len(order)
    for step in range(lens[0]):
        while lens[live - 1] <= step:
            live -= 1
        at = first[:live] + step
        dt = t[at][:, :, None]
        wide = Bm[at].repeat_interleave(per, 1)
        h[:live] = torch.exp(dt * A) * h[:live] + dt * x[at][:, :, None] * wide
        o[at] = (h[:live] * Cm[at].repeat_interleave(per, 1)).sum(-1)
    o = o + s["D"].double() * x
    if s["z"] is not None:
        z = s["z"].double()
        o = o * z * torch.sigmoid(z)
    state = torch.empty_like(h)
    state[order] = h
    return dict(o=o, state=state)


def _exact_append(s):
    page = s["c"]["page"]
    pages, offs = (s["slots"] // page).tolist(), (s["slots"] % page).tolist()
    begin, end, low = {}, {}, {}
    for i, (p, f) in enumerate(zip(pages, offs)):
        begin.setdefault(p, i)
        low[p] = min(low.get(p, page), f)
        end[p] = i + 1
    out = dict(k=None, v=None)
    for name in ("k", "v"):
        # every scale that the call does not touch is 0 in a page's first use, and as it was otherwise
        scale = s[name + "_scale"].double().clone()
        rows = s[name].double().abs().amax(-1) / 127
        for p in begin:
            top = rows[begin[p]:end[p]].amax(0)
            scale[p] = torch.maximum(scale[p], top) if low[p] > 0 else top
        out[name + "_scale"] = scale
    return out


def _exact_attend(s):
    c = s["c"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (i, j) in enumerate(_spans(s)):
        kv = int(s["kv_lens"][b])
        pages = s["table"][b, :_ceil(kv, c["page"])].long()
        k, v = ((s[m + "_cache"][pages].double() * s[m + "_scale"][pages].double()[..., None, None])
                .transpose(0, 1).flatten(1, 2)[:, :kv].repeat_interleave(G, 0) for m in ("k", "v"))
        q = s["q"][i:j].double().transpose(0, 1)
        w = q @ k.transpose(1, 2) / math.sqrt(D)
        w = w + torch.full((j - i, kv), float("-inf"), dtype=torch.float64, device="cuda").triu(kv - (j - i) + 1)
        o[i:j] = (torch.softmax(w, -1) @ v).transpose(0, 1)
    return o


# ------------------------------------------------------------------------------------ the work


def work(c):
    op = c["op"]
    size = 2 if c.get("dtype") == "bf16" else 4
    if op in ("conv", "scan"):
        n, B, C = sum(_lengths(c["B"], c["low"], c["high"])), c["B"], c["C"]
        if op == "conv":
            W = c["W"]
            return dict(bytes=2 * n * C * size + 2 * B * (W - 1) * C * size + 4 * C * W, flops=n * C * (2 * W + 4))
        N, G = c["N"], c["G"]
        rows = n * (C * (4 if c["gate"] else 3) + 2 * G * N) * size
        return dict(bytes=rows + 8 * B * C * N + 4 * C * N, flops=n * C * (7 * N + 8))
    page = c["page"]
    if op == "plan":
        new, old = _lengths(c["B"], c["new_low"], c["new_high"]), list(reversed(_lengths(c["B"], 0, c["old"])))
        fresh = sum(_ceil(a + b, page) - _ceil(a, page) for a, b in zip(old, new))
        return dict(bytes=16 * c["B"] + 8 * fresh + 16 * (sum(new) + c["pad"]), flops=4 * (sum(new) + c["B"]))
    if op == "append":
        n = sum(_lengths(c["B"], c["low"], c["high"]))
        held = sum(1 for a, b in zip(_old_lengths(c), _lengths(c["B"], c["low"], c["high"])) if b)
        elements = 2 * n * c["Hkv"] * c["D"]
        return dict(bytes=elements * (size + 1) + 8 * n + 16 * c["Hkv"] * (held + n // page), flops=4 * elements)
    q_lens, kv_lens = _lengths(c["B"], c["q_low"], c["q_high"]), _lengths(c["B"], c["kv_low"], c["kv_high"])
    seen = sum(q * kv - q * (q - 1) // 2 for q, kv in zip(q_lens, kv_lens))
    cached = sum(kv_lens) * c["Hkv"] * 2 * (c["D"] + 4 / page)
    return dict(bytes=cached + 2 * sum(q_lens) * c["Hq"] * c["D"] * size, flops=4 * seen * c["Hq"] * c["D"])
