"""Measured cases of the operators around a layer's state: norm, 8-bit products, rotary positions.

Six kinds of call, each with its plain torch form (``own`` false) and the library call (``own``
true): the root-mean-square norm with the residual's addition, the same with an output in 8 bits
(e4m3, a scale for each 128 values), the quantisers of rows and of weights, the matrix product of
such operands, and the rotation of queries and keys by their positions.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # before the projections of a decode step of 64 requests, width of 32 heads of 128
        dict(name="norm-step", op="norm8", n=64, H=1, C=4096, dtype="bf16", residual=True, pad=0),
        # the same layer with prompts of 4001 tokens in all
        dict(name="norm-prompt", op="norm8", n=4001, H=1, C=4096, dtype="bf16", residual=True, pad=0),
        # every query head by itself, read from a packed row
        dict(name="norm-heads", op="norm", n=4000, H=32, C=128, dtype="bf16", residual=False, pad=4096),
        # the output of an attention layer, before the projection that follows it
        dict(name="quantize-rows", op="rows", n=4001, K=4096, dtype="bf16", pad=0),
        # a projection's weights, once when they are loaded
        dict(name="quantize-weight", op="blocks", N=12288, K=4096, dtype="bf16"),
        # q | k | v of one token
        dict(name="matmul-one", op="matmul", n=1, N=12288, K=4096, out="bf16", pad=0),
        # of a decode step of 64 requests
        dict(name="matmul-step", op="matmul", n=64, N=12288, K=4096, out="bf16", pad=0),
        # of prompts of 4001 tokens
        dict(name="matmul-prompt", op="matmul", n=4001, N=12288, K=4096, out="bf16", pad=0),
        # of a short prompt into a narrow, ragged output in 32 bits, as logits or decay rates are wanted
        dict(name="matmul-ragged", op="matmul", n=517, N=1003, K=4112, out="f32", pad=48),
        # a decode step of 64 requests at up to a million positions, 32 heads on 8
        dict(name="rotary-step", op="rotary", n=64, Hq=32, Hk=8, D=128, R=128, far=1 << 20, interleaved=False, dtype="bf16", skip=0),
        # prompts of 4000 tokens, rows of the packed projection
        dict(name="rotary-prompt", op="rotary", n=4000, Hq=32, Hk=8, D=128, R=128, far=8000, interleaved=False, dtype="bf16", skip=0),
        # a part of each head, neighbouring channels turned together, padding behind the tokens
        dict(name="rotary-part", op="rotary", n=4011, Hq=24, Hk=24, D=96, R=48, far=131072, interleaved=True, dtype="f32", skip=11),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw(rng):
    op = rng.choice(["norm", "norm8", "rows", "blocks", "matmul", "matmul", "matmul", "rotary", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm8"):
        heads = op == "norm" and rng.random() < 0.4
        C = 8 * (rng.choice([4, 8, 16, 24, 32]) if heads else _log_int(rng, 8, 2048))
        return dict(op=op, n=_log_int(rng, 1, 8000), H=_log_int(rng, 2, 64) if heads else 1, C=C, dtype=dtype,
                    residual=rng.random() < 0.6, pad=8 * rng.choice([0, 0, 1, 5]))
    if op == "rows":
        return dict(op=op, n=_log_int(rng, 1, 8000), K=8 * _log_int(rng, 8, 1536), dtype=dtype, pad=8 * rng.choice([0, 0, 3]))
    if op == "blocks":
        return dict(op=op, N=_log_int(rng, 8, 12288), K=8 * _log_int(rng, 8, 1536), dtype=dtype)
    if op == "matmul":
        return dict(op=op, n=_log_int(rng, 1, 8000), N=_log_int(rng, 8, 12288), K=16 * _log_int(rng, 4, 768),
                    out=rng.choice(["bf16", "bf16", "f32"]), pad=16 * rng.choice([0, 0, 2]))
    D = rng.choice([32, 64, 80, 96, 128, 128, 256])
    Hk = rng.choice([1, 2, 4, 8, 8, 24])
    return dict(op=op, n=_log_int(rng, 1, 8000), Hq=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, D=D,
                R=rng.choice([D, D, D // 2, 8 * rng.randint(1, D // 8)]), far=_log_int(rng, 100, 1 << 20),
                interleaved=rng.random() < 0.4, dtype=dtype, skip=rng.choice([0, 0, 5]))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    tops = {}
    for c in listed():
        op = c["op"].rstrip("8")
        tops[op] = max(tops.get(op, 0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= tops[c["op"].rstrip("8")]:
            return c


# ------------------------------------------------------------------------------------ inputs

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0                       # the largest e4m3 value
LEAST = 2.0 ** -126               # the least scale


def _ceil(a, b):
    return -(-a // b)


def _by_groups(x, rows):
    """x [n, K] in 32 bits as blocks of ``rows`` x 128 values, zeros behind the end: [blocks, rows, blocks, 128]."""
    n, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128, 0, -n % rows)).unflatten(1, (-1, 128)).unflatten(0, (-1, rows))


def _quantised(x, rows):
    """8-bit values and scales of x [n, K]."""
    g = _by_groups(x, rows)
    top = g.abs().amax((1, 3))
    scale = (top * (1 / TOP)).clamp(min=LEAST)
    y = (g * (1 / scale)[:, None, :, None]).clamp(-TOP, TOP)
    return y.flatten(0, 1).flatten(1)[:x.shape[0], :x.shape[1]].to(E4M3), scale


def _wide(y, scale, rows):
    """The values that 8-bit ones stand for."""
    n, K = y.shape
    return y.to(scale.dtype) * scale.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :K]


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s, op = dict(c=c), c["op"]
    if op in ("norm", "norm8"):
        n, H, C, dt = c["n"], c["H"], c["C"], DTYPES[c["dtype"]]
        # channels of different sizes, a few of them large, as in a residual stream
        size = torch.exp(randn(C) * 0.7)
        rows = randn(n, H * C + c["pad"]).to(dt)[:, c["pad"]:]
        s["x"] = rows if H == 1 else rows.unflatten(1, (H, C))
        s["residual"] = (randn(*s["x"].shape) * 3 * size).to(dt) if c["residual"] else None
        s["weight"] = 1 + 0.2 * randn(C)
        return s
    if op == "rows":
        s["x"] = (randn(c["n"], c["K"] + c["pad"]) * torch.exp(randn(c["n"], 1))).to(DTYPES[c["dtype"]])[:, c["pad"]:]
        return s
    if op == "blocks":
        s["w"] = (randn(c["N"], c["K"]) / math.sqrt(c["K"])).to(DTYPES[c["dtype"]])
        return s
    if op == "matmul":
        n, N, K = c["n"], c["N"], c["K"]
        y, s["xs"] = _quantised(randn(n, K) * torch.exp(randn(K) * 0.5), 1)
        s["x"] = torch.nn.functional.pad(y.view(torch.uint8), (0, c["pad"])).view(E4M3)[:, :K]
        s["w"], s["ws"] = _quantised(randn(N, K) / math.sqrt(K), 128)
        return s
    n, Hq, Hk, D, R, dt = c["n"], c["Hq"], c["Hk"], c["D"], c["R"], DTYPES[c["dtype"]]
    # q | k | v as a projection leaves them
    row = randn(n, (Hq + 2 * Hk) * D).to(dt)
    s["q"], s["k"] = (t.unflatten(1, (-1, D)) for t in row.split([Hq * D, Hk * D, Hk * D], 1)[:2])
    pos = torch.randint(0, c["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
    pos[n - min(c["skip"], n - 1):] = -1              # rows behind the last token
    s["pos"] = pos
    s["freq"] = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    return s


# ------------------------------------------------------------------------------------ the passes


def run(s):
    op = s["c"]["op"]
    if own:
        return {"norm": _own_norm, "norm8": _own_norm8, "rows": _own_rows, "blocks": _own_blocks, "matmul": _own_matmul,
                "rotary": _own_rotary}[op](s)
    return {"norm": _plain_norm, "norm8": _plain_norm, "rows": _plain_rows, "blocks": _plain_blocks, "matmul": _plain_matmul,
            "rotary": _plain_rotary}[op](s)


def _own_norm(s):
    import gated_delta_rule_channelwise_gb300 as cg
    return dict(o=cg.rms_norm(s["x"], s["weight"], residual=s["residual"]), residual=s["residual"])


def _own_norm8(s):
    import gated_delta_rule_channelwise_gb300 as cg
    y, scale = cg.rms_norm_fp8(s["x"], s["weight"], residual=s["residual"])
    return dict(y=y, scale=scale, residual=s["residual"])


def _own_rows(s):
    import gated_delta_rule_channelwise_gb300 as cg
    y, scale = cg.fp8_quantize(s["x"])
    return dict(y=y, scale=scale)


def _own_blocks(s):
    import gated_delta_rule_channelwise_gb300 as cg
    y, scale = cg.fp8_quantize_weight(s["w"])
    return dict(y=y, scale=scale)


def _own_matmul(s):
    import gated_delta_rule_channelwise_gb300 as cg
    return cg.fp8_matmul(s["x"], s["xs"], s["w"], s["ws"], dtype=DTYPES[s["c"]["out"]])


def _own_rotary(s):
    import gated_delta_rule_channelwise_gb300 as cg
    cg.rotary(s["q"], s["k"], s["pos"], s["freq"], interleaved=s["c"]["interleaved"])
    return dict(q=s["q"], k=s["k"])


def _plain_norm(s):
    x, r = s["x"], s["residual"]
    h = x.float()
    if r is not None:
        h = h + r.float()
        r.copy_(h)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    if s["c"]["op"] == "norm":
        return dict(o=y.to(x.dtype), residual=r)
    y, scale = _quantised(y, 1)
    return dict(y=y, scale=scale, residual=r)


def _plain_rows(s):
    y, scale = _quantised(s["x"].float(), 1)
    return dict(y=y, scale=scale)


def _plain_blocks(s):
    y, scale = _quantised(s["w"].float(), 128)
    return dict(y=y, scale=scale)


def _plain_matmul(s):
    o = _wide(s["x"], s["xs"], 1) @ _wide(s["w"], s["ws"], 128).t()
    return o.to(DTYPES[s["c"]["out"]])


def _plain_rotary(s):
    c, pos = s["c"], s["pos"]
    a = pos.double()[:, None] * s["freq"]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    R = c["R"]
    for x in (s["q"], s["k"]):
        part = x[..., :R].float()
        u, v = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :R // 2], part[..., R // 2:])
        turned = u * cos - v * sin, v * cos + u * sin
        turned = torch.stack(turned, -1).flatten(-2) if c["interleaved"] else torch.cat(turned, -1)
        x[..., :R] = torch.where((pos >= 0)[:, None, None], turned, part).to(x.dtype)
    return dict(q=s["q"], k=s["k"])


# ------------------------------------------------------------------------------------ 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "norm8": _exact_norm, "rows": lambda s: _exact_scales(s["x"].double(), 1),
            "blocks": lambda s: _exact_scales(s["w"].double(), 128), "matmul": _exact_matmul, "rotary": _exact_rotary}[c["op"]](s)


def _exact_scales(x, rows):
    """The values in 8 bits are rounded ones; their scales are numbers."""
    top = torch.stack([torch.stack([b.abs().max() for b in part.split(128, 1)]) for part in x.split(rows)]) if rows > 1 else \
        torch.stack([part.abs().amax(1) for part in x.split(128, 1)], 1)
    return dict(y=None, scale=(top / TOP).clamp(min=LEAST))


def _exact_norm(s):
    h, r = s["x"].double(), s["residual"]
    if r is not None:
        h = h + r.double()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].double()
    out = dict(o=y) if s["c"]["op"] == "norm" else _exact_scales(y, 1)
    return dict(out, residual=None if r is None else h)


def _exact_matmul(s):
    x, w, n = s["x"].double(), s["w"].double(), s["x"].shape[0]
    o = torch.zeros(n, w.shape[0], dtype=torch.float64, device="cuda")
    by = s["ws"].double().repeat_interleave(128, 0)[:w.shape[0]]
    for b, (xb, wb) in enumerate(zip(x.split(128, 1), w.split(128, 1))):
        o += (xb * s["xs"][:, b:b + 1].double()) @ (wb * by[:, b:b + 1]).t()
    return o


def _exact_rotary(s):
    c, keep = s["c"], (s["pos"] < 0)[:, None]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"])
    turn = torch.where(keep, torch.ones_like(turn), turn)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        part = x[..., :c["R"]]
        pairs = part.unflatten(-1, (-1, 2)) if c["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        out[name] = torch.cat([z, x[..., c["R"]:]], -1)
    return out


# ------------------------------------------------------------------------------------ the work


def work(c):
    op = c["op"]
    size = 2 if c.get("dtype") == "bf16" else 4
    if op in ("norm", "norm8"):
        rows, C = c["n"] * c["H"], c["C"]
        moved = size * (3 if c["residual"] else 1) + (size if op == "norm" else 1)
        return dict(bytes=rows * C * moved + 4 * C + (4 * rows * _ceil(C, 128) if op == "norm8" else 0), flops=6 * rows * C)
    if op == "rows":
        return dict(bytes=c["n"] * (c["K"] * (size + 1) + 4 * _ceil(c["K"], 128)), flops=3 * c["n"] * c["K"])
    if op == "blocks":
        return dict(bytes=c["N"] * c["K"] * (size + 1) + 4 * _ceil(c["N"], 128) * _ceil(c["K"], 128), flops=3 * c["N"] * c["K"])
    if op == "matmul":
        n, N, K = c["n"], c["N"], c["K"]
        blocks = _ceil(K, 128)
        return dict(bytes=(n + N) * K + 4 * blocks * (n + _ceil(N, 128)) + n * N * (2 if c["out"] == "bf16" else 4), flops=2 * n * N * K)
    turned = c["n"] * (c["Hq"] + c["Hk"]) * c["R"]
    return dict(bytes=2 * size * turned + 4 * c["n"] + 4 * c["R"], flops=3 * turned)
