"""A small hybrid decoder served with this library: delta-rule, selective-scan and attention layers.

    python examples/hybrid_decoder.py

Random weights, torch for the projections, and the library for everything that carries state: the
short causal convolution in front of the recurrent layers, the channelwise gated delta rule, the
selective scan, and a paged 8-bit cache whose block tables are built on the GPU.  Requests of
different lengths are packed into one step; a step of prompts and a step of single tokens take the
same path, and a prompt followed by tokens gives the logits of the whole sequence (up to the
rounding of bf16 and of the cache, whose scales depend on what a page has held so far).
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_channelwise_gb300 as cg  # noqa: E402

BF = torch.bfloat16


class HybridDecoder:
    """``layers`` of "delta", "scan" and "attend" over a width of heads x 128; serves ``B`` requests."""

    def __init__(self, layers=("delta", "scan", "attend", "delta"), heads=4, kv_heads=2, vocab=512, states=16, taps=4,
                 B=3, pages=64, page=64, table_width=16, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.kinds, self.H, self.Hkv, self.d = layers, heads, kv_heads, 128
        self.C, self.N, self.W, self.B, self.page = heads * 128, states, taps, B, page
        C = self.C

        def weight(n_in, n_out):
            return (torch.randn(n_in, n_out, generator=g, device=device) / math.sqrt(n_in)).to(BF)

        def rand(*shape):
            return torch.rand(*shape, generator=g, device=device)

        self.embedding, self.head = weight(vocab, C) * math.sqrt(vocab), weight(C, vocab)
        self.layers = []
        for kind in layers:
            p = dict(kind=kind, out=weight(C, C))
            if kind == "delta":                       # q | k | v in one row, per-channel decay and write strength
                p.update(qkv=weight(C, 3 * C), decay=weight(C, C), beta=weight(C, heads), taps=rand(3 * C, taps) - 0.5)
            elif kind == "scan":
                p.update(xz=weight(C, 2 * C), dt=weight(C, C), bc=weight(C, 2 * states), taps=rand(C, taps) - 0.5,
                         A_log=torch.log(torch.arange(1, states + 1, device=device).float()).repeat(C, 1),
                         D=torch.ones(C, device=device), dt_bias=rand(C) * 4 - 6)
            else:
                p.update(qkv=weight(C, C + 2 * kv_heads * 128))
            self.layers.append(p)
        # what the requests keep: conv rows and recurrent states, caches, one block table for all attention layers
        zeros = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=device)
        self.state = []
        for p in self.layers:
            if p["kind"] == "delta":
                self.state.append(dict(conv=zeros(B, taps - 1, 3 * C, dtype=BF), S=zeros(B, heads, 128, 128)))
            elif p["kind"] == "scan":
                self.state.append(dict(conv=zeros(B, taps - 1, C, dtype=BF), h=zeros(B, C, states)))
            else:
                cache = lambda: zeros(pages, kv_heads, page, 128, dtype=torch.int8)
                self.state.append(dict(k=cache(), v=cache(), ks=zeros(pages, kv_heads), vs=zeros(pages, kv_heads)))
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((B, table_width), -1, **i32)
        self.lens = torch.zeros(B, **i32)
        self.free_pages, self.free_count = torch.arange(pages, **i32), torch.full((1,), pages, **i32)
        self.status = torch.zeros(1, **i32)

    @staticmethod
    def norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(BF)

    def step(self, tokens, lens):
        """``tokens``: the new ids of all requests, packed; ``lens``: how many of each (known on the host, as
        the ids are).  Returns the logits of every new token."""
        n, longest = sum(lens), max(lens)
        single = longest == min(lens) == 1
        new = torch.tensor(lens, dtype=torch.int32).to(self.lens.device, non_blocking=True)
        plan = cg.cache_plan(self.table, self.lens, new, self.free_pages, self.free_count, n, self.page,
                             num_pages=self.free_pages.numel(), status=self.status)
        self.lens, self.free_count = plan.kv_lens, plan.free_count
        x = self.embedding[tokens]
        for p, s in zip(self.layers, self.state):
            x = x + getattr(self, "_" + p["kind"])(p, s, self.norm(x), plan, lens, longest, single) @ p["out"]
        return self.norm(x) @ self.head

    def _conv(self, x, taps, state, plan, single):
        return cg.conv_decode(x, taps, state) if single else cg.conv_prefill(x, taps, state, cu_seqlens=plan.cu_seqlens)

    def _delta(self, p, s, x, plan, lens, longest, single):
        rows = self._conv(x @ p["qkv"], p["taps"], s["conv"], plan, single)
        q, k, v = (t.unflatten(-1, (self.H, self.d)) for t in rows.split(self.C, -1))       # views of the packed row
        g = -torch.nn.functional.softplus((x @ p["decay"]).float()).unflatten(-1, (self.H, self.d)) * 0.1
        beta = torch.sigmoid((x @ p["beta"]).float())
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
        if single:
            cg.decode(q, k, v, s["S"], o, g=g, beta=beta)
        else:
            at = 0
            for b, l in enumerate(lens):              # the chunked prefill takes one length a call
                r = slice(at, at + l)
                if l:
                    cg.prefill(q[None, r], k[None, r], v[None, r], s["S"][b:b + 1], o[None, r], g=g[None, r],
                               beta=beta[None, r])
                at += l
        return o.flatten(1)

    def _scan(self, p, s, x, plan, lens, longest, single):
        u, z = (x @ p["xz"]).split(self.C, -1)
        u = self._conv(u, p["taps"], s["conv"], plan, single)
        Bm, Cm = (x @ p["bc"]).unsqueeze(1).split(self.N, -1)
        kw = dict(D=p["D"], z=z, dt_bias=p["dt_bias"])
        if single:
            return cg.scan_decode(u, x @ p["dt"], p["A_log"], Bm, Cm, s["h"], **kw)
        return cg.scan_prefill(u, x @ p["dt"], p["A_log"], Bm, Cm, s["h"], cu_seqlens=plan.cu_seqlens, **kw)

    def _attend(self, p, s, x, plan, lens, longest, single):
        q, k, v = (x @ p["qkv"]).split([self.C, self.Hkv * self.d, self.Hkv * self.d], -1)
        q, k, v = (t.unflatten(-1, (-1, self.d)) for t in (q, k, v))
        cg.cache_append(k, v, plan.slots, s["k"], s["v"], s["ks"], s["vs"], status=self.status)
        return cg.cache_attend(q, s["k"], s["v"], s["ks"], s["vs"], self.table, self.lens, plan.cu_seqlens, max_q=longest,
                               status=self.status).flatten(1)


def compare(lens=(70, 1, 133), tail=5, seed=0):
    """Largest logit difference, over the logits' RMS, between whole sequences in one step and prompts
    followed by ``tail`` steps of single tokens."""
    B = len(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = [torch.randint(0, 512, (l + tail,), generator=g, device="cuda") for l in lens]
    whole, parts = HybridDecoder(B=B), HybridDecoder(B=B)
    full = whole.step(torch.cat(ids), [l + tail for l in lens]).split([l + tail for l in lens])
    got = [parts.step(torch.cat([t[:l] for t, l in zip(ids, lens)]), list(lens)).split(list(lens))]
    for k in range(tail):
        got.append(parts.step(torch.stack([t[l + k] for t, l in zip(ids, lens)]), [1] * B).split([1] * B))
    assert int(whole.status) == int(parts.status) == cg.OK
    joined = [torch.cat([step[b] for step in got]) for b in range(B)]
    ref = torch.cat(full).float()
    return float((torch.cat(joined).float() - ref).abs().max() / ref.square().mean().sqrt())


if __name__ == "__main__":
    print("prompts then tokens against whole sequences: largest difference %.3f of the logits' RMS" % compare())
