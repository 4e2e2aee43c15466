"""Plain 64-bit forms of the serving operators, on the CPU, straight from their formulas."""
from __future__ import annotations

import math

import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def silu(x):
    return x / (1 + torch.exp(-x))


def spans_of(B, T, cu):
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    cu = cu.cpu().tolist()
    return list(zip(cu[:-1], cu[1:]))


def conv(x, weight, state, bias, act, spans):
    """Packed rows x [n, C]; returns (y [n, C], new state)."""
    x, w, state, bias = f64(x), f64(weight), f64(state), f64(bias)
    W = w.shape[1]
    y, new = torch.zeros_like(x), state.clone()
    for b, (i, j) in enumerate(spans):
        u = torch.cat([state[b], x[i:j]])
        acc = sum(w[:, k] * u[k:k + j - i] for k in range(W)) + (0 if bias is None else bias)
        y[i:j] = silu(acc) if act else acc
        new[b] = u[u.shape[0] - (W - 1):]
    return y, new


def scan(x, dt, A_log, Bm, Cm, state, D, z, dt_bias, softplus, spans):
    """Packed rows x [n, C], Bm [n, G, N]; returns (y [n, C], new state)."""
    x, dt, A_log, Bm, Cm, h0, D, z, dt_bias = map(f64, (x, dt, A_log, Bm, Cm, state, D, z, dt_bias))
    per = x.shape[1] // Bm.shape[1]
    A = -torch.exp(A_log)
    d = dt if dt_bias is None else dt + dt_bias
    if softplus:
        d = torch.where(d > 20, d, torch.log1p(torch.exp(d.clamp(max=20))))
    y, new = torch.zeros_like(x), h0.clone()
    for b, (i, j) in enumerate(spans):
        h = h0[b].clone()
        for t in range(i, j):
            h = torch.exp(A * d[t][:, None]) * h + (d[t] * x[t])[:, None] * Bm[t].repeat_interleave(per, 0)
            y[t] = (Cm[t].repeat_interleave(per, 0) * h).sum(-1)
        new[b] = h
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * silu(z)
    return y, new


def plan(table, seq, new, free, count, n_tokens, page):
    """Returns a dict of lists, the table updated in place; None if the pages or the table do not suffice."""
    need = [-(-(s + a) // page) - -(-s // page) for s, a in zip(seq, new)]
    if sum(need) > count or sum(new) > n_tokens or any(-(-(s + a) // page) > len(r) for s, a, r in zip(seq, new, table)):
        return None
    out = dict(cu=[0], kv=[], slots=[], requests=[], positions=[])
    for b, (s, a) in enumerate(zip(seq, new)):
        for k in range(need[b]):
            count -= 1
            table[b][-(-s // page) + k] = free[count]
        for pos in range(s, s + a):
            out["slots"].append(table[b][pos // page] * page + pos % page)
            out["requests"].append(b)
            out["positions"].append(pos)
        out["cu"].append(out["cu"][-1] + a)
        out["kv"].append(s + a)
    for name in ("slots", "requests", "positions"):
        out[name] += [-1] * (n_tokens - len(out[name]))
    out["count"] = count
    return out


def append(x, slots, cache, scale):
    """x [n, Hkv, D] into (int8 cache, fp32 scales), in fp32 steps: the rounding is part of the definition."""
    x, cache, scale = x.detach().cpu().float(), cache.cpu().clone(), scale.cpu().clone()
    page, slots, n = cache.shape[2], slots.cpu().tolist(), len(slots)
    i = 0
    while i < n:
        if slots[i] < 0:
            i += 1
            continue
        p, off = divmod(slots[i], page)
        j = i + 1
        while j < n and slots[j] == slots[j - 1] + 1 and slots[j] % page:
            j += 1
        had = scale[p] if off else torch.zeros_like(scale[p])
        grown = torch.maximum(had, x[i:j].abs().amax((0, 2)) * torch.tensor(1.0 / 127.0, dtype=torch.float32))
        by = torch.where(grown > 0, grown, torch.ones_like(grown))[:, None, None]
        if off:
            kept = torch.round(cache[p, :, :off].float() * had[:, None, None] / by).to(torch.int8)
            cache[p, :, :off] = torch.where((grown > had)[:, None, None], kept, cache[p, :, :off])
        cache[p, :, off:off + j - i] = torch.round(x[i:j].transpose(0, 1) / by).to(torch.int8)
        scale[p] = grown
        i = j
    return cache, scale


def attend(q, kc, vc, ks, vs, table, kv_lens, spans, scale=None):
    """Returns (o, sum p |v|), both [n, Hq, D]: the second is what absolute errors are measured by."""
    q = f64(q)
    n, Hq, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    kc, vc, ks, vs = f64(kc), f64(vc), f64(ks), f64(vs)
    o, size = torch.zeros_like(q), torch.zeros_like(q)
    for b, (i, j) in enumerate(spans):
        kv = int(kv_lens[b])
        pages = table[b, :-(-kv // page)].long().cpu() if kv > 0 else torch.zeros(0, dtype=torch.long)
        K = (kc[pages] * ks[pages][..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :max(kv, 0)]
        V = (vc[pages] * vs[pages][..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :max(kv, 0)]
        for t in range(i, j):
            see = min(kv, kv - (j - i) + (t - i) + 1)
            if see <= 0:
                continue
            for h in range(Hq):
                k, v = K[h // (Hq // Hkv), :see], V[h // (Hq // Hkv), :see]
                p = torch.softmax(k @ q[t, h] * (1 / math.sqrt(D) if scale is None else scale), 0)
                o[t, h], size[t, h] = p @ v, p @ v.abs()
    return o, size
