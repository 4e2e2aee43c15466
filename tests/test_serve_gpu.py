"""GPU parity of the serving operators (cgdr_serve.h) against their plain 64-bit forms.

Tolerances, derived from the kernels' arithmetic (u = 2^-24, RMS of the reference r):

* convolution, fp32: at most W+1 roundings of terms of up to 6 r, and an activation whose
  exponential and reciprocal are good to 2^-21: 1e-5 r.  bf16 rounds the result once more: + 2^-8 |y|.
* scan, fp32: every step multiplies the state by an exponential good to 2^-21, so T <= 300 steps
  leave at most 1.5e-4 of it, in one direction only if all errors agree: 1e-4 r.  bf16 outputs: + 2^-8 |y|.
* attention: probabilities rounded to fp16 (2^-11 each) and, in bf16, the result to 2^-8: with
  m = sum p |v|, 2^-10 m + 2^-8 |o|.  fp32: two fp16 parts, scores good to 2^-20 of about 20: 3e-5 m.
* plan and append are defined to the bit and compared for equality.
"""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
import serve_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)


def close(got, want, atol, dtype=F32):
    """|got - want| <= atol + one rounding to dtype; non-finite values have to agree."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = (got - want).abs()[fine] - (want.abs()[fine] * 2.0 ** -8 if dtype == BF else 0)
    bound = (atol if not torch.is_tensor(atol) else atol[fine])
    assert bool((off <= bound).all()), float((off - bound).max())


def rms(t):
    return float(t.pow(2).mean().sqrt().clamp_min(1e-30)) if t.numel() else 0.0


# ------------------------------------------------------------------------------------ convolution


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2], [3, 1, 1, 2], [0, 5, 0, 0, 77, 1], [8] * 9, [65, 0, 1, 130], [1] * 40 + [0]])
@pytest.mark.parametrize("silu,bias", [(True, False), (False, True)])
def test_conv_packed(dtype, W, lens, silu, bias):
    g = gen(W + sum(lens))
    C, n = 40, sum(lens)
    x = randn(g, n, C + 24).to(dtype)[:, 16:16 + C]                    # rows of a wider projection
    w, b = randn(g, C, W), randn(g, C) if bias else None
    state = randn(g, len(lens), W - 1, C).to(dtype)
    cu = offsets(lens)
    want, new = ref.conv(x, w, state, b, silu, ref.spans_of(0, 0, cu))
    o = cg.conv_prefill(x, w, state, bias=b, silu=silu, cu_seqlens=cu)
    close(o, want, 1e-5 * rms(want), dtype)
    assert torch.equal(state.cpu().double(), new)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (3, 1, 1032), (70, 1, 64), (2, 2, 8), (3, 100, 72), (1, 257, 2056)])
def test_conv_dense(dtype, B, T, C):
    g = gen(B + T + C)
    W = 4
    x = randn(g, B, T + 3, C + 8).to(dtype)[:, 2:2 + T, 8:]
    w, b = randn(g, C, W), randn(g, C)
    state = randn(g, B, W - 1, C).to(dtype)
    want, new = ref.conv(x.reshape(-1, C), w, state, b, True, ref.spans_of(B, T, None))
    o = cg.conv_prefill(x, w, state, bias=b)
    close(o, want.view(B, T, C), 1e-5 * rms(want), dtype)
    assert torch.equal(state.cpu().double(), new)


def test_conv_prompt_then_tokens_equals_one_prompt():
    g = gen(3)
    B, T, C, W = 3, 50, 48, 4
    x, w = randn(g, B, T, C).to(BF), randn(g, C, W)
    zero = lambda: torch.zeros(B, W - 1, C, dtype=BF, device=DEV)
    s1, s2 = zero(), zero()
    whole = cg.conv_prefill(x, w, s1)
    parts = [cg.conv_prefill(x[:, :30], w, s2)] + [cg.conv_decode(x[:, t], w, s2)[:, None] for t in range(30, T)]
    assert torch.equal(whole, torch.cat(parts, 1)) and torch.equal(s1, s2)


def test_conv_non_finite_values_stay_in_their_window():
    g = gen(4)
    C, W = 8, 4
    x, w, state = randn(g, 40, C), randn(g, C, W), randn(g, 2, W - 1, C)
    x[7, 3], x[20, 5] = float("nan"), float("inf")
    cu = offsets([9, 31])
    want, _ = ref.conv(x, w, state, None, False, ref.spans_of(0, 0, cu))
    got = cg.conv_prefill(x, w, state, silu=False, cu_seqlens=cu)
    close(got, want, 1e-5 * rms(want[torch.isfinite(want)]))


# ------------------------------------------------------------------------------------ scan


def scan_inputs(g, n, B, C, N, G, dtype, gate):
    s = dict(x=randn(g, n, C).to(dtype), dt=randn(g, n, C).to(dtype), Bm=randn(g, n, G, N).to(dtype),
             Cm=randn(g, n, G, N).to(dtype), z=randn(g, n, C).to(dtype) if gate else None,
             A_log=torch.rand(C, N, generator=g, device=DEV) * 3 - 1, D=randn(g, C) if gate else None,
             dt_bias=randn(g, C) - 2, state=randn(g, B, C, N))
    return s


def scan_ref(s, spans, softplus=True):
    return ref.scan(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], s["D"], s["z"], s["dt_bias"], softplus, spans)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,G,C", [(16, 1, 24), (16, 2, 48), (32, 1, 8), (64, 3, 120), (128, 1, 40)])
@pytest.mark.parametrize("lens", [[1], [31, 0, 1, 33], [64, 2, 200]])
@pytest.mark.parametrize("gate", [False, True])
def test_scan_packed(dtype, N, G, C, lens, gate):
    g = gen(N + C + sum(lens))
    n, B, cu = sum(lens), len(lens), offsets(lens)
    s = scan_inputs(g, n, B, C, N, G, dtype, gate)
    want, new = scan_ref(s, ref.spans_of(0, 0, cu))
    o = cg.scan_prefill(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                        cu_seqlens=cu)
    close(o, want, 1e-4 * rms(want), dtype)
    close(s["state"], new, 1e-4 * rms(new))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,N", [(1, 1, 8, 16), (5, 1, 72, 16), (3, 1, 40, 128), (2, 2, 16, 16), (2, 300, 24, 32),
                                     (3, 65, 2560, 16)])
def test_scan_dense_and_step(dtype, B, T, C, N):
    g = gen(B + T + C)
    s = scan_inputs(g, B * T, B, C, N, 1, dtype, True)
    want, new = scan_ref(s, ref.spans_of(B, T, None))
    v = lambda t: t.unflatten(0, (B, T))
    if T == 1:
        o = cg.scan_decode(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    else:
        wide = torch.zeros(B, T + 1, C + 16, dtype=F32, device=DEV)      # a strided fp32 output
        o = cg.scan_prefill(v(s["x"]), v(s["dt"]), s["A_log"], v(s["Bm"]), v(s["Cm"]), s["state"], wide[:, 1:, 8:8 + C],
                            D=s["D"], z=v(s["z"]), dt_bias=s["dt_bias"])
        assert not wide[:, 0].any() and not wide[:, :, :8].any() and not wide[:, :, 8 + C:].any()
    close(o.reshape(B * T, C), want, 1e-4 * rms(want), dtype if T == 1 else F32)
    close(s["state"], new, 1e-4 * rms(new))


def test_scan_raw_steps_and_extremes():
    """softplus off; with it, arguments over the whole range (large, tiny and negative steps)."""
    g = gen(9)
    s = scan_inputs(g, 40, 1, 16, 16, 1, F32, False)
    s["dt"] = torch.linspace(0, 3, 40 * 16, device=DEV).view(40, 16)
    s["dt_bias"] = None
    want, new = scan_ref(s, [(0, 40)], softplus=False)
    o = cg.scan_prefill(s["x"][None], s["dt"][None], s["A_log"], s["Bm"][None], s["Cm"][None], s["state"], softplus=False)
    close(o[0], want, 1e-4 * rms(want))
    s["dt"] = torch.linspace(-60, 60, 40 * 16, device=DEV).view(40, 16)
    want, new = scan_ref(s, [(0, 40)])
    o = cg.scan_prefill(s["x"][None], s["dt"][None], s["A_log"], s["Bm"][None], s["Cm"][None], s["state"])
    close(o[0], want, 1e-4 * rms(want))
    close(s["state"], new, 1e-4 * rms(new))


def test_scan_prompt_then_tokens():
    """A prompt in one call, in two, and token by token: the same recurrence up to rounding."""
    g = gen(10)
    B, T, C, N = 2, 90, 32, 16
    s = scan_inputs(g, B * T, B, C, N, 1, F32, True)
    v = {k: s[k].unflatten(0, (B, T)) for k in ("x", "dt", "Bm", "Cm", "z")}
    kw = dict(D=s["D"], dt_bias=s["dt_bias"])
    s1, s2 = s["state"].clone(), s["state"].clone()
    whole = cg.scan_prefill(v["x"], v["dt"], s["A_log"], v["Bm"], v["Cm"], s1, z=v["z"], **kw)
    parts = [cg.scan_prefill(v["x"][:, :70], v["dt"][:, :70], s["A_log"], v["Bm"][:, :70], v["Cm"][:, :70], s2,
                             z=v["z"][:, :70], **kw)]
    for t in range(70, T):
        parts.append(cg.scan_decode(v["x"][:, t], v["dt"][:, t], s["A_log"], v["Bm"][:, t], v["Cm"][:, t], s2,
                                    z=v["z"][:, t], **kw)[:, None])
    close(torch.cat(parts, 1), whole.cpu(), 1e-4 * rms(whole.double().cpu()))
    close(s2, s1.cpu(), 1e-4 * rms(s1.double().cpu()))


# ------------------------------------------------------------------------------------ cache plan


def run_plan(seq, new, page, width, free, n_tokens, count=None, num_pages=None):
    B = len(seq)
    table = [[1000 + 50 * b + k if k < -(-seq[b] // page) else -1 for k in range(width)] for b in range(B)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    t = i32(table).view(B, width)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    count = len(free) if count is None else count
    p = cg.cache_plan(t, i32(seq), i32(new), i32(free), i32([count]), n_tokens, page, status=status, num_pages=num_pages)
    before = [list(r) for r in table]
    want = ref.plan(table, seq, new, free, count, n_tokens, page)
    return p, t, int(status), want, table if want is not None else before


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("seq,new,extra", [
    ([0], [1], 0), ([0], [0], 3), ([15, 16, 17], [1, 1, 1], 0), ([0, 0, 5, 128], [300, 0, 128, 1], 7),
    (list(range(0, 600, 2)), [i % 3 for i in range(300)], 11), ([100] * 3, [2500, 0, 1], 0)])
def test_plan(page, seq, new, extra):
    width = max(-(-(s + a) // page) for s, a in zip(seq, new)) + 1
    need = sum(-(-(s + a) // page) - -(-s // page) for s, a in zip(seq, new))
    free = [7 * k + 3 for k in range(need + 2)]
    p, t, status, want, table = run_plan(seq, new, page, width, free, sum(new) + extra)
    assert status == cg.OK
    assert p.slots.tolist() == want["slots"] and p.requests.tolist() == want["requests"]
    assert p.positions.tolist() == want["positions"] and p.cu_seqlens.tolist() == want["cu"]
    assert p.kv_lens.tolist() == want["kv"] and p.free_count.tolist() == [want["count"]]
    assert t.tolist() == table


@pytest.mark.parametrize("kw,code", [
    (dict(seq=[5, 60], new=[1, 8], page=16, width=8, free=[], n_tokens=9), cg.ERR_CAPACITY),       # no free page
    (dict(seq=[5, 60], new=[1, 80], page=16, width=8, free=[1] * 9, n_tokens=81), cg.ERR_CAPACITY),  # a row too narrow
    (dict(seq=[5, 60], new=[1, 8], page=16, width=8, free=[1, 2], n_tokens=8), cg.ERR_CAPACITY),   # outputs too short
    (dict(seq=[5, 60], new=[1, 2 ** 31 - 1], page=16, width=8, free=[1, 2], n_tokens=8), cg.ERR_CAPACITY),
    (dict(seq=[5, 60], new=[1, -1], page=16, width=8, free=[1, 2], n_tokens=8), cg.ERR_INVALID_ARG),
    (dict(seq=[5, -3], new=[1, 1], page=16, width=8, free=[1, 2], n_tokens=8), cg.ERR_INVALID_ARG),
    (dict(seq=[5, 64], new=[1, 1], page=16, width=8, free=[9], n_tokens=2, num_pages=9), cg.ERR_INVALID_ARG),
    (dict(seq=[5, 64], new=[1, 1], page=16, width=8, free=[9], n_tokens=2, count=2), cg.ERR_INVALID_ARG),
])
def test_plan_takes_all_or_nothing(kw, code):
    seq, count = kw["seq"], kw.get("count", len(kw["free"]))
    B, width = len(seq), kw["width"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    before, status = table.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    p = cg.cache_plan(table, i32(seq), i32(kw["new"]), i32(kw["free"]), i32([count]), kw["n_tokens"], kw["page"],
                      status=status, num_pages=kw.get("num_pages"))
    assert int(status) == code and torch.equal(table, before)
    assert p.kv_lens.tolist() == seq and p.free_count.tolist() == [count] and not p.cu_seqlens.any()
    for t in (p.slots, p.requests, p.positions):
        assert t.tolist() == [-1] * kw["n_tokens"]


def test_plan_many_requests_and_no_request():
    g = torch.Generator().manual_seed(1)
    seq = torch.randint(0, 200, (8192,), generator=g).tolist()
    new = torch.randint(0, 4, (8192,), generator=g).tolist()
    p, t, status, want, table = run_plan(seq, new, 16, 14, list(range(8192)), sum(new) + 1)
    assert status == cg.OK and p.slots.tolist() == want["slots"] and t.tolist() == table
    assert p.cu_seqlens.tolist() == want["cu"] and p.free_count.tolist() == [want["count"]]
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    p = cg.cache_plan(z.view(0, 4), z, z, z, torch.zeros(1, dtype=torch.int32, device=DEV), 3, 16)
    assert p.slots.tolist() == [-1] * 3 and p.cu_seqlens.tolist() == [0] and p.free_count.tolist() == [0]


# ------------------------------------------------------------------------------------ append


def random_cache(g, pages, Hkv, page, D, lo=0.01):
    c = lambda: torch.randint(-127, 128, (pages, Hkv, page, D), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    s = lambda: (torch.rand(pages, Hkv, generator=g, device=DEV) + 0.5) * lo
    return c(), c(), s(), s()


def slots_for(tables, starts, news, page):
    return [t[p // page] * page + p % page for t, s, a in zip(tables, starts, news) for p in range(s, s + a)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,Hkv,page", [(128, 2, 64), (64, 3, 16), (32, 1, 128)])
@pytest.mark.parametrize("spread", [0.1, 10.0])                          # scales that stay, scales that grow
@pytest.mark.parametrize("starts,news", [([0], [1]), ([5, 0, 63], [1, 1, 1]), ([10, 0, 100], [150, 300, 0]), ([15, 17], [2, 128])])
def test_append(dtype, D, Hkv, page, spread, starts, news):
    g = gen(D + page + sum(news))
    tables, nxt = [], 1
    for s, a in zip(starts, news):
        k = -(-(s + a) // page)
        tables.append(list(range(nxt + k - 1, nxt - 1, -1)))
        nxt += k
    n = sum(news)
    kc, vc, ks, vs = random_cache(g, nxt + 1, Hkv, page, D)
    k = (randn(g, n, Hkv + 1, D) * spread).to(dtype)[:, 1:]
    v = (randn(g, n, Hkv, D) * spread).to(dtype)
    slots = torch.tensor(slots_for(tables, starts, news, page) + [-1], device=DEV)
    k, v = torch.cat([k, k[:1]]), torch.cat([v, v[:1]])                   # a padding token
    want = ref.append(k, slots, kc, ks) + ref.append(v, slots, vc, vs)
    cg.cache_append(k, v, slots, kc, vc, ks, vs)
    for got, w in zip((kc, ks, vc, vs), want):
        assert torch.equal(got.cpu(), w)


def test_append_zeros_out_of_range_slots_and_non_finite_values():
    g = gen(2)
    kc, vc, ks, vs = random_cache(g, 4, 1, 16, 32)
    old = kc.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.zeros(3, 1, 32, device=DEV)
    slots = torch.tensor([16, 64, 1 << 40], device=DEV)                   # the second and third lie outside
    cg.cache_append(k, k, slots, kc, vc, ks, vs, status=status)
    assert int(status) == cg.ERR_BOUNDS and float(ks[1, 0]) == 0 and not kc[1, 0, 0].any()
    old[1, 0, 0] = 0
    assert torch.equal(kc, old)
    k[0, 0, 3] = float("nan")
    cg.cache_append(k[:1], k[1:2], slots[:1], kc, vc, ks, vs)
    assert torch.isnan(ks[1, 0]) and not torch.isnan(ks[0, 0])


# ------------------------------------------------------------------------------------ attention


def attend_case(seed, q_lens, kv_lens, Hq, Hkv, D, page, dtype, spare=3):
    g = gen(seed)
    counts = [-(-max(k, 0) // page) for k in kv_lens]
    pool, width = sum(counts) + spare, max(counts + [1]) + 1
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(kv_lens), width), -7, dtype=torch.int32, device=DEV)     # never read past the pages
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    kc, vc, ks, vs = random_cache(g, pool, Hkv, page, D, 0.02)
    q = (randn(g, sum(q_lens), Hq, D) * 1.5).to(dtype)
    return q, kc, vc, ks, vs, table, torch.tensor(kv_lens, dtype=torch.int32, device=DEV), offsets(q_lens)


def check_attend(case, dtype, scale=None, **kw):
    q, kc, vc, ks, vs, table, kv, cu = case
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = (cu[1:] - cu[:-1]).tolist()
    kw = dict(max_q=max(lens), max_kv=max(int(kv.max()), 0), **kw)
    o = cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, status=status, scale=scale, **kw)
    want, size = ref.attend(q, kc, vc, ks, vs, table, kv.tolist(), ref.spans_of(0, 0, cu), scale)
    assert int(status) == cg.OK
    close(o, want, size * (2.0 ** -10 if dtype == BF else 3e-5), dtype)
    return o


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 128), (64, 32), (32, 16)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (32, 1)])
def test_attend_single_tokens(dtype, D, page, Hq, Hkv):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 300]
    check_attend(attend_case(D + page, [1] * len(kv), kv, Hq, Hkv, D, page, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 1, 0, 5], [3, 9, 40, 200]), ([2, 8], [1, 4]), ([33, 70], [40, 71]),
                                            ([150, 1], [150, 20])])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 1, 64), (2, 2, 32)])
def test_attend_several_tokens(dtype, q_lens, kv_lens, Hq, Hkv, D):
    """Causal rows, empty requests, and more query tokens than cached ones (rows that see nothing are zero)."""
    case = attend_case(sum(q_lens), q_lens, kv_lens, Hq, Hkv, D, 16, dtype)
    o = check_attend(case, dtype)
    at = 0
    for ql, kv in zip(q_lens, kv_lens):
        blind = max(0, ql - kv)
        assert not o[at:at + blind].any()
        at += ql


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,page", [
    ([1], [1], 1, 1, 16), ([70], [70], 1, 1, 64), ([33, 0, 70], [40, 9, 71], 4, 2, 16), ([300], [1000], 2, 1, 128),
    ([130, 5, 1], [130, 600, 350], 3, 1, 32), ([150, 1], [150, 20], 4, 2, 64), ([200, 3], [50, 0], 2, 2, 16),
    ([65, 129], [127, 193], 2, 1, 64), ([90], [4097], 8, 1, 16)])
def test_attend_tiles(q_lens, kv_lens, Hq, Hkv, page):
    """The tensor-memory kernel: one and two row tiles, ragged ends, pages smaller and larger than a step, blind rows."""
    case = attend_case(sum(q_lens) + page, q_lens, kv_lens, Hq, Hkv, 128, page, BF)
    o = check_attend(case, BF, path=cg.ATTEND_TILES)
    at = 0
    for ql, kv in zip(q_lens, kv_lens):
        assert not o[at:at + max(0, ql - kv)].any()
        at += ql
    other = cg.cache_attend(*case, max_q=max(q_lens), path=cg.ATTEND_ROWS)
    close(other, o.cpu(), float(o.float().abs().max()) * 2.0 ** -8, BF)


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,page", [
    ([70], [3001], 4, 1, 64), ([9, 0, 33], [1500, 700, 2049], 16, 2, 16), ([129, 2], [600, 4000], 2, 2, 128)])
def test_attend_tiles_over_a_cache_in_parts(q_lens, kv_lens, Hq, Hkv, page):
    sizes = (len(q_lens), sum(q_lens), Hq, Hkv, 128, page, -(-max(kv_lens) // page) + 1)
    assert cg.cache_attend_workspace_size(*sizes, max_q=max(q_lens), max_kv=max(kv_lens), path=cg.ATTEND_TILES) > 0
    check_attend(attend_case(sum(q_lens) + page, q_lens, kv_lens, Hq, Hkv, 128, page, BF), BF, path=cg.ATTEND_TILES)


def test_attend_tiles_a_wait_that_gives_up():
    """The test hook: every block's first wait runs out, the status says so, and the next call is as if nothing had been."""
    case = attend_case(7, [150, 20], [700, 300], 4, 2, 128, 64, BF)
    q, kc, vc, ks, vs, table, kv, cu = case
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, max_q=150, max_kv=700, path=cg.ATTEND_TILES, status=status, wait_polls=-4)
    torch.cuda.synchronize()
    assert int(status) == cg.ERR_TIMEOUT
    check_attend(case, BF, path=cg.ATTEND_TILES)


def test_attend_tiles_reports_what_it_cuts_off():
    q, kc, vc, ks, vs, table, kv, cu = attend_case(13, [1, 40], [100, 200], 2, 1, 128, 16, BF)
    for kw in (dict(max_q=40, max_kv=150), dict(max_q=39, max_kv=200)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, path=cg.ATTEND_TILES, status=status, **kw)
        assert int(status) == cg.ERR_CAPACITY


def test_attend_tiles_scales_and_non_finite_values():
    """Scales of many magnitudes, zeros, pages outside the cache, NaN scales that no row sees, a NaN query row."""
    case = list(attend_case(40, [140], [333], 2, 1, 128, 16, BF))
    q, kc, vc, ks, vs, table, kv, cu = case
    vs *= 10.0 ** torch.linspace(-12, 3, vs.numel(), device=DEV).view_as(vs)
    vs[3], vs[7] = 0, 0
    ks[5] = 0
    first = check_attend(tuple(case), BF, path=cg.ATTEND_TILES)
    used = set(table[table >= 0].tolist())
    for p in set(range(kc.shape[0])) - used:
        ks[p], vs[p] = float("nan"), float("inf")
    q[7, 1] = float("nan")
    again = cg.cache_attend(*case, max_q=140, path=cg.ATTEND_TILES)
    assert torch.isnan(again[7, 1]).all()
    again[7, 1] = first[7, 1]
    assert torch.equal(again, first)
    bad, status = table.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    bad[0, 2], bad[0, 9] = -3, kc.shape[0]
    o = cg.cache_attend(q, kc, vc, ks, vs, bad, kv, cu, max_q=140, path=cg.ATTEND_TILES, status=status)
    assert int(status) == cg.ERR_BOUNDS
    rows = cg.cache_attend(q, kc, vc, ks, vs, bad, kv, cu, max_q=140, path=cg.ATTEND_ROWS)
    ok = torch.ones_like(o, dtype=torch.bool)
    ok[7, 1] = False
    close(o[ok], rows[ok].cpu(), float(rows[ok].float().abs().max()) * 2.0 ** -8, BF)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attend_long_cache_is_split_and_joined(dtype):
    check_attend(attend_case(5, [1, 1], [6000, 4097], 4, 2, 64, 16, dtype), dtype)
    check_attend(attend_case(6, [3, 2], [2500, 700], 2, 1, 128, 128, dtype), dtype, scale=0.3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 2, 128, 64), (16, 1, 64, 16), (6, 3, 32, 128), (16, 2, 128, 16)])
def test_attend_units_of_unequal_lengths_share_the_blocks(dtype, Hq, Hkv, D, page):
    q_lens, kv_lens = [1, 2, 0, 5, 1, 1], [1100, 0, 40, 1537, 130, 1025]
    check_attend(attend_case(17, q_lens, kv_lens, Hq, Hkv, D, page, dtype), dtype)


def test_attend_one_prompt_among_many_single_tokens():
    q_lens = [1] * 20 + [600] + [0, 1] * 10
    kv_lens = [(37 * i) % 300 for i in range(20)] + [700] + [5, 129] * 10
    check_attend(attend_case(18, q_lens, kv_lens, 8, 2, 64, 32, F32), F32)


def test_attend_empty_cache_gives_zeros():
    case = attend_case(1, [1, 2], [0, 0], 2, 1, 64, 16, BF)
    assert not check_attend(case, BF).any()


def test_attend_extreme_scales():
    """Scales of many magnitudes in one request, zero among them, and large and tiny queries."""
    case = list(attend_case(8, [1, 4], [500, 90], 4, 1, 64, 16, F32))
    q, ks, vs = case[0], case[3], case[4]
    vs *= 10.0 ** torch.linspace(-12, 3, vs.numel(), device=DEV).view_as(vs)
    vs[3], vs[7] = 0, 0
    ks[5] = 0
    q[1] *= 1e-20
    q[2] *= 3.0
    check_attend(tuple(case), F32)


def test_attend_ignores_what_no_row_sees():
    """Non-finite scales on pages outside the tables, and whatever stands behind a request's last token."""
    case = list(attend_case(12, [1, 3], [70, 33], 4, 2, 128, 32, BF))
    q, kc, vc, ks, vs, table, kv, cu = case
    used = set(table[table >= 0].tolist())
    out1 = check_attend(tuple(case), BF)
    for p in set(range(kc.shape[0])) - used:
        ks[p], vs[p] = float("nan"), float("inf")
    kc[table[0, 2].item(), :, 70 - 64:] = 127
    vc[table[0, 2].item(), :, 70 - 64:] = -127
    out2 = check_attend(tuple(case), BF)
    assert torch.equal(out1, out2)
    # a NaN query spoils its own rows only
    q[1, 2] = float("nan")
    out3 = cg.cache_attend(*case[:5], table, kv, cu, max_q=3)
    assert torch.isnan(out3[1, 2]).all()
    keep = torch.ones_like(out3, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out3[keep], out1[keep])


def test_attend_reports_bad_pages_and_lengths():
    q, kc, vc, ks, vs, table, kv, cu = attend_case(13, [1, 2], [100, 50], 2, 1, 64, 16, F32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, max_q=2, status=status)
    bad = table.clone()
    bad[0, 1], bad[1, 0] = kc.shape[0], -5
    cg.cache_attend(q, kc, vc, ks, vs, bad, kv, cu, max_q=2, status=status)
    assert int(status) == cg.ERR_BOUNDS
    status.zero_()
    o = cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, max_q=2, max_kv=60, status=status)
    assert int(status) == cg.ERR_CAPACITY and torch.equal(o[1:], good[1:])
    assert torch.isfinite(o).all()


# ------------------------------------------------------------------------------------ streams, graphs


def test_calls_on_another_stream_and_in_a_graph():
    g = gen(20)
    case = attend_case(21, [1, 1], [3000, 200], 4, 2, 128, 64, BF)
    s = scan_inputs(g, 300, 1, 24, 16, 1, F32, True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = cg.cache_attend(*case, max_q=1, stream=side)
    y = cg.scan_prefill(s["x"][None], s["dt"][None], s["A_log"], s["Bm"][None], s["Cm"][None], s["state"].clone(),
                        dt_bias=s["dt_bias"], stream=side)
    side.synchronize()
    assert torch.equal(o, cg.cache_attend(*case, max_q=1))
    assert torch.equal(y, cg.scan_prefill(s["x"][None], s["dt"][None], s["A_log"], s["Bm"][None], s["Cm"][None],
                                          s["state"].clone(), dt_bias=s["dt_bias"]))
    out = torch.empty_like(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cg.cache_attend(*case[:-1], case[-1], out, max_q=1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o)


def test_results_do_not_change_from_run_to_run():
    case = attend_case(30, [1, 5, 1], [5000, 900, 17], 8, 2, 128, 16, BF)
    first = cg.cache_attend(*case, max_q=5)
    for _ in range(5):
        assert torch.equal(cg.cache_attend(*case, max_q=5), first)
