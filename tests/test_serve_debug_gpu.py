"""The serving operators through the index-checking build: no check fires, and the results are the release build's."""
import ctypes

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import build as cbuild
from gated_delta_rule_channelwise_gb300 import serve

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def checked():
    cbuild.build_all()
    L = ctypes.CDLL(cbuild.LIB_DEBUG)
    for name, res, args in serve.SIGNATURES:
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


def both(monkeypatch, checked, call):
    """call(status) with the release library, then with the checked one."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = call(status)
    with monkeypatch.context() as m:
        m.setattr(serve, "lib", lambda: checked)
        got = call(status)
    torch.cuda.synchronize()
    assert int(status) == cg.OK
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def rand(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_conv_and_scan(monkeypatch, checked, dtype):
    lens, C, N = [1, 0, 70, 3], 72, 32
    cu = torch.tensor([0, 1, 1, 71, 74], dtype=torch.int32, device=DEV)
    x, w = rand(74, C + 8, dtype=dtype)[:, 8:], rand(C, 4, seed=1)

    def conv(status):
        state = rand(len(lens), 3, C, dtype=dtype, seed=2)
        return cg.conv_prefill(x, w, state, cu_seqlens=cu, status=status), state

    def conv_step(status):
        state = rand(74, 3, C, dtype=dtype, seed=2)
        return cg.conv_decode(x, w, state, status=status), state

    A, D = rand(C, N, seed=3), rand(C, seed=4)
    Bm, Cm, dt = rand(74, 1, N, dtype=dtype, seed=5), rand(74, 1, N, dtype=dtype, seed=6), rand(74, C, dtype=dtype, seed=7)

    def scan(status):
        state = rand(len(lens), C, N, seed=8)
        return cg.scan_prefill(x, dt, A, Bm, Cm, state, D=D, z=x, cu_seqlens=cu, status=status), state

    def scan_step(status):
        state = rand(74, C, N, seed=8)
        return cg.scan_decode(x, dt, A, Bm, Cm, state, D=D, z=x, status=status), state

    def scan_dense(status):
        state = rand(2, C, N, seed=8)
        d = lambda t: t.unflatten(0, (2, 37))
        return cg.scan_prefill(d(x), d(dt), A, d(Bm), d(Cm), state, D=D, status=status), state

    for call in (conv, conv_step, scan, scan_step, scan_dense):
        both(monkeypatch, checked, call)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("old,new", [([0, 5, 130], [1, 1, 1]), ([3, 0, 100], [140, 0, 61]), ([2000, 1], [2, 0])])
def test_plan_append_attend(monkeypatch, checked, dtype, D, old, new):
    B, page, width, pages, n = len(old), 16, 160, 400, sum(new)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)

    def call(status, path=cg.ATTEND_AUTO):
        table, taken = torch.full((B, width), -1, dtype=torch.int32, device=DEV), 0
        for b, m in enumerate(old):
            held = -(-m // page)
            table[b, :held] = torch.arange(taken, taken + held, device=DEV, dtype=torch.int32)
            taken += held
        free = torch.arange(pages - 1, taken - 1, -1, device=DEV, dtype=torch.int32)
        p = cg.cache_plan(table, ints(old), ints(new), free, ints([free.numel()]), n + 3, page, num_pages=pages, status=status)
        g = torch.Generator(device=DEV).manual_seed(1)
        kc, vc = (torch.randint(-127, 128, (pages, 2, page, D), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
                  for _ in range(2))
        ks, vs = rand(pages, 2, seed=3).abs() * 0.01 + 0.01, rand(pages, 2, seed=4).abs() * 0.01 + 0.01
        k, v = rand(n + 3, 2, D, dtype=dtype, seed=5), rand(n + 3, 2, D, dtype=dtype, seed=6)
        cg.cache_append(k, v, p.slots, kc, vc, ks, vs, status=status)
        o = cg.cache_attend(rand(n + 3, 8, D, dtype=dtype, seed=7)[:n], kc, vc, ks, vs, table, p.kv_lens, p.cu_seqlens,
                            max_q=max(new), max_kv=max(old) + max(new), path=path, status=status)
        return o, kc, vc, ks, vs, table, p.slots, p.kv_lens, p.free_count

    both(monkeypatch, checked, call)
    both(monkeypatch, checked, lambda status: call(status, cg.ATTEND_TILES))
