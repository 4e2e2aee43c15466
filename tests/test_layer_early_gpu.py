"""Inputs that the kernel directly before a call has written: every operator around a layer's state, every input, call after call.

The kernels of these calls may be set up while the one before them ends, so each input in turn is rewritten directly before the
call, with other values every time, on the stream and in a graph.
"""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from test_layer_gpu import BF, E4M3, F32, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def norm(n):
    x, r, w = [rand(i, n, 4096, dtype=BF) for i in (1, 2)], [rand(i, n, 4096, dtype=BF) for i in (3, 4)], [rand(i, 4096) for i in (5, 6)]
    return dict(x=x, r=r, w=w), lambda x, r, w: (cg.rms_norm(x, w, residual=r), r)


def norm8(n):
    inputs, _ = norm(n)
    return inputs, lambda x, r, w: (*cg.rms_norm_fp8(x, w, residual=r), r)


def rows(n):
    return dict(x=[rand(i, n, 1024) for i in (1, 2)]), lambda x: cg.fp8_quantize(x)


def blocks(n):
    return dict(x=[rand(i, n, 1024) for i in (1, 2)]), lambda x: cg.fp8_quantize_weight(x)


def product(path):
    def make(n):
        x, w = [cg.fp8_quantize(rand(i, n, 1024)) for i in (1, 2)], [cg.fp8_quantize_weight(rand(i, 1000, 1024)) for i in (3, 4)]
        x[1][1].mul_(3), w[1][1].mul_(5)
        parts = lambda t, i: [p[i] for p in t]
        return dict(x=parts(x, 0), xs=parts(x, 1), w=parts(w, 0), ws=parts(w, 1)), lambda x, xs, w, ws: (cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path),)
    return make


def rotary(n):
    q, k = [rand(i, n, 8, 128, dtype=BF) for i in (1, 2)], [rand(i, n, 2, 128, dtype=BF) for i in (3, 4)]
    pos = [torch.arange(n, dtype=torch.int32, device="cuda") + i for i in (0, 1000)]
    freq = [cg.rotary_frequencies(128, base=b)[0] for b in (1e4, 1e6)]
    return dict(q=q, k=k, pos=pos, freq=freq), lambda q, k, pos, freq: cg.rotary(q, k, pos, freq)


MAKE = dict(norm=norm, norm8=norm8, rows=rows, blocks=blocks, few=product(cg.MATMUL_FEW), tiles=product(cg.MATMUL_TILES), rotary=rotary)


def same(a, b):
    return all(torch.equal(*(t.contiguous().view(torch.uint8) for t in p)) for p in zip(a, b))


@pytest.mark.parametrize("n", [1, 50, 700])
@pytest.mark.parametrize("name", MAKE)
def test_inputs_written_directly_before(name, n):
    inputs, call = MAKE[name](n)
    names = list(inputs)
    copies = lambda picks: {m: inputs[m][i].clone() for m, i in zip(names, picks)}
    raw = lambda t: t.view(torch.uint8) if t.dtype == E4M3 else t

    def want(picks):
        now = copies(picks)
        torch.cuda.synchronize()
        out = [t.clone() for t in call(**now)]
        torch.cuda.synchronize()
        return out

    # one input at a time changes, and is the last to be written
    sequence, picks = [], [0] * len(names)
    for step in range(3 * len(names)):
        turn = step % len(names)
        picks[turn] ^= 1
        sequence.append((turn, tuple(picks)))
    wants = [want(p) for _, p in sequence]

    here = copies([0] * len(names))

    def run():
        got = []
        for turn, p in sequence:
            for m in [*range(turn), *range(turn + 1, len(names)), turn]:
                raw(here[names[m]]).copy_(raw(inputs[names[m]][p[m]]))
            got.append([t.clone() for t in call(**here)])
        return got

    got = run()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, wants))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, wants))
