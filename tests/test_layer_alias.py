"""Operators around a layer's state whose outputs have an input's address: the norm's o may be x, everything else is refused.

The refusals need no GPU: the pointers are made up."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from test_layer_abi import INV, MATMUL, NORM, NORM8, P, QUANTIZE, call, lib  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("name,good,kw", [
    ("norm", NORM, dict(o=P, o_st=128)), ("norm", NORM, dict(H=2, x_sh=64, x_st=128, residual_sh=64, residual_st=128, o=P, o_sh=192, o_st=64)),
    ("norm", NORM, dict(residual=P)), ("norm", NORM, dict(residual=4 * P)), ("norm", NORM, dict(o=P, residual=P)),
    ("norm", NORM8, dict(y8=P)), ("norm", NORM8, dict(y8=2 * P)), ("quantize", QUANTIZE, dict(y8=P)), ("quantize", QUANTIZE, dict(y8=P, block_rows=128)),
    ("matmul", MATMUL, dict(o=P)), ("matmul", MATMUL, dict(o=3 * P))])
def test_refused(lib, name, good, kw):  # noqa: F811
    assert call(lib, name, good, **kw) == INV


F32, BF = torch.float32, torch.bfloat16


@pytest.fixture
def built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    return cg.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,H,C", [(1, 1, 8), (700, 1, 4096), (5000, 1, 264), (3, 1, 32768), (9, 1, 12288), (900, 12, 128), (2000, 1, 128), (50, 3, 72)])
def test_norm_in_place(built, dtype, residual, n, H, C):
    """Bit for bit what the norm gives into another tensor, heads in the middle of packed rows among them; the rest of the row stays.
    Many more rows than fit at once, so that a block asks for rows that no block has come to."""
    g = torch.Generator(device="cuda").manual_seed(80)
    row = torch.randn(n, (H + 2) * C, generator=g, device="cuda").to(dtype)
    w = torch.randn(C, generator=g, device="cuda")
    r = torch.randn(n, H, C, generator=g, device="cuda").to(dtype) if residual else None
    r2, before = r.clone() if residual else None, row.clone()
    x = row[:, C:(H + 1) * C].unflatten(1, (H, C))
    if H == 1:
        x, r, r2 = x[:, 0], r[:, 0] if residual else None, r2[:, 0] if residual else None
    want = cg.rms_norm(x, w, residual=r)
    assert cg.rms_norm(x, w, x, residual=r2) is x
    assert torch.equal(x, want) and (not residual or torch.equal(r, r2))
    assert torch.equal(row[:, :C], before[:, :C]) and torch.equal(row[:, (H + 1) * C:], before[:, (H + 1) * C:])


@pytest.mark.gpu
def test_norm_in_place_in_a_graph(built):
    x0, w = torch.randn(600, 8, 128, device="cuda").to(BF), torch.randn(128, device="cuda")
    x, want = x0.clone(), x0
    for _ in range(3):
        want = cg.rms_norm(want, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            cg.rms_norm(x, w, x)
    for _ in range(2):
        x.copy_(x0)
        graph.replay()
        assert torch.equal(x, want)


@pytest.mark.gpu
def test_python_calls_refused(built):
    x, w = torch.randn(4, 256, device="cuda"), torch.ones(256, device="cuda")
    r = torch.randn(4, 256, device="cuda")
    for o, residual in ((None, x), (r, r), (x, x)):
        with pytest.raises(cg.CgdrError, match="INVALID"):
            cg.rms_norm(x, w, o, residual=residual)
    wide = torch.randn(4, 512, device="cuda")
    with pytest.raises(cg.CgdrError, match="INVALID"):                    # the same address, other rows
        cg.rms_norm(wide[:, :256], w, wide.view(8, 256)[:4])
