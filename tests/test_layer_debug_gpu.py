"""The operators around a layer's state through the index-checking build: no check fires, and the results are the release build's."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import layer
from test_serve_debug_gpu import checked, rand  # noqa: F401 (checked is a fixture)

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def both(monkeypatch, checked, call):  # noqa: F811
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(status)
    with monkeypatch.context() as m:
        m.setattr(layer, "lib", lambda: checked)
        got = call(status)
    torch.cuda.synchronize()
    assert int(status) == cg.OK
    bits = lambda t: t.contiguous().view(torch.uint8)
    for a, b in zip(want, got):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,H,C", [(1, 1, 8), (33, 3, 136), (5, 1, 4096), (3, 1, 9000), (2, 1, 32768)])
def test_norm(monkeypatch, checked, dtype, n, H, C):  # noqa: F811
    x, w = rand(n, (H + 1) * C, dtype=dtype)[:, C:].unflatten(1, (H, C)), rand(C, seed=1)

    def norm(status):
        r = rand(n, H, C, dtype=dtype, seed=2)
        return cg.rms_norm(x, w, residual=r, status=status), r

    def norm8(status):
        r = rand(n, C, dtype=dtype, seed=2)
        return *cg.rms_norm_fp8(x[:, 0], w, residual=r, status=status), r

    both(monkeypatch, checked, norm)
    both(monkeypatch, checked, norm8)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,K,N", [(1, 16, 8), (7, 200, 130), (70, 1024, 257), (260, 600, 1003)])
def test_quantize_and_matmul(monkeypatch, checked, dtype, n, K, N):  # noqa: F811
    x, w = rand(n, K + 8, dtype=dtype)[:, 8:], rand(N, K, dtype=dtype, seed=1)
    for path in (cg.MATMUL_AUTO, cg.MATMUL_FEW, cg.MATMUL_TILES):
        def call(status, path=path):
            y, ys = cg.fp8_quantize(x, status=status)
            v, vs = cg.fp8_quantize_weight(w, status=status)
            return y, ys, v, vs, cg.fp8_matmul(y, ys, v, vs, dtype=dtype, path=path, status=status)

        both(monkeypatch, checked, call)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,D,half", [(1, 1, 8, 1), (700, 5, 96, 24), (9, 40, 128, 64), (3, 2, 512, 256)])
def test_rotary(monkeypatch, checked, dtype, interleaved, n, H, D, half):  # noqa: F811
    pos, freq = torch.arange(n, device="cuda", dtype=torch.int32) * 77 - 77, cg.rotary_frequencies(2 * half)[0]

    def call(status):
        row = rand(n, (H + 3) * D, dtype=dtype)
        cg.rotary(row[:, :H * D].unflatten(1, (H, D)), row[:, H * D:(H + 2) * D].unflatten(1, (2, D)), pos, freq, interleaved=interleaved, status=status)
        return row,

    both(monkeypatch, checked, call)
