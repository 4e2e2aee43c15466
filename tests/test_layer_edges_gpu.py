"""The operators around a layer's state where sizes, strides and callers are unusual.  Tolerances as in test_layer_gpu.py."""
import threading

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
import layer_ref as ref
from test_layer_gpu import BF, E4M3, F32, PATHS, U, check_matmul, near, operands, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def far_rows(t, step):
    """A copy of [n, C] whose rows are ``step`` values apart in memory."""
    n, C = t.shape
    buffer = torch.empty((n - 1) * step + C, dtype=t.dtype, device="cuda")
    wide = buffer.as_strided((n, C), (step, 1))
    wide.view(torch.uint8).copy_(t.view(torch.uint8)) if t.dtype == E4M3 else wide.copy_(t)
    return wide


FAR = (1 << 30) + 128                                  # three rows: past 2^31 values


def test_rows_farther_apart_than_32_bits():
    x, w = rand(1, 3, 256, dtype=BF), 1 + 0.1 * rand(2, 256)
    want, r0 = cg.rms_norm(x, w), rand(3, 3, 256, dtype=BF)
    far, o = far_rows(x, FAR), far_rows(torch.zeros_like(x), FAR)
    assert torch.equal(cg.rms_norm(far, w, o), want) and torch.equal(o, want)
    r, rfar = r0.clone(), far_rows(r0, FAR)
    want = cg.rms_norm(x, w, residual=r)
    assert torch.equal(cg.rms_norm(far, w, residual=rfar), want) and torch.equal(rfar, r)
    for call in (cg.fp8_quantize, cg.fp8_quantize_weight):
        (a, s), (b, t) = call(x), call(far)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(s, t)
    del o, rfar
    pos, (freq, _) = torch.tensor([3, 1 << 20, 7], dtype=torch.int32, device="cuda"), cg.rotary_frequencies(128)
    near_by = x.clone().unflatten(1, (2, 128))
    cg.rotary(near_by, None, pos, freq)
    cg.rotary(far.unflatten(1, (2, 128)), None, pos, freq)
    assert torch.equal(far, near_by.flatten(1))


@pytest.mark.parametrize("path", PATHS[:2])
def test_product_of_rows_farther_apart_than_32_bits(path):
    x, xs, w, ws = operands(4, 3, 136, 256)
    want = cg.fp8_matmul(x, xs, w, ws, path=path)
    o = far_rows(torch.zeros_like(want), FAR)
    cg.fp8_matmul(far_rows(x, FAR), xs, w, ws, o, path=path)
    assert torch.equal(o, want)


@pytest.mark.parametrize("path", PATHS[:2])
@pytest.mark.parametrize("n,N,K", [(3, 40, 16), (70, 200, 130), (130, 257, 400)])
def test_product_of_operands_between_nan(path, n, N, K):
    """e4m3's NaN before and behind every row, and before and behind all rows: none of it is read into a result."""
    x, xs, w, ws = operands(7, n, N, K)

    def among(t):
        rows, cols = t.shape
        wide = torch.full((rows + 4, (cols + 15) // 16 * 16 + 32), 0x7F, dtype=torch.uint8, device="cuda")
        wide[2:-2, 16:16 + cols] = t.contiguous().view(torch.uint8)
        return wide.view(E4M3)[2:-2, 16:16 + cols]

    check_matmul(x, xs, w, ws, cg.fp8_matmul(among(x), xs, among(w), ws, dtype=F32, path=path), F32)


@pytest.mark.parametrize("n,H,C", [(300000, 1, 8), (70000, 3, 16), (100, 2000, 24)])
def test_norm_of_many_short_rows(n, H, C):
    x = rand(8, n, H, C)
    want, _ = ref.norm(x, None)
    near(cg.rms_norm(x, None), want, 40 * U * want.abs(), F32)


@pytest.mark.parametrize("n,H,R", [(100000, 1, 8), (3, 3000, 32)])
def test_rotary_of_many_tokens_and_heads(n, H, R):
    q, pos, (freq, _) = rand(9, n, H, R), torch.arange(n, dtype=torch.int32, device="cuda"), cg.rotary_frequencies(R)
    want, size = ref.rotary(q, pos, freq, False, 1.0)
    cg.rotary(q, None, pos, freq)
    near(q, want, 6 * U * size, F32)


def test_quantize_many_rows():
    x = rand(10, 70001, 136)
    y, s = cg.fp8_quantize(x)
    want, ws = ref.quantize(x, 1)
    assert torch.equal(s.cpu(), ws) and torch.equal(y.cpu().view(torch.uint8), want.view(torch.uint8))


def test_product_of_many_rows_and_few_columns():
    """More tiles of rows than CTAs, one tile of columns, and the other way round."""
    for n, N in ((40000, 24), (5, 40000)):
        x, xs, w, ws = operands(11, n, N, 272)
        for path in PATHS:
            o = cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path)
            rows = torch.arange(0, n, max(1, n // 300), device="cuda")
            check_matmul(x[rows], xs[rows], w, ws, o[rows], F32)


def test_calls_of_two_threads_on_two_streams():
    cases = [operands(20 + i, n, 520, 1024) for i, n in enumerate((9, 200))]
    want = [cg.fp8_matmul(*c, dtype=F32) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(50):
                if not torch.equal(cg.fp8_matmul(*cases[i], dtype=F32), want[i]):
                    wrong.append(i)
        side.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_two_graphs_side_by_side():
    """Nothing is shared between captured calls: two graphs of different inputs replayed on two streams at once."""
    sides, graphs, outs, wants = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for i, n in enumerate((40, 300)):
        x, xs, w, ws = operands(30 + i, n, 640, 2048)
        wants.append(cg.fp8_matmul(x, xs, w, ws))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append([cg.fp8_matmul(x, xs, w, ws) for _ in range(4)])
    for _ in range(5):
        for side, graph in zip(sides, graphs):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert all(torch.equal(o, want) for o in out)


def test_results_are_there_for_what_follows():
    """Chains of short calls, each reading what the one before has just written, give the same every time."""
    w, ws = cg.fp8_quantize_weight(rand(40, 256, 256, size=0.1))
    x0 = rand(41, 33, 256, dtype=BF)

    def chain():
        x = x0
        for _ in range(20):
            y, s = cg.rms_norm_fp8(x, None)
            x = cg.fp8_matmul(y, s, w, ws)
        return x

    first = chain()
    assert all(torch.equal(chain(), first) for _ in range(20))


def test_given_outputs_and_refusals():
    x = rand(42, 5, 264)
    y, s = torch.empty(5, 272, dtype=torch.uint8, device="cuda").view(E4M3)[:, :264], torch.empty(5, 3, device="cuda")
    got = cg.fp8_quantize(x, y, s)
    assert got[0] is y and got[1] is s and torch.equal(y.float(), cg.fp8_quantize(x)[0].float())
    with pytest.raises(cg.CgdrError, match="ALIGNMENT"):              # rows of 264 bytes
        cg.fp8_quantize(x, torch.empty(5, 264, dtype=E4M3, device="cuda"), s)
    with pytest.raises(cg.CgdrError, match="INVALID"):                # a broadcast output
        cg.rms_norm(x, None, torch.empty(264, device="cuda").expand(5, 264))
    with pytest.raises(cg.CgdrError, match="INVALID"):
        cg.rotary(rand(1, 4, 1, 64).expand(4, 3, 64), None, torch.zeros(4, dtype=torch.int32, device="cuda"), cg.rotary_frequencies(64)[0])
    with pytest.raises(TypeError, match="residual"):
        cg.rms_norm(x, None, residual=x.to(BF))
    with pytest.raises(ValueError, match="w_scale must have shape"):
        cg.fp8_matmul(*cg.fp8_quantize(x), *[cg.fp8_quantize_weight(rand(43, 200, 264))[0], s])
    with pytest.raises(ValueError, match="innermost"):
        cg.rms_norm(rand(44, 64, 8).t(), None)
    with pytest.raises(TypeError, match="float64"):
        cg.rotary(rand(1, 4, 1, 64), None, torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"))


def test_one_token_of_any_stride():
    """The strides of a dimension of size 1 say nothing: a row made of a column is a row."""
    def row(t):                                       # the same values, with the strides of a transposed column
        assert t.shape[0] == 1
        r = t.reshape(-1, 1).clone().t()
        assert r.stride() == (1, 1)
        return r

    x, w = rand(71, 1, 264, dtype=BF), 1 + 0.1 * rand(72, 264)
    assert torch.equal(cg.rms_norm(row(x), w), cg.rms_norm(x, w))
    r, s = row(x), x.clone()
    o = row(torch.zeros_like(x))
    cg.rms_norm(row(x), w, o, residual=r)
    assert torch.equal(o, cg.rms_norm(x, w, residual=s)) and torch.equal(r, s)
    for call in (cg.fp8_quantize, cg.fp8_quantize_weight):
        (a, s), (b, t) = call(x), call(row(x))
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(s, t)
    x8, xs = cg.fp8_quantize(x)
    narrow = row(x8.view(torch.uint8)).view(E4M3)
    for path in PATHS:
        want = cg.fp8_matmul(x8, xs, x8, xs, path=path)
        assert torch.equal(cg.fp8_matmul(narrow, xs, narrow, xs, path=path), want)
    pos, (freq, _) = torch.tensor([12345], dtype=torch.int32, device="cuda"), cg.rotary_frequencies(64)
    q = x[:, :256].reshape(1, 4, 64).clone()
    odd = torch.empty_strided((1, 4, 64), (7, 64, 1), dtype=BF, device="cuda").copy_(q)
    cg.rotary(q, None, pos, freq)
    cg.rotary(odd, None, pos, freq)
    assert torch.equal(odd, q)
    one = torch.empty_strided((5, 1, 64), (64, 3, 1), dtype=BF, device="cuda").copy_(rand(74, 5, 1, 64, dtype=BF))
    assert torch.equal(cg.rms_norm(one, None), cg.rms_norm(one.reshape(5, 1, 64).contiguous(), None))
