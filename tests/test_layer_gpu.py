"""GPU tests of the operators around a layer's state against the plain 64-bit forms.

Tolerances, from the roundings of each operator.  A value rounded to its type is off by half a step of it,
eps/2 relative.  Norm: every fp32 step is 2^-24; a sum of squares of up to 32768 values goes through at most 32 values of a
thread, 5 shuffles and 32 warps, so it is off by 70 2^-24, its root by half of that, and four products follow: 40 2^-24.
Products: at most K/32 + K/128 + 8 additions and 3 products one after the other, each off by 2^-23 of the magnitudes that are
summed at most (the tensor core may cut where fp32 would round).  Rotary: cos and sin
by an ulp, times scale, two products and a sum: 6 2^-24 of |u| + |v|.
"""
import math

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def rand(seed, *shape, dtype=F32, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def near(got, want, off, dtype):
    """|got - want| <= off, elementwise, and the rounding to dtype; NaN and infinities in the same places."""
    got = got.detach().cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    fine = want.isfinite()
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()])
    over = (got - want).abs()[fine] - (off + half_step(dtype) * (want.abs() + off))[fine]
    assert not over.numel() or float(over.max()) <= 0


# ------------------------------------------------------------------------------------ norm


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,C", [(1, 8), (3, 64), (17, 128), (5, 136), (64, 1000), (33, 2048), (9, 4096), (4, 12288), (2, 32768), (700, 256)])
def test_norm(dtype, residual, n, C):
    x, w = rand(1, n, C + 24, dtype=dtype)[:, 24:], 1 + 0.3 * rand(2, C)
    r = rand(3, n, C + 8, dtype=dtype, size=3)[:, :C] if residual else None
    want, h = ref.norm(x, w, r)
    o = cg.rms_norm(x, w, residual=r)
    near(o, want, 40 * U * want.abs(), dtype)
    if residual:
        near(r, h, U * h.abs(), dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,H,D", [(1, 1, 128), (7, 5, 64), (40, 8, 128), (3, 2, 256), (6, 3, 72)])
def test_norm_of_heads_in_a_packed_row(dtype, n, H, D):
    row = rand(4, n, (H + 2) * D, dtype=dtype)
    x = row[:, D:(H + 1) * D].unflatten(1, (H, D))
    want, _ = ref.norm(x, None)
    out = torch.zeros(H, n, D, dtype=dtype, device="cuda")               # head-major
    assert cg.rms_norm(x, None, out.transpose(0, 1)).data_ptr() == out.data_ptr()
    near(out.transpose(0, 1), want, 40 * U * want.abs(), dtype)
    again = cg.rms_norm(x, None)
    assert again.is_contiguous() and torch.equal(again, out.transpose(0, 1))


def check_eight(y, scale, want, off):
    """y and scale against values in 64 bits that are known to ``off`` relative."""
    g = ref.groups(want, 1)
    top = g.abs().amax(3)[:, 0]
    near(scale, (top / 448).clamp(min=2.0 ** -126), (off + 2 * U) * top / 448, F32)
    s = scale.cpu().double().repeat_interleave(128, 1)[:, :want.shape[1]]
    got = y.cpu().float().double() * s
    # half a step of e4m3: 2^-4 relative, 2^-10 of the scale below its normal values; and what fp32 has lost before
    assert ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s) + (2 * off + 8 * U) * (want.abs() + s)).all()
    # the largest of each group takes the largest value
    assert (y.cpu().float().abs().amax(1) == 448).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,C", [(1, 8), (5, 128), (3, 200), (64, 4096), (2, 1000), (2, 32768), (130, 264)])
def test_norm_in_8_bits(dtype, residual, n, C):
    x, w = rand(5, n, C, dtype=dtype), 1 + 0.3 * rand(6, C)
    r = rand(7, n, C, dtype=dtype, size=2) if residual else None
    want, h = ref.norm(x, w, r)
    y, scale = cg.rms_norm_fp8(x, w, residual=r)
    check_eight(y, scale, want, 40 * U)
    if residual:
        near(r, h, U * h.abs(), dtype)


def test_norm_eps_and_zero_rows():
    x = rand(8, 4, 512, size=1e-3)
    x[1] = 0
    for eps in (1e-6, 1e-2):
        want, _ = ref.norm(x, None, eps=eps)
        o = cg.rms_norm(x, None, eps=eps)
        near(o, want, 40 * U * want.abs(), F32)
        assert not o[1].any()
    assert cg.rms_norm(x, None, eps=0.0)[1].isnan().all()                 # 0 / 0, as the formula has it
    y, scale = cg.rms_norm_fp8(x, None)
    assert not y[1].float().any() and (scale[1] == 2.0 ** -126).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_norm_keeps_what_is_not_finite_to_its_row(bad):
    x = rand(9, 6, 384, dtype=BF)
    clean = cg.rms_norm(x, None)
    x[2, 200] = bad
    o = cg.rms_norm(x, None)
    keep = torch.arange(6, device="cuda") != 2
    assert torch.equal(o[keep], clean[keep]) and o[2, 200].isnan()
    y, scale = cg.rms_norm_fp8(x, None)
    assert scale[keep].isfinite().all() and y[keep].float().isfinite().all() and not scale[2, 1].isfinite()


# ------------------------------------------------------------------------------------ quantisers


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("n,C", [(1, 8), (3, 128), (130, 200), (127, 16), (257, 1160), (64, 4096)])
def test_quantize(dtype, rows, n, C):
    x = (rand(10, n, C + 8) * torch.exp(2 * rand(11, n, 1))).to(dtype)[:, 8:]
    x[n // 2, C // 2:] *= 1e-3
    call = cg.fp8_quantize if rows == 1 else cg.fp8_quantize_weight
    y, scale = call(x)
    want, ws = ref.quantize(x, rows)
    assert torch.equal(scale.cpu(), ws)
    assert torch.equal(y.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("size", [1e-44, 1e-40, 1e-36, 1e-30, 1e30, 3e38])
def test_quantize_extreme_magnitudes(rows, size):
    x = rand(12, 5, 256).clamp(-1, 1) * size
    x[1] = 0
    call = cg.fp8_quantize if rows == 1 else cg.fp8_quantize_weight
    y, scale = call(x)
    want, ws = ref.quantize(x, rows)
    assert torch.equal(scale.cpu(), ws) and torch.equal(y.cpu().float(), want.float())
    assert ((ref.wide(y, scale, rows) - x.cpu().double()).abs() <= torch.maximum(x.cpu().double().abs() / 16, 2.0 ** -9 * ws.double().max())).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_quantize_keeps_what_is_not_finite_to_its_group(bad):
    x = rand(13, 260, 304, dtype=BF)[:, :296]
    x[131, 130] = bad
    for rows, call in ((1, cg.fp8_quantize), (128, cg.fp8_quantize_weight)):
        y, scale = call(x)
        want, ws = ref.quantize(x, rows)
        assert torch.equal(scale.isfinite().cpu(), ws.isfinite()) and int((~scale.isfinite()).sum()) == 1
        values, fine = ref.wide(y, scale, rows), torch.ones(260, 296, dtype=torch.bool)
        fine[131 if rows == 1 else slice(128, 256), 128:256] = False
        assert torch.equal(values.isfinite(), fine)
        assert torch.equal(values[fine], ref.wide(want, ws, rows)[fine])


# ------------------------------------------------------------------------------------ products


def operands(seed, n, N, K, pad=0):
    """8-bit operands; scales that differ from block to block."""
    x, xs = cg.fp8_quantize(rand(seed, n, K + -K % 8) * torch.exp(rand(seed + 1, 1, K + -K % 8)))
    w, ws = cg.fp8_quantize_weight(rand(seed + 2, N, K + -K % 8) / math.sqrt(K))
    widen = lambda t: torch.nn.functional.pad(t.view(torch.uint8), (0, -K % 16 + pad)).view(E4M3)[:, :K] if K % 16 or pad else t
    return widen(x[:, :K].contiguous()), xs, widen(w[:, :K].contiguous()), ws


def check_matmul(x, xs, w, ws, o, dtype):
    want, size = ref.matmul(x, xs, w, ws)
    K = x.shape[1]
    off = (K / 32 + K / 128 + 11) * 2.0 ** -23 * size
    near(o, want, torch.where(off.isfinite(), off, torch.zeros_like(off)), dtype)


PATHS = [cg.MATMUL_FEW, cg.MATMUL_TILES, cg.MATMUL_AUTO]
SIZES = [(1, 8, 16), (1, 128, 128), (2, 1, 1), (16, 256, 256), (17, 130, 272), (33, 300, 1000), (64, 512, 4096), (65, 129, 384), (128, 1003, 640),
         (129, 257, 130), (200, 500, 2064), (300, 1111, 512), (517, 640, 1024)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,N,K", SIZES)
def test_matmul(path, dtype, n, N, K):
    x, xs, w, ws = operands(20, n, N, K)
    check_matmul(x, xs, w, ws, cg.fp8_matmul(x, xs, w, ws, dtype=dtype, path=path), dtype)


@pytest.mark.parametrize("path", PATHS[:2])
@pytest.mark.parametrize("n", [1, 5, 40, 150])
def test_matmul_strided_rows(path, n):
    """Padded operands, an output inside a wider row: what lies around it stays."""
    x, xs, w, ws = operands(23, n, 203, 500, pad=32)
    wide = torch.full((n, 240), 7.0, device="cuda", dtype=BF)
    o = wide[:, 16:219]
    assert cg.fp8_matmul(x, xs, w, ws, o, path=path) is o
    check_matmul(x, xs, w, ws, o, BF)
    assert (wide[:, :16] == 7).all() and (wide[:, 219:] == 7).all()


@pytest.mark.parametrize("path", PATHS[:2])
@pytest.mark.parametrize("n", [3, 70, 140])
def test_matmul_keeps_what_is_not_finite_to_its_row(path, n):
    x, xs, w, ws = operands(26, n, 300, 400)
    clean = cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path)
    xs, ws, w = xs.clone(), ws.clone(), w.clone()
    xs[1, 2] = math.nan
    xs[2, 0] = math.inf
    w.view(torch.uint8)[5, 17] = 0x7F                                     # e4m3's NaN
    o = cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path)
    fine = torch.ones(n, 300, dtype=torch.bool, device="cuda")
    fine[1:3] = False
    fine[:, 5] = False
    assert torch.equal(o[fine], clean[fine]) and not o[~fine].isfinite().any()
    ws[1, 3] = math.nan                                                   # 128 rows of w
    o = cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path)
    fine[:, 128:256] = False
    assert torch.equal(o[fine], clean[fine]) and not o[~fine].isfinite().any()


@pytest.mark.parametrize("path", PATHS[:2])
@pytest.mark.parametrize("n,N,K", [(4, 640, 512), (300, 640, 512)])
def test_matmul_wait_that_gives_up(path, n, N, K):
    """The status word says so, nothing hangs, and the next call is right."""
    x, xs, w, ws = operands(29, n, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cg.fp8_matmul(x, xs, w, ws, path=path, status=status, wait_polls=-3)
    assert int(status) == cg.ERR_TIMEOUT
    status.zero_()
    check_matmul(x, xs, w, ws, cg.fp8_matmul(x, xs, w, ws, path=path, status=status), BF)
    assert int(status) == cg.OK


def test_matmul_repeats_itself():
    """No order of arrival decides a sum."""
    for n, path in ((7, cg.MATMUL_FEW), (100, cg.MATMUL_FEW), (400, cg.MATMUL_TILES)):
        x, xs, w, ws = operands(32, n, 1000, 4096)
        first = cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path)
        for _ in range(5):
            assert torch.equal(cg.fp8_matmul(x, xs, w, ws, dtype=F32, path=path), first)


# ------------------------------------------------------------------------------------ rotary


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hk,D,R", [(1, 1, 0, 32, 32), (5, 8, 2, 128, 128), (70, 3, 3, 80, 32), (33, 4, 1, 96, 24), (9, 2, 2, 64, 10), (300, 32, 8, 128, 64),
                                         (2, 5, 1, 512, 512), (1300, 4, 2, 64, 64), (4, 1, 1, 8, 2)])
def test_rotary(dtype, interleaved, n, Hq, Hk, D, R):
    row = rand(40, n, (Hq + 2 * Hk + 1) * D, dtype=dtype)
    before = row.clone()
    q, k = row[:, :Hq * D].unflatten(1, (Hq, D)), row[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    g = torch.Generator(device="cuda").manual_seed(41)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    if n > 4:
        pos[2], pos[3], pos[n - 1] = 2 ** 31 - 1, 1 << 20, -1
    freq, _ = cg.rotary_frequencies(R)
    wants = [ref.rotary(t, pos, freq, interleaved, 1.25) for t in (q, k) if t is not None]
    got = cg.rotary(q, k, pos, freq, interleaved=interleaved, scale=1.25)
    assert got[0] is q and got[1] is k
    for t, (want, size) in zip((q, k), wants):
        # four roundings of 2^-53 between the two angles, relative to 2^31 / (2 pi) turns at most: 2^-20
        near(t, want, 6 * U * size + 2.0 ** -19 * size * (pos.cpu().double() / 2 ** 31)[:, None, None].clamp(min=0), dtype)
    assert torch.equal(row[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    if n > 4:
        assert torch.equal(row[n - 1], before[n - 1])
    part = before.unflatten(1, (-1, D))[..., R:]
    assert torch.equal(row.unflatten(1, (-1, D))[..., R:], part)


def test_rotary_head_major_and_round_trip():
    """Heads before tokens in memory; turning by the opposite frequencies gives the input back."""
    base = rand(42, 6, 50, 64)
    q = base.clone().transpose(0, 1)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 20000
    freq, _ = cg.rotary_frequencies(64)
    cg.rotary(q, None, pos, freq)
    want, size = ref.rotary(base.transpose(0, 1), pos, freq, False, 1.0)
    near(q, want, 6 * U * size, F32)
    cg.rotary(q, None, pos, -freq)
    assert (q.transpose(0, 1) - base).abs().max() <= 16 * U * size.max()


def test_rotary_angles_of_far_positions():
    """Of neighbouring positions near 2^31 the angles differ by one frequency: nothing of them is lost."""
    n = 64
    q = torch.zeros(n, 1, 128, device="cuda")
    q[..., :64] = 1
    pos = torch.arange(2 ** 31 - n, 2 ** 31, device="cuda").to(torch.int32)
    freq = torch.full((64,), 0.4, dtype=torch.float64, device="cuda") * torch.rand(64, device="cuda", dtype=torch.float64)
    cg.rotary(q, None, pos, freq)
    z = torch.complex(q[:, 0, :64].double(), q[:, 0, 64:].double())
    step = z[1:] / z[:-1]
    assert (step - torch.polar(torch.ones_like(freq), freq)).abs().max() <= 24 * U
    # and one known angle: 2^30 times a sixteenth of a turn and a bit
    x = torch.zeros(1, 1, 2, device="cuda")
    x[..., 0] = 1
    y = torch.nn.functional.pad(x, (0, 6))
    cg.rotary(y, None, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"),
              torch.tensor([2 * math.pi * (2.0 ** -3 + 2.0 ** -32)], dtype=torch.float64, device="cuda"))
    assert abs(float(y[0, 0, 0])) <= 2e-6 and abs(float(y[0, 0, 1]) - 1) <= 1e-6      # a quarter turn


def test_rotary_nan_frequency_and_values_stay_in_their_pairs():
    q = rand(43, 5, 2, 64)
    q[1, 0, 3] = math.nan
    freq, _ = cg.rotary_frequencies(64)
    freq[7] = math.nan
    pos = torch.arange(1, 6, dtype=torch.int32, device="cuda")
    cg.rotary(q, None, pos, freq)
    bad = q.isnan()
    want = torch.zeros_like(bad)
    want[:, :, [7, 39]] = True
    want[1, 0, [3, 35]] = True
    assert torch.equal(bad, want)


# ------------------------------------------------------------------------------------ calls


def test_nothing_to_do():
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")
    assert cg.rms_norm(e(0, 64), None).shape == (0, 64)
    y, s = cg.rms_norm_fp8(e(0, 64), None)
    assert y.shape == (0, 64) and s.shape == (0, 1)
    y, s = cg.fp8_quantize(e(0, 256))
    w, ws = cg.fp8_quantize_weight(rand(1, 8, 256))
    assert cg.fp8_matmul(y, s, w, ws).shape == (0, 8)
    x, xs = cg.fp8_quantize(rand(1, 3, 256))
    assert cg.fp8_matmul(x, xs, w[:0], ws[:0]).shape == (3, 0)
    cg.rotary(e(0, 2, 64), e(0, 1, 64), e(0, dtype=torch.int32), cg.rotary_frequencies(64)[0])


def chain(x, residual, weight, w, ws, pos, freq):
    """norm -> product -> rotary -> quantise, as a layer does."""
    y, s = cg.rms_norm_fp8(x, weight, residual=residual)
    qk = cg.fp8_matmul(y, s, w, ws)
    q, k = qk[:, :512].unflatten(1, (4, 128)), qk[:, 512:].unflatten(1, (2, 128))
    cg.rotary(q, k, pos, freq)
    return (qk, *cg.fp8_quantize(qk))


@pytest.mark.parametrize("n", [1, 24, 300])
def test_chain_on_another_stream_and_in_a_graph(n):
    weight, (w, ws) = 1 + 0.1 * rand(50, 512), cg.fp8_quantize_weight(rand(51, 768, 512, size=0.05))
    freq, pos = cg.rotary_frequencies(128)[0], torch.arange(n, dtype=torch.int32, device="cuda")
    x, r0 = rand(52, n, 512, dtype=BF), rand(53, n, 512, dtype=BF)
    r = r0.clone()
    want = [t.clone() for t in chain(x, r, weight, w, ws, pos, freq)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2 = r0.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain(x, r2, weight, w, ws, pos, freq)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8) if a.dtype == E4M3 else a, b.view(torch.uint8) if b.dtype == E4M3 else b)
    assert torch.equal(r2, r)
    # captured with other inputs, then replayed with these, twice
    xi, ri, pi = torch.zeros_like(x), torch.zeros_like(r0), torch.zeros_like(pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(xi, ri, weight, w, ws, pi, freq)
    for _ in range(2):
        xi.copy_(x), ri.copy_(r0), pi.copy_(pos)
        graph.replay()
        for a, b in zip(want, out):
            assert torch.equal(a.view(torch.uint8) if a.dtype == E4M3 else a, b.view(torch.uint8) if b.dtype == E4M3 else b)
        assert torch.equal(ri, r)


def test_stream_argument():
    side = torch.cuda.Stream()
    x, w = rand(54, 40, 256, dtype=BF), rand(55, 64, 256, dtype=BF)
    want = cg.fp8_matmul(*cg.fp8_quantize(x), *cg.fp8_quantize_weight(w))
    side.wait_stream(torch.cuda.current_stream())
    got = cg.fp8_matmul(*cg.fp8_quantize(x, stream=side), *cg.fp8_quantize_weight(w, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(want, got)
