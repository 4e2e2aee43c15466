"""Rotary positions: sines and cosines to their own size, not only to that of the values that they turn."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def turned(u, v, pos, freq, interleaved):
    half = freq.shape[0]
    q = torch.empty(pos.shape[0], 1, 2 * half, device="cuda")
    a, b = (q[..., 0::2], q[..., 1::2]) if interleaved else (q[..., :half], q[..., half:])
    a.fill_(u), b.fill_(v)
    cg.rotary(q, None, pos, freq, interleaved=interleaved)
    return a[:, 0].double().cpu(), b[:, 0].double().cpu()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,kw", [(1e4, {}), (1e6, {}), (1e7, {}), (1e7, dict(scaling="linear", factor=64.0)), (5e5, dict(scaling="turns", factor=8.0))])
def test_sine_and_cosine_to_their_own_size(base, kw, interleaved):
    """(0, 1) and (1, 0) turned give the sine and the cosine themselves.  The fraction of a turn is cut at 2^-64, which is 2^-32
    of the slowest frequency here (2e-9 rad, 3e-10 turns) and less of the others; the remainder's rounding to fp32 is 2^-24 of it, and near a quarter turn, where
    the other function is small, of that function; sine and cosine are off by an ulp, 2^-23; products with 0 and 1 and the sum are
    exact.  3 2^-24, and one more for the orders left out and the 64-bit form, whose angle of up to 50 rad is off by 2^-48."""
    freq, _ = cg.rotary_frequencies(128, base=base, **kw)
    pos = torch.arange(1, 51, dtype=torch.int32, device="cuda")
    angle = pos.cpu().double()[:, None] * freq.cpu()
    for (u, v), (first, second) in (((0.0, 1.0), (-angle.sin(), angle.cos())), ((1.0, 0.0), (angle.cos(), angle.sin()))):
        for got, want in zip(turned(u, v, pos, freq, interleaved), (first, second)):
            assert ((got - want).abs() <= 4 * U * want.abs()).all()


def test_slow_pairs_turn_at_all():
    """Angles below the smallest step of a 32-bit fraction of a turn (1.5e-9 rad) are angles, not zeros."""
    freq = torch.tensor([2.0 ** -30, 2.0 ** -33, 2.0 ** -36, -2.0 ** -36], dtype=torch.float64, device="cuda")
    first, second = turned(0.0, 1.0, torch.tensor([1, 3], dtype=torch.int32, device="cuda"), freq, False)
    want = torch.tensor([[1.0], [3.0]], dtype=torch.float64) * freq.cpu()
    assert ((first + want).abs() <= 4 * U * want.abs()).all() and (second == 1).all()
