"""Where the norm's squares leave fp32: right up to the bound on their sum, zero behind it, and no row disturbs another."""
import math

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
import layer_ref as ref
from test_layer_gpu import BF, F32, U, near, rand

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("C", [8, 512, 4096, 12288, 32768])
def test_large_rows(dtype, C):
    """All values of one size, with a sum of squares of 0.9 and 1.1 of fp32's largest (before their rounding to dtype, 2^-8 each at most, so
    2^-7 of the sum; the sum itself is off by 70 2^-24 at most)."""
    sign = torch.where(rand(1, 6, C) > 0, 1.0, -1.0)
    x = sign * math.sqrt(MOST / C * 0.9)
    x[1] = sign[1] * math.sqrt(MOST / C * 1.1)
    x[2], x[2, C // 2] = 0, 1.8e19                     # one value alone: 1.8446e19 is the largest whose square is finite
    x[3], x[3, C // 2] = 0, -1.9e19
    x[4] = sign[4]
    x = x.to(dtype)
    want, _ = ref.norm(x, None)
    want[1] = want[3] = 0
    o = cg.rms_norm(x, None)
    near(o, want, 40 * U * want.abs(), dtype)
    assert o[0].any() and o[2].any() and not o[1].any() and not o[3].any()
    y, scale = cg.rms_norm_fp8(x, None)
    assert not y[1].float().any() and not y[3].float().any() and (y[0].float().abs() == 448).all()
    assert y.float().isfinite().all() and scale.isfinite().all()
