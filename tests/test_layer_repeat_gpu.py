"""Norm, quantisers and rotary positions at the sizes of prompts: the same bits every time, whatever the blocks' order."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from test_layer_gpu import BF, F32, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def norm(dtype):
    x, r, w = rand(1, 4001, 4096, dtype=dtype), rand(2, 4001, 4096, dtype=dtype), rand(3, 4096)

    def call():
        now = r.clone()
        return cg.rms_norm(x, w, residual=now), now
    return call


def norm8(dtype):
    x, r, w = rand(1, 4001, 4096, dtype=dtype), rand(2, 4001, 4096, dtype=dtype), rand(3, 4096)

    def call():
        now = r.clone()
        return *cg.rms_norm_fp8(x, w, residual=now), now
    return call


def heads(dtype):
    row, w = rand(4, 4000, 40 * 128, dtype=dtype), rand(5, 128)
    return lambda: (cg.rms_norm(row[:, 1024:].unflatten(1, (32, 128)), w),)


def rows(dtype):
    x = rand(6, 4001, 4096, dtype=dtype)
    return lambda: cg.fp8_quantize(x)


def blocks(dtype):
    x = rand(7, 4001, 4096, dtype=dtype)
    return lambda: cg.fp8_quantize_weight(x)


def rotary(dtype):
    q0, pos, (freq, _) = rand(8, 4000, 40, 128, dtype=dtype), torch.arange(4000, dtype=torch.int32, device="cuda"), cg.rotary_frequencies(128)

    def call():
        q = q0.clone()
        return cg.rotary(q[:, :32], q[:, 32:], pos, freq)
    return call


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("make", [norm, norm8, heads, rows, blocks, rotary])
def test_repeats_itself(make, dtype):
    call = make(dtype)
    bits = lambda out: [t.contiguous().view(torch.uint8).clone() for t in out]
    first = bits(call())
    for _ in range(30):
        assert all(torch.equal(a, b) for a, b in zip(bits(call()), first))
