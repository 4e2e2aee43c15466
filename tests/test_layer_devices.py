"""The operators around a layer's state refuse tensors that are not all on the current device; no GPU needed."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import layer, serve
from test_devices import I32, at

E, F64 = torch.float8_e4m3fn, torch.float64


def norm(d, **kw):
    return cg.rms_norm, [d(2, 8), d(8)], dict(o=d(2, 8), residual=d(2, 8), **kw)


def norm8(d, **kw):
    return cg.rms_norm_fp8, [d(2, 8), d(8)], dict(y=d(2, 8, dtype=E), y_scale=d(2, 1), residual=d(2, 8), **kw)


def quantize(d, **kw):
    return cg.fp8_quantize, [d(2, 8), d(2, 8, dtype=E), d(2, 1)], kw


def quantize_weight(d, **kw):
    return cg.fp8_quantize_weight, [d(2, 8), d(2, 8, dtype=E), d(1, 1)], kw


def matmul(d, **kw):
    return cg.fp8_matmul, [d(2, 16, dtype=E), d(2, 1), d(8, 16, dtype=E), d(1, 1)], dict(o=d(2, 8), **kw)


def rotary(d, **kw):
    return cg.rotary, [d(2, 1, 8), d(2, 1, 8), d(2, dtype=I32), d(4, dtype=F64)], kw


CALLS = [norm, norm8, quantize, quantize_weight, matmul, rotary]


@pytest.fixture(autouse=True)
def _device_zero(monkeypatch):
    monkeypatch.setattr(cg, "_device_now", lambda: 0)
    monkeypatch.setattr(serve, "_here", lambda: 0)
    monkeypatch.setattr(layer, "lib", lambda: pytest.fail("the library was reached"))


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_a_device_that_is_not_current(call):
    fn, args, kw = call(lambda *a, **k: at(1, *a, **k))
    with pytest.raises(ValueError, match="current device is 0"):
        fn(*args, **kw)


@pytest.mark.parametrize("call", CALLS)
def test_each_tensor_on_another_device_than_the_rest(call):
    made = [0]

    def count(*a, **k):
        made[0] += 1
        return at(0, *a, **k)

    call(count)
    for odd in range(made[0]):
        seen = [-1]

        def one_odd(*a, **k):
            seen[0] += 1
            return at(1 if seen[0] == odd else 0, *a, **k)

        fn, args, kw = call(one_odd)
        with pytest.raises(ValueError, match="one device"):
            fn(*args, **kw)


@pytest.mark.parametrize("call", CALLS)
def test_status_word_of_another_device(call):
    fn, args, kw = call(lambda *a, **k: at(0, *a, **k), status=at(1, 1, dtype=I32))
    with pytest.raises(ValueError, match="device"):
        fn(*args, **kw)
