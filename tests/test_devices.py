"""Calls refuse tensors that are not all on the current device; no GPU needed, the device numbers are made up."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import serve


class At(torch.Tensor):
    """A CPU tensor that says it is on CUDA device ``index``."""
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index


def at(device, *shape, dtype=torch.float32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(At)
    t.index = device
    return t


I32, I64, I8 = torch.int32, torch.int64, torch.int8


def conv(d, **kw):
    return cg.conv_prefill, [d(1, 2, 8), d(8, 4), d(1, 3, 8)], dict(o=d(1, 2, 8), bias=d(8), **kw)


def conv_step(d, **kw):
    return cg.conv_decode, [d(1, 8), d(8, 4), d(1, 3, 8)], dict(o=d(1, 8), **kw)


def scan(d, **kw):
    return cg.scan_prefill, [d(2, 8), d(2, 8), d(8, 16), d(2, 1, 16), d(2, 1, 16), d(1, 8, 16)], \
        dict(o=d(2, 8), D=d(8), z=d(2, 8), dt_bias=d(8), cu_seqlens=d(2, dtype=I32), workspace=d(8), **kw)


def plan(d, **kw):
    return cg.cache_plan, [d(2, 4, dtype=I32)] + [d(n, dtype=I32) for n in (2, 2, 9, 1)] + [3, 16], kw


def cache(d):
    return [d(2, 1, 16, 32, dtype=I8), d(2, 1, 16, 32, dtype=I8), d(2, 1), d(2, 1)]


def append(d, **kw):
    return cg.cache_append, [d(1, 1, 32), d(1, 1, 32), d(1, dtype=I64), *cache(d)], kw


def attend(d, **kw):
    return cg.cache_attend, [d(1, 1, 32), *cache(d), d(1, 2, dtype=I32), d(1, dtype=I32), d(2, dtype=I32)], \
        dict(o=d(1, 1, 32), max_q=1, workspace=d(8), **kw)


def decode(d, **kw):
    return cg.decode, [d(1, 1, 64), d(1, 1, 64), d(1, 1, 64), d(1, 1, 64, 64)], \
        dict(o=d(1, 1, 64), g=d(1, 1, 64), beta=d(1, 1), **kw)


def prefill(d, **kw):
    return cg.prefill, [d(1, 9, 1, 64), d(1, 9, 1, 64), d(1, 9, 1, 64), d(1, 1, 64, 64)], \
        dict(o=d(1, 9, 1, 64), g=d(1, 9, 1, 64), beta=d(1, 9, 1), workspace=d(8), **kw)


CALLS = [conv, conv_step, scan, plan, append, attend, decode, prefill]


@pytest.fixture(autouse=True)
def _device_zero(monkeypatch):
    monkeypatch.setattr(cg, "_device_now", lambda: 0)
    monkeypatch.setattr(serve, "_here", lambda: 0)
    monkeypatch.setattr(cg, "lib", lambda: pytest.fail("the library was reached"))
    monkeypatch.setattr(serve, "lib", lambda: pytest.fail("the library was reached"))


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


def test_plan_into_buffers_of_another_device():
    fn, args, kw = plan(lambda *a, **k: at(0, *a, **k))
    out = cg.CachePlan(2, 3, device="cpu")
    out._buffer = out._buffer.as_subclass(At)
    out._buffer.index = 1
    with pytest.raises(ValueError, match="one device"):
        fn(*args, out=out)


@pytest.mark.parametrize("need", [0, 4])
def test_prefill_looks_at_a_workspace_only_where_it_needs_one(monkeypatch, need):
    """A host tensor (an empty one, say) is fine for a kernel that needs none, and refused where its address would be used."""
    class Library:
        cgdr_prefill_workspace_size = staticmethod(lambda args: need)
        cgdr_prefill = staticmethod(lambda *args: cg.OK)

    monkeypatch.setattr(cg, "lib", Library)
    monkeypatch.setattr(cg, "_stream_handle", lambda stream: None)
    fn, args, kw = prefill(lambda *a, **k: at(0, *a, **k))
    kw["workspace"] = torch.zeros(8)
    if need:
        with pytest.raises(ValueError, match="CUDA device"):
            fn(*args, **kw)
    else:
        assert fn(*args, **kw) is kw["o"]
