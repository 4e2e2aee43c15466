"""examples/hybrid_decoder.py: no layers at all, and products whose waits give up."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from test_hybrid_example_gpu import example  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def ids(n):
    return torch.randint(0, 512, (n,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")


def test_a_wait_that_gives_up_reaches_the_status_word(example, monkeypatch):  # noqa: F811
    """A product that gives up leaves undefined values: the decoder's status word says so."""
    d = example.HybridDecoder(layers=("attend",), eight_bit=True)
    d.step(ids(9), [4, 2, 3])
    assert int(d.status) == cg.OK
    product, calls = cg.fp8_matmul, []

    def hasty(*args, **kw):
        calls.append(kw)
        return product(*args, **dict(kw, wait_polls=-3))

    monkeypatch.setattr(example.cg, "fp8_matmul", hasty)
    d.step(ids(3), [1, 1, 1])
    assert len(calls) == 2 and int(d.status) == cg.ERR_TIMEOUT
    # each of the two by itself
    assert all(kw.get("status") is d.status for kw in calls)
