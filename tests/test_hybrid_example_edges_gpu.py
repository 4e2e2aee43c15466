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


@pytest.mark.parametrize("eight_bit", [False, True])
def test_no_layers(example, eight_bit):  # noqa: F811
    """A decoder of no layers: the logits of the normed embeddings.  Two bf16 roundings, 2^-8 each: the norm's, whose errors of up to
    2^-8 |h_i| meet the head's column with at most 2^-8 |h| |w|, and the logits'; a tenth more for fp32 sums and their product."""
    d = example.HybridDecoder(layers=(), eight_bit=eight_bit)
    tokens = ids(9)
    got = d.step(tokens, [4, 2, 3]).double()
    x = d.embedding[tokens].double()
    h = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    want = h @ d.head.double()
    size = h.square().sum(-1, keepdim=True).sqrt() * d.head.double().square().sum(0).sqrt()
    assert ((got - want).abs() <= 2.0 ** -8 * (want.abs() + 1.1 * size)).all()
