"""8-bit projections against bf16 ones: the same decoder, tokens and steps."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from test_hybrid_example_gpu import example  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [(70, 1, 133), (1, 1, 1), (5, 200, 16)])
def test_8_bit_projections_compute_what_bf16_ones_do(example, lens):  # noqa: F811
    """One attention layer over embeddings that are small beside what it adds (the norm in front of it takes their size out), so that
    the logits are its output and nothing else: a product that is zero, turned over or wrongly scaled is off by their whole RMS.

    A rounding to e4m3 is off by 2^-4 of the value at most, an RMS of 2^-4 / sqrt 3 = 0.036 of it; a product of two such operands by
    0.051.  So are q, k and v.  Scores q k / sqrt 128 of values of RMS 1 are then off by 0.051 sqrt 2 = 0.072, and with them the
    weights of a row, and o by that and v's 0.051: 0.088.  The cache's 8 bits (a step of 1/127 of a page's largest value, some 4 RMS: 0.009,
    in k and v, and the scales differ between the two) add 0.02, the second product 0.051: together 0.104 of the RMS.  The final norm takes a
    common factor out and adds nothing.  These are RMS over 1e5 values, whose estimate is good to a few percent, but q and k of a row share their
    errors over all its scores: 0.15.  The bound from below, a tenth of one rounding, is there to see that the 8 bits were used."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    tail = 2
    tokens = [torch.randint(0, 512, (l + tail,), generator=g, device="cuda") for l in lens]
    logits = []
    for eight_bit in (False, True):
        d = example.HybridDecoder(layers=("attend",), eight_bit=eight_bit)
        d.embedding *= 0.01
        steps = [d.step(torch.cat([t[:l] for t, l in zip(tokens, lens)]), list(lens))]
        for k in range(tail):
            steps.append(d.step(torch.stack([t[l + k] for t, l in zip(tokens, lens)]), [1] * len(lens)))
        assert int(d.status) == cg.OK
        logits.append([s.double() for s in steps])
    for plain, eight in zip(*logits):
        off = float((eight - plain).square().mean().sqrt() / plain.square().mean().sqrt())
        assert 0.0036 < off < 0.15
