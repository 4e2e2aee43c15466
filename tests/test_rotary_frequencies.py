"""Frequencies of rotary positions whose base gives the ramp no pairs to go by."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_ramp_refuses_frequencies_that_do_not_fall(base):
    with pytest.raises(ValueError, match="base must be above 1"):
        cg.rotary_frequencies(8, base=base, scaling="ramp", factor=2.0, device="cpu")
    freq, scale = cg.rotary_frequencies(8, base=base, scaling="linear", factor=2.0, device="cpu")
    assert scale == 1.0 and torch.allclose(freq, base ** (-torch.arange(0, 8, 2, dtype=torch.float64) / 8) / 2, rtol=1e-15)
