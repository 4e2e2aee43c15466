"""What the binding of the serving operators refuses before it looks at the tensors; no GPU needed."""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan")])
def test_attention_scale_is_above_zero(scale):
    """Not taken for the default, which the C call selects by such a value."""
    z = torch.zeros(1, 1, 1, 32)
    with pytest.raises(ValueError, match="scale"):
        cg.cache_attend(z[0], z, z, z[0, 0], z[0, 0], z[0, 0], z[0, 0, 0], z[0, 0, 0], max_q=1, scale=scale)
