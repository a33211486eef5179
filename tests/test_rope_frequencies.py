"""Frequencies and the factor on cos and sin (no GPU)."""
import pytest
import torch

import selective_state_space_causal_amd as ssm


@pytest.mark.parametrize("factor", [0.25, 0.999, 1.0])
def test_yarn_leaves_magnitudes_alone_up_to_a_factor_of_one(factor):
    """The published method's factor 0.1 ln(s) + 1 is for contexts that grow (s > 1); it is 1 otherwise."""
    assert ssm.rope_frequencies(64, scaling="yarn", factor=factor, device="cpu")[1] == 1.0


def test_a_factor_needs_a_scaling():
    """Without one it would change nothing, silently."""
    with pytest.raises(ValueError, match="scaling"):
        ssm.rope_frequencies(64, factor=4.0, device="cpu")
    assert torch.equal(ssm.rope_frequencies(64, factor=1.0, device="cpu")[0], ssm.rope_frequencies(64, device="cpu")[0])
