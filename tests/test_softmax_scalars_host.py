"""Numbers that the Softmax branch's calls refuse instead of taking a default
for them, without a GPU: they are looked at before any tensor."""

import pytest

torch = pytest.importorskip("torch")

from frame_wise_delta_vda_b200 import api

Q = torch.zeros(3, 4, 64)


@pytest.mark.parametrize("scale", [0.0, -0.5, 1e-50, 2.0 ** -151, float("nan"), float("inf"), 1e30, 1e300])
def test_scales_that_float32_does_not_hold_are_refused(scale):
    """0 stands for the default in the argument block: what rounds to it must not become 1 / sqrt(d)."""
    with pytest.raises(ValueError, match="scale"):
        api.vda_paged_attention(Q, None, None, None, None, None, scale=scale)


@pytest.mark.parametrize("scale", [None, 1, 0.125, 2.0 ** -149, 9e29])
def test_other_scales_pass_on_to_the_tensors(scale):
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_paged_attention(Q, None, None, None, None, None, scale=scale)
