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


K = torch.zeros(3, 2, 64)
EPS = [0.0, -1e-6, 1e-50, float("nan"), float("inf"), 1e39, 1e300]


@pytest.mark.parametrize("eps", EPS)
def test_eps_that_would_become_the_default_is_refused(eps):
    """0 stands for 1e-6 in the argument block: another norm than the one asked for."""
    with pytest.raises(ValueError, match="eps"):
        api.vda_qk_norm_rope(Q, K, eps=eps)
    with pytest.raises(ValueError, match="eps"):
        api.vda_qk_norm_rope_backward(Q, K, Q, K, eps=eps)


@pytest.mark.parametrize("eps", [1e-6, 1, 2.0 ** -149, 3e38])
def test_other_eps_pass_on_to_the_tensors(eps):
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_qk_norm_rope(Q, K, eps=eps)
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_qk_norm_rope_backward(Q, K, Q, K, eps=eps)


@pytest.mark.parametrize("eps", [float("nan"), float("inf")])
def test_the_library_refuses_eps_that_is_no_number(eps):
    import ctypes

    from frame_wise_delta_vda_b200 import _lib
    from test_softmax_refusals_host import INVALID, P, grad_args, qk_args
    L = _lib.lib()
    # an empty batch: nothing else is refused, and nothing is launched
    assert L.vda_qk_norm_rope(ctypes.byref(qk_args(N=0))) == 0
    assert L.vda_qk_norm_rope(ctypes.byref(qk_args(N=0, eps=eps))) == INVALID
    none = dict(N=0, dq_weight=None, dk_weight=None)
    assert L.vda_qk_norm_rope_backward(ctypes.byref(grad_args(**none)), P, 1 << 30) == 0
    assert L.vda_qk_norm_rope_backward(ctypes.byref(grad_args(**none, eps=eps)), P, 1 << 30) == INVALID
