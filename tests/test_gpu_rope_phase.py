"""The angles of vda_qk_norm_rope at high frequencies and far positions, against
angles in rational arithmetic.

Tolerance, before the first run, as in test_gpu_qk_norm_rope: the phase is off
by 2^-25 + 2^31 2^-64 turns, so cos and sin by 2^-22 together with the
functions' own error, and a rotated value by 2^-19 (|z_i| + |z_j|)."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import softmax_ref as ref
from test_gpu_qk_norm_rope import _case, _np

torch = pytest.importorskip("torch")


def _two_pi(bits=300):
    """2 pi as a fraction, by Machin's formula."""
    one = 1 << bits

    def arctan_inverse(n):
        x = total = one // n
        k, sign = 3, -1
        while x:
            x //= n * n
            total += sign * (x // k)
            k, sign = k + 2, -sign
        return total

    return Fraction(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


def _phases(positions, frequencies):
    """[N, pairs] radians within half a turn, rounded once."""
    turn = _two_pi()
    steps = [Fraction(float(f)) / turn for f in frequencies]
    out = [[float((p * s - round(p * s)) * turn) for s in steps] for p in map(int, positions)]
    return np.array(out)


def test_phases_are_the_angles():
    f = np.array([1.0, 0.01, 6.1, -3.7, 100.0])
    p = np.array([0, 1, 5, -7, 1000])
    phi = _phases(p, f)
    np.testing.assert_allclose(np.cos(phi), np.cos(p[:, None] * f), atol=1e-10)
    np.testing.assert_allclose(np.sin(phi), np.sin(p[:, None] * f), atol=1e-10)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_high_frequencies_at_far_positions(interleaved):
    from frame_wise_delta_vda_b200 import api
    c, _, g = _case(64, 2, 1, 64, torch.float32, 64)
    n = 32
    f = np.concatenate([[100.0, -100.0, 6.2831, 6.2832, 3.1, -1.5, 1e3, 1e6, 2.0 ** 40, 1e-9, 0.0],
                        np.exp(np.random.default_rng(1).uniform(-5, 12, n - 11))])
    p = 2 ** 31 - 1 - np.arange(64) * 77
    p[::3] *= -1
    c["frequencies"] = torch.from_numpy(f).cuda()
    c["positions"] = torch.from_numpy(p.astype(np.int32)).view(64, 1).cuda()
    phi = _phases(p, f)
    qo, _ = api.vda_qk_norm_rope(**c, interleaved=interleaved)
    z = ref.norm(_np(c["q"]), 1e-6)[0] * _np(c["q_weight"])
    size = 2.0 ** -19 * ref.paired_magnitude(z, 64, interleaved)
    bad = (np.abs(_np(qo) - ref.rotate(z, phi, interleaved)) / size).max((0, 1))
    assert bad.max() <= 1.0, bad

    dy = torch.randn(64, 2, 64, generator=g).cuda()
    dq, _, _, _ = api.vda_qk_norm_rope_backward(dy, c["k"], **c, interleaved=interleaved)
    x, w = _np(c["q"]), _np(c["q_weight"])
    want, _ = ref.norm_rope_backward(_np(dy), x, w, phi, interleaved)
    u, inv = ref.norm(x, 1e-6)
    m = ref.paired_magnitude(_np(dy), 64, interleaved) * np.abs(w)
    size = 2.0 ** -18 * inv * (m + np.abs(u) * (m * np.abs(u)).mean(-1, keepdims=True))
    bad = (np.abs(_np(dq) - want) / size).max((0, 1))
    assert bad.max() <= 1.0, bad
