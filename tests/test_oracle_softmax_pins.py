"""The Softmax branch's float64 oracle against closed forms and differences."""

import numpy as np
import pytest

from oracle import softmax_ref as ref


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_each_pair_by_its_angle(interleaved):
    rng = np.random.default_rng(0)
    z = rng.standard_normal((3, 2, 8))
    phi = rng.standard_normal((3, 3))
    y = ref.rotate(z, phi, interleaved)
    for p in range(3):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + 3)
        want = (z[..., i] + 1j * z[..., j]) * np.exp(1j * phi[:, p])[:, None]
        np.testing.assert_allclose(y[..., i] + 1j * y[..., j], want, atol=1e-14)
    np.testing.assert_array_equal(y[..., 6:], z[..., 6:])


def test_rotated_products_depend_on_position_differences():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 1, 16))
    freq, axis = 10.0 ** -np.arange(8.0), np.zeros(8, int)
    at = lambda p: ref.rotate(x, ref.angles([[p]], freq, axis))[0, 0]  # noqa: E731
    np.testing.assert_allclose(at(5) @ at(9), at(1005) @ at(1009), rtol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_against_differences(interleaved):
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((2, 3, 16)), rng.standard_normal(16), rng.standard_normal((2, 3, 16))
    phi = rng.standard_normal((2, 4))
    dx, dw = ref.norm_rope_backward(dy, x, w, phi, interleaved)
    loss = lambda x, w: (dy * ref.norm_rope(x, w, phi, interleaved)).sum()  # noqa: E731
    h = 1e-6
    for idx in [(0, 0, 0), (1, 2, 5), (0, 1, 9), (1, 0, 15)]:
        e = np.zeros_like(x)
        e[idx] = h
        np.testing.assert_allclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[idx], rtol=1e-6, atol=1e-8)
    for c in (0, 3, 8, 15):
        e = np.zeros_like(w)
        e[c] = h
        np.testing.assert_allclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[c], rtol=1e-6, atol=1e-8)


def test_visible_is_causal_by_tokens_and_by_blocks():
    np.testing.assert_array_equal(ref.visible([2, 3], 4, 1, -1, 0), [[1, 1, 1, 0], [1, 1, 1, 1]])
    np.testing.assert_array_equal(ref.visible([2, 3], 4, 1, 1, 0), [[0, 1, 1, 0], [0, 0, 1, 1]])
    # one anchor, blocks of two behind it: positions 1-2, 3-4, 5-6
    np.testing.assert_array_equal(ref.visible([0, 1, 4, 6], 7, 2, 0, 1),
                                  [[1, 0, 0, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0, 0], [1, 0, 0, 1, 1, 0, 0],
                                   [1, 0, 0, 0, 0, 1, 1]])
    np.testing.assert_array_equal(ref.visible([-1, 0], 2, 1, -1, 0), [[0, 0], [1, 0]])
    np.testing.assert_array_equal(ref.visible([-1, 0], 2, 0, -1, 0), [[0, 0], [1, 1]])


def test_attention_of_equal_scores_is_the_mean_and_of_nothing_is_zero():
    rng = np.random.default_rng(3)
    v = rng.standard_normal((5, 4))
    see = np.array([[1, 1, 0, 1, 0], [0, 0, 0, 0, 0]], bool)
    o, lse = ref.attend(np.zeros((2, 1, 4)), rng.standard_normal((5, 4)), v, see, 0.5)
    np.testing.assert_allclose(o[0, 0], v[[0, 1, 3]].mean(0))
    np.testing.assert_allclose(lse[0, 0], np.log(3))
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()


def test_paged_attention_reads_the_table_and_skips_absent_pages():
    rng = np.random.default_rng(4)
    kc, vc = rng.standard_normal((6, 2, 4, 8)), rng.standard_normal((6, 2, 4, 8))
    q = rng.standard_normal((3, 4, 8))
    table = np.array([[5, 1, 2], [3, -1, 0]])
    out, _ = ref.paged_attention(q, kc, vc, table, [10, 9], [0, 2, 3])
    k = np.concatenate([kc[p, 1] for p in (5, 1, 2)])[:10]
    v = np.concatenate([vc[p, 1] for p in (5, 1, 2)])[:10]
    s = q[0, 2] @ k[:9].T / np.sqrt(8)
    e = np.exp(s - s.max())
    np.testing.assert_allclose(out[0, 2], e @ v[:9] / e.sum(), rtol=1e-12)
    k = np.concatenate([kc[3, 0], kc[0, 0, :1]])
    v = np.concatenate([vc[3, 0], vc[0, 0, :1]])
    s = q[2, 1] @ k.T / np.sqrt(8)
    e = np.exp(s - s.max())
    np.testing.assert_allclose(out[2, 1], e @ v / e.sum(), rtol=1e-12)
