"""Pins of the oracle of the operators beside the 8-bit products (no GPU): closed forms and invariants."""
import numpy as np
import pytest

from oracle import layer


def table(P, rot):
    angle = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    T, H, D, rot = 5, 3, 12, 8
    x, tab, pos = rng.standard_normal((T, H, D)), table(9, rot), np.array([[0, 3, 8, 1, 2]])
    out, mag = layer.head_norm_rope(x, None, 0.0, tab, pos, [4], rot, interleaved)
    first, second = (np.arange(0, 8, 2), np.arange(1, 8, 2)) if interleaved else (np.arange(4), np.arange(4, 8))
    turn = (tab[pos[0], :4] + 1j * tab[pos[0], 4:])[:, None]
    z = (x[..., first] + 1j * x[..., second]) * turn
    assert np.allclose(out[..., first], z.real, atol=1e-15) and np.allclose(out[..., second], z.imag, atol=1e-15)
    assert np.array_equal(out[..., rot:], x[..., rot:]) and np.array_equal(out[0], x[0])
    assert np.all(mag >= np.abs(out) - 1e-15)
    # lengths stay
    assert np.allclose(np.linalg.norm(out, axis=2), np.linalg.norm(x, axis=2))


def test_rotation_goes_by_the_difference_of_positions():
    rng = np.random.default_rng(2)
    a, b, tab = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16)), table(100, 16)

    def at(x, p):
        return layer.head_norm_rope(x, None, 0.0, tab, np.array([[p]]), [8], 16, False)[0].ravel()

    assert np.isclose(at(a, 7) @ at(b, 3), at(a, 94) @ at(b, 90))


def test_axes_turn_their_own_pairs():
    rng = np.random.default_rng(3)
    x, tab = rng.standard_normal((1, 2, 12)), table(20, 12)
    out = layer.head_norm_rope(x, None, 0.0, tab, np.array([[5], [0], [9]]), [2, 3, 1], 12, False)[0]
    for p, pairs in ((5, [0, 1]), (0, [2, 3, 4]), (9, [5])):
        one = layer.head_norm_rope(x, None, 0.0, tab, np.array([[p]]), [6], 12, False)[0]
        for i in pairs:
            assert np.array_equal(out[..., [i, i + 6]], one[..., [i, i + 6]])


def test_norm_makes_heads_of_the_weight_s_length():
    rng = np.random.default_rng(4)
    x, w = 50 * rng.standard_normal((4, 2, 32)), np.full(32, 3.0)
    out = layer.head_norm_rope(x, w, 0.0, table(4, 32), np.array([[0, 1, 2, 3]]), [16], 32, True)[0]
    assert np.allclose(np.sqrt(np.mean(out ** 2, axis=2)), 3.0)


def test_positions_outside_the_table():
    x = np.ones((3, 1, 4))
    out = layer.head_norm_rope(x, None, 0.0, table(4, 4), np.array([[-1, 4, 3]]), [2], 4, False)[0]
    assert np.isnan(out[:2]).all() and np.isfinite(out[2]).all()
