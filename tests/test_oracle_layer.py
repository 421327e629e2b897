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


@pytest.mark.parametrize("renormalize", [False, True])
def test_softmax_routing_is_the_plain_router(renormalize):
    import oracle

    rng = np.random.default_rng(5)
    logits = rng.standard_normal((40, 12)).astype(np.float32)
    ids, w = layer.route_grouped(logits, 3, "softmax", None, 1, 1, 1, renormalize, 1.0)
    ids0, w0 = oracle.topk_softmax(logits, 3, renormalize)
    assert np.array_equal(ids, ids0) and np.allclose(w, w0, rtol=1e-6)
    st, off, row_of = layer.dispatch(ids, 12)
    st0, off0, row0 = oracle.moe_align(ids0, 12)
    assert np.array_equal(st, st0) and np.array_equal(off, off0) and np.array_equal(row_of, row0)


def test_groups_and_bias_by_hand():
    # scores of the sigmoid: 0 -> 0.5, large -> 1
    l = np.array([[0, 0, 9, -9, 1, 1, -1, 2]], np.float32)   # groups (0 0) (9 -9) (1 1) (-1 2)
    args = dict(kind="sigmoid", groups=4, renormalize=False, scale=2.0)
    ids, w = layer.route_grouped(l, 2, bias=None, topk_groups=1, group_top=1, **args)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, 2 / (1 + np.exp([[-9.0, 9.0]])))
    ids, _ = layer.route_grouped(l, 2, bias=None, topk_groups=1, group_top=2, **args)
    assert ids.tolist() == [[4, 5]]
    bias = np.array([0.9, 0.8, 0, 0, 0, 0, 0, 0])
    ids, w = layer.route_grouped(l, 3, bias=bias, topk_groups=2, group_top=2, **args)
    assert ids.tolist() == [[0, 1, 4]] and np.allclose(w[0, :2], 1.0)   # the bias is not in the weights
    bias = np.array([0, 0, 0, 0, -np.inf, 0, 0, np.nan])
    ids, _ = layer.route_grouped(l, 8, bias=bias, topk_groups=4, group_top=2, **args)
    assert ids.tolist() == [[2, 5, 0, 1, 6, 3, 4, 7]]


def test_rows_of_nothing():
    l = np.full((2, 4), -np.inf)
    l[1, 2] = np.nan
    for kind in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            ids, w = layer.route_grouped(l, 2, kind, None, 1, 1, 1, renormalize, 1.0)
            assert ids.tolist() == [[0, 1], [0, 1]] and not w.any()
    l[0, 3] = l[0, 1] = np.inf
    ids, w = layer.route_grouped(l, 2, "softmax", None, 1, 1, 1, False, 1.0)
    assert ids[0].tolist() == [1, 3] and w[0].tolist() == [0.5, 0.5]


def test_adapters_are_a_change_of_the_weight():
    rng = np.random.default_rng(6)
    M, N, K, L, R = 6, 10, 7, 3, 2
    x, y, a, b = (rng.standard_normal(s) for s in ((M, K), (M, N), (L, 2 * R, K), (L, N, R)))
    s, adapter = np.array([0.5, 2.0, -1.0]), np.array([2, 0, -1, 1, 3, 2])
    out, of_t, of_x = layer.lora_add(y, x, a, b, s, adapter, [4, 6])
    for m in range(M):
        e = adapter[m]
        if not 0 <= e < L:
            assert np.array_equal(out[m], y[m]) and not of_t[m].any()
            continue
        change = s[e] * np.concatenate([b[e, :4] @ a[e, :R], b[e, 4:] @ a[e, R:]])
        assert np.allclose(out[m], y[m] + change @ x[m])
        assert np.all(of_x[m] >= of_t[m] - 1e-12) and np.all(of_t[m] >= np.abs(out[m] - y[m]) - 1e-12)
    assert np.allclose(layer.lora_add(y, x, a, b, None, adapter, [4, 6])[0][1], layer.lora_add(
        y, x, a, b, np.ones(3), adapter, [4, 6])[0][1])
