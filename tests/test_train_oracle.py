"""Pins of the fp64 oracles of the balance loss and of the MX format against
values worked out by hand, and of the gradient against differences."""
import numpy as np
import pytest

from oracle import train_oracle as O


def test_even_router_has_losses_of_one():
    E, k, T = 8, 2, 4
    idx = np.arange(T * k).reshape(T, k) % E
    stats, counts, prob = O.balance(np.zeros((T, E)), idx)
    assert np.allclose(stats, [1.0, np.log(8) ** 2, 4, 1.0])
    assert np.array_equal(counts, np.ones(E)) and np.allclose(prob, 1 / 8)


def test_rows_that_do_not_count():
    l = np.array([[0.0, 0.0], [-np.inf, -np.inf], [np.nan, np.nan], [-np.inf, 1.0]])
    assert O.counted(l, [1, 1, 0, 1]).tolist() == [True, False, False, True]
    stats, counts, prob = O.balance(l, np.array([[0], [0], [0], [1]]), [1, 1, 0, 1])
    assert stats[2] == 2 and counts.tolist() == [1, 1] and np.allclose(prob, [0.25, 0.75])
    assert not np.any(O.balance(l, np.zeros((4, 1), int), np.zeros(4))[0])


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    T, E, k = 5, 7, 3
    l = rng.normal(size=(T, E))
    l[1, 2] = -np.inf
    l[3] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k]
    mask = [1, 1, 0, 1, 1]
    e = np.exp(l - np.maximum(l.max(1, keepdims=True), -1e30))
    g = np.take_along_axis(e, idx, 1)
    with np.errstate(invalid="ignore"):
        gate = g / (g.sum(1, keepdims=True) if renorm else e.sum(1, keepdims=True))
    dl, dg = [0.3, 0.2], rng.normal(size=(T, k))
    d, _ = O.balance_grad(l, idx, gate, mask, dl, dg, renorm)
    h = 1e-6
    for t in range(T):
        for i in range(E):
            if not np.isfinite(l[t, i]):
                assert d[t, i] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, i] += h
            b[t, i] -= h
            num = (O.balance_total(a, idx, mask, dl, dg, renorm) - O.balance_total(b, idx, mask, dl, dg, renorm)) / (2 * h)
            assert abs(num - d[t, i]) < 1e-7


@pytest.mark.parametrize("renorm", [True, False])
def test_a_choice_that_names_no_expert_takes_no_part(renorm):
    """Its gate and gradient are not looked at; the others' gradient is that of the sum over the named choices, whose
    softmax may have a constant beside them."""
    rng = np.random.default_rng(4)
    E, k, beside = 6, 3, 0.8
    l, dg, idx = rng.normal(size=(1, E)), rng.normal(size=(1, k)), np.array([[4, E, 1]])

    def gates(l):
        e = np.exp(l[0])
        return e[[4, 1]] / (e[[4, 1]].sum() + beside if renorm else e.sum())

    g = gates(l)
    gate = np.array([[g[0], np.nan, g[1]]])
    d, size = O.balance_grad(l, idx, gate, None, [0, 0], dg, renorm)
    dg[0, 1] = np.inf
    again, _ = O.balance_grad(l, idx, gate, None, [0, 0], dg, renorm)
    assert np.array_equal(d, again) and np.isfinite(size).all()
    h = 1e-6
    for i in range(E):
        a, b = l.copy(), l.copy()
        a[0, i] += h
        b[0, i] -= h
        num = ((gates(a) - gates(b)) * dg[0, [0, 2]]).sum() / (2 * h)
        if renorm and i not in (4, 1):
            assert d[0, i] == 0
        assert abs(num - d[0, i]) < 1e-8


def test_quantised_values_by_hand():
    x = np.zeros((1, 64))
    x[0, :12] = [4, 0.25, 0.26, -0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.01, 7.9, -0.1]
    x[0, 32] = 1e-45
    codes, scales = O.mx4_quantize(x)
    assert scales[0, :2].tolist() == [127, 0]
    v = O.mx4_values(codes, scales)[0]
    assert v[:12].tolist() == [4, 0, 0.5, -1, 1, 2, 2, 4, 4, -6, 6, 0]
    assert codes[0, 5] >> 4 == 8  # -0.1 keeps its sign
    x[0, 40] = np.inf
    codes, scales = O.mx4_quantize(x)
    assert scales[0, 1] == 255 and np.isnan(O.mx4_values(codes, scales)[0, 32:]).all()


def test_values_survive_a_second_quantisation():
    x = np.random.default_rng(2).normal(size=(3, 96)) * 10
    v = O.mx4_values(*O.mx4_quantize(x))
    assert np.array_equal(O.mx4_values(*O.mx4_quantize(v)), v)
    assert (np.abs(v - x) <= np.abs(x).max() / 4).all()
