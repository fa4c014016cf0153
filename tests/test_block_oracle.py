"""The fp64 definitions of norm, gate and linear are themselves checked: gradients against central
differences, selections against brute force and hand-worked cases."""
import itertools

import numpy as np
import pytest

from oracle import block_oracle as B


def central(f, x, d, h=1e-6):
    """Directional derivative of the scalar f at x along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("H", [1, 7, 64])
def test_norm_gradient_is_the_difference_quotient(kind, H):
    rng = np.random.default_rng(H)
    x, r, dy, ds = (rng.normal(size=(5, H)) for _ in range(4))
    w, b = rng.normal(size=H), rng.normal(size=H)

    def loss(x_, w_, b_):
        y, h, _, _ = B.norm_fwd(x_, r, w_, b_, kind, 1e-2)
        return (y * dy).sum() + (h * ds).sum()

    _, h, mean, rstd = B.norm_fwd(x, r, w, b, kind, 1e-2)
    dx, dw, db = B.norm_bwd(dy, ds, h, w, mean, rstd, kind)
    for _ in range(3):
        d, e, f = rng.normal(size=x.shape), rng.normal(size=H), rng.normal(size=H)
        assert np.isclose(central(lambda v: loss(v, w, b), x, d), (dx * d).sum(), rtol=1e-6, atol=1e-7)
        assert np.isclose(central(lambda v: loss(x, v, b), w, e), (dw * e).sum(), rtol=1e-6, atol=1e-7)
        assert np.isclose(central(lambda v: loss(x, w, v), b, f), (db * f).sum(), rtol=1e-6, atol=1e-7)


def test_norm_of_a_layer_row_has_zero_mean_and_unit_variance():
    x = np.random.default_rng(0).normal(3.0, 2.0, size=(4, 50))
    y, _, _, _ = B.norm_fwd(x, None, np.ones(50), None, "layer", 0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(6, 12))
    dw = rng.normal(size=(6, 4))
    idx, _ = B.gate_select(l, None, 4, score)
    f = lambda v: (B.gate_weights(v, idx, score, renorm, 2.5) * dw).sum()
    dl = B.gate_bwd(l, idx, dw, score, renorm, 2.5)
    for _ in range(4):
        d = rng.normal(size=l.shape)
        assert np.isclose(central(f, l, d), (dl * d).sum(), rtol=1e-6, atol=1e-8)


def test_gate_selection_is_brute_force():
    """With distinct choice scores the chosen set maximises the score sum over every allowed set."""
    rng = np.random.default_rng(4)
    l, bias = rng.normal(size=(10, 12)), 0.1 * rng.normal(size=12)
    idx, _ = B.gate_select(l, bias, 3, "sigmoid", n_group=4, topk_group=2, group_take=2)
    _, s = B.gate_scores(l, "sigmoid")
    for t in range(10):
        c = s[t] + bias
        best_groups = max(itertools.combinations(range(4), 2),
                          key=lambda gs: sum(np.sort(c[3 * g:3 * g + 3])[-2:].sum() for g in gs))
        cand = [e for g in best_groups for e in range(3 * g, 3 * g + 3)]
        best = max(itertools.combinations(cand, 3), key=lambda es: sum(c[e] for e in es))
        assert sorted(idx[t]) == sorted(best)
        assert list(idx[t]) == sorted(best, key=lambda e: -c[e])


def test_gate_ties_and_masks_by_hand():
    inf = np.inf
    l = np.array([[1.0, 2.0, 2.0, 1.0],           # tie for the first slot: lower expert
                  [-inf, 0.0, -inf, -inf],        # one expert left: the masked ones follow, lowest first
                  [-inf, -inf, -inf, -inf],       # nothing left
                  [np.nan, 3.0, inf, 0.0]])       # NaN masks; +inf takes all of the softmax
    idx, _ = B.gate_select(l, None, 3, "softmax")
    assert idx.tolist() == [[1, 2, 0], [1, 0, 2], [0, 1, 2], [2, 1, 3]]
    w = B.gate_weights(l, idx, "softmax", True, 1.0)
    assert np.allclose(w[1], [1, 0, 0]) and np.allclose(w[2], 0) and np.allclose(w[3], [1, 0, 0])
    # a bias never brings a masked expert in front of an unmasked one
    idx, _ = B.gate_select(l, np.array([9.0, -9.0, 9.0, 9.0]), 1, "sigmoid")
    assert idx[1, 0] == 1
    # a group with one expert left counts what it has, a group without any is kept last
    idx, _ = B.gate_select(np.array([[-inf, -inf, 0.0, -inf]]), None, 2, "sigmoid", 2, 1, 2)
    assert idx.tolist() == [[2, 3]]


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_gradient_is_the_difference_quotient(name):
    rng = np.random.default_rng(5)
    x, w, b, dy = rng.normal(size=(4, 6)), rng.normal(size=(6, 5)), rng.normal(size=5), rng.normal(size=(4, 5))
    f = lambda x_, w_, b_: (B.linear_fwd(x_, w_, b_, None, name)[0] * dy).sum()
    _, pre = B.linear_fwd(x, w, b, None, name)
    dx, dw, db, _ = B.linear_bwd(dy, x, w, pre, name)
    for _ in range(3):
        p, q, r = rng.normal(size=x.shape), rng.normal(size=w.shape), rng.normal(size=5)
        assert np.isclose(central(lambda v: f(v, w, b), x, p), (dx * p).sum(), rtol=1e-6, atol=1e-7)
        assert np.isclose(central(lambda v: f(x, v, b), w, q), (dw * q).sum(), rtol=1e-6, atol=1e-7)
        assert np.isclose(central(lambda v: f(x, w, v), b, r), (db * r).sum(), rtol=1e-6, atol=1e-7)
