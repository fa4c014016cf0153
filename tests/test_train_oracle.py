"""Pins of the fp64 definitions of the training operators: autograd, differences, grids worked out by hand."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as O


@pytest.mark.parametrize("score,z", [("softmax", 0.0), ("softmax", 0.3), ("sigmoid", 0.0)])
def test_balance_gradient_by_differences(score, z):
    r = np.random.default_rng(0)
    T, E, k = 9, 6, 2
    l = r.normal(size=(T, E))
    idx = np.argsort(-l, axis=1)[:, :k]
    start = np.array([1, 1, 4, 8])
    _, count, _ = O.balance_fwd(l, idx, start, score, 0.7, z)
    dl = O.balance_bwd(l, count, start, k, score, 0.7, z, 1.5)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            d = (O.balance_fwd(a, idx, start, score, 0.7, z)[0].sum() - O.balance_fwd(b, idx, start, score, 0.7, z)[0].sum()) / (2 * h)
            assert abs(1.5 * d - dl[t, e]) < 1e-8
    assert np.all(dl[0] == 0) and np.all(dl[8] == 0) and np.all(count[0] == 0)


def test_balance_of_an_even_routing_is_alpha():
    T, E, k = 32, 8, 2
    idx = np.array([[(t * k + j) % E for j in range(k)] for t in range(T)])
    loss, count, prob = O.balance_fwd(np.zeros((T, E)), idx, None, "softmax", 0.25, 0.0)
    assert np.isclose(loss[0], 0.25) and np.all(count == T * k // E) and np.allclose(prob, 1 / E)


def test_balance_masks():
    l = np.array([[0.0, -np.inf, np.nan, 1.0], [-np.inf] * 4, [np.inf, 0.0, np.inf, 1.0]])
    p, lse = O.balance_probs(l, "softmax")
    assert np.allclose(p[0], [1 / (1 + np.e), 0, 0, np.e / (1 + np.e)]) and np.all(p[1] == 0)
    assert np.allclose(p[2], [0.5, 0, 0.5, 0]) and np.isneginf(lse[1]) and np.isposinf(lse[2])
    s, _ = O.balance_probs(np.array([[-800.0, -801.0]]), "sigmoid")
    assert np.allclose(s, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])


@pytest.mark.parametrize("z", [0.0, 0.01])
def test_xent_against_autograd(z):
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((7, 5), (5, 11)))
    target = torch.tensor([3, 0, 10, -100, 3, 7, 11])
    d = torch.rand(7, generator=g, dtype=torch.float64)
    l = x @ w
    ok = (target >= 0) & (target < 11)
    ce = torch.nn.functional.cross_entropy(l, torch.where(ok, target, 0), reduction="none")
    loss = torch.where(ok, ce + z * torch.logsumexp(l, 1) ** 2, 0.0)
    dx, dw = torch.autograd.grad((loss * d).sum(), (x, w))
    X, W = x.detach().numpy(), w.detach().numpy()
    got, lse, total, _ = O.xent_fwd(X, W, target.numpy(), z)
    assert np.allclose(got, loss.detach().numpy()) and total[1] == 5
    DX, DW, _ = O.xent_bwd(X, W, target.numpy(), z, d.numpy())
    assert np.allclose(DX, dx.numpy()) and np.allclose(DW, dw.numpy())


def test_adamw_against_torch():
    g = torch.Generator().manual_seed(2)
    p = torch.nn.Parameter(torch.randn(40, generator=g, dtype=torch.float64))
    opt = torch.optim.AdamW([p], lr=0.02, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    P, M, V = p.detach().numpy().copy(), np.zeros(40), np.zeros(40)
    for step in range(1, 6):
        p.grad = torch.randn(40, generator=g, dtype=torch.float64)
        P, M, V = O.adamw(P, p.grad.numpy(), M, V, 0.02, 0.8, 0.95, 1e-6, step, 0.3, 1.0)
        opt.step()
        assert np.allclose(P, p.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_e4m3_grid():
    """Every code's value stays; between two neighbours the nearer wins, ties go to the even one."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.round_e4m3(codes), codes) and codes[-1] == 448 and codes[1] == 2.0 ** -9
    mid = (codes[:-1] + codes[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, codes[:-1], codes[1:])
    assert np.array_equal(O.round_e4m3(mid), even)
    assert np.array_equal(O.round_e4m3(-mid * 1.001), -codes[1:]) and O.round_e4m3(500.0) == 448


def test_quantise_blocks():
    x = np.zeros(300)
    x[0], x[1], x[299] = 1.0, 1e-7, -2.0
    q, s = O.quantise(x, False)
    assert len(s) == 2 and q[0] == 448 and q[1] == 0 and q[299] == -448 and s[1] == 2.0 / 448
    q, s = O.quantise(np.abs(x), True)
    assert q[1] == 2.0 ** -9 and np.all(q[2:299] == 0)
    assert O.quantise(np.zeros(5), False)[1][0] == 2.0 ** -126
