"""fp64 definitions of the operators of a training step: balance loss, vocabulary cross entropy, AdamW.

Plain numpy on the CPU, one definition per function, sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- balance loss
def balance_probs(logits, score):
    """(p, lse): p = softmax, or sigmoids over their sum; masked logits (-inf, NaN) have p = 0."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    p, lse = np.zeros_like(l), np.full(len(l), -np.inf)
    for t in range(len(l)):
        ok = l[t] > -np.inf
        if not ok.any():
            continue
        m = l[t].max()
        if score == "softmax":
            if m == np.inf:
                p[t] = (l[t] == m) / (l[t] == m).sum()
                lse[t] = np.inf
                continue
            e = np.where(ok, np.exp(np.where(ok, l[t], m) - m), 0.0)
            p[t] = e / e.sum()
            lse[t] = m + np.log(e.sum())
        else:  # log sigma(l) = -log(1 + e^-l), relative to the largest
            ls = np.where(ok, -np.logaddexp(0.0, -np.where(ok, l[t], 0.0)), -np.inf)
            e = np.exp(ls - ls.max())
            p[t] = e / e.sum()
    return p, lse


def z_rows(lse):
    """Rows that have a z loss: those whose lse is an ordinary number (not the lowest value of a type, nor infinite)."""
    return np.abs(lse) < 9.2e18


def balance_spans(T, start):
    return [(0, T)] if start is None else list(zip(start[:-1], start[1:]))


def balance_fwd(logits, idx, start, score, alpha, z):
    """(loss[2], count[S, E], prob[S, E])."""
    T, E = logits.shape
    k = idx.shape[1]
    spans = balance_spans(T, start)
    N = max(1, spans[-1][1] - spans[0][0])
    p, lse = balance_probs(logits, score)
    count, prob = np.zeros((len(spans), E), np.int64), np.zeros((len(spans), E))
    loss = np.zeros(2)
    for s, (a, b) in enumerate(spans):
        for e in idx[a:b].ravel():
            if 0 <= e < E:
                count[s, e] += 1
        if b > a:
            prob[s] = p[a:b].mean(axis=0)
            loss[0] += alpha * (b - a) / N * np.sum(E * count[s] / (k * (b - a)) * prob[s])
            f = lse[a:b][z_rows(lse[a:b])]
            if score == "softmax":
                loss[1] += z / N * np.sum(f * f)
    return loss, count, prob


def balance_bwd(logits, count, start, k, score, alpha, z, u):
    T, E = logits.shape
    spans = balance_spans(T, start)
    N = max(1, spans[-1][1] - spans[0][0])
    p, lse = balance_probs(logits, score)
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    dl = np.zeros_like(p)
    for s, (a, b) in enumerate(spans):
        for t in range(a, b):
            c = alpha * E * count[s] / (k * N * (b - a))
            d = p[t] * (c - p[t] @ c)
            if score == "softmax":
                if z_rows(lse[t]):
                    d = d + 2 * z * lse[t] / N * p[t]
            else:
                with np.errstate(over="ignore"):
                    d = d / (1.0 + np.exp(l[t]))  # 1 - sigma
            dl[t] = u * d
    return dl


# ---------------------------------------------------------------- cross entropy
def xent_fwd(x, w, target, z):
    """(loss, lse, total, logits); w[H, V]; targets outside [0, V) are not counted."""
    l = x @ w
    m = l.max(axis=1)
    lse = m + np.log(np.exp(l - m[:, None]).sum(axis=1))
    ok = (target >= 0) & (target < l.shape[1])
    at = np.where(ok, target, 0)
    loss = np.where(ok, lse - l[np.arange(len(l)), at] + z * lse * lse, 0.0)
    return loss, lse, np.array([loss.sum(), ok.sum()]), l


def xent_bwd(x, w, target, z, d):
    """(dx, dw, dl) of sum_t d_t loss_t."""
    _, lse, _, l = xent_fwd(x, w, target, z)
    ok = (target >= 0) & (target < l.shape[1])
    d = np.where(ok, d, 0.0)
    dl = np.exp(l - lse[:, None]) * (1 + 2 * z * lse)[:, None] * d[:, None]
    dl[np.arange(len(l))[ok], target[ok]] -= d[ok]
    return dl @ w.T, x.T @ dl, dl


# ---------------------------------------------------------------- optimiser
def round_e4m3(u):
    """To the nearest value with 4 exponent and 3 mantissa bits (largest 448, smallest 2^-9), ties to even."""
    u = np.asarray(u, np.float64)
    mag = np.abs(u)
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6, 8)
    step = 2.0 ** (e - 3)
    return np.sign(u) * np.minimum(np.round(mag / step) * step, 448.0)


def quantise(x, root):
    """(codes as their values, scales) of blocks of 256; root: values above zero stay so."""
    n = len(x)
    b = np.zeros((-(-n // 256), 256))
    b.ravel()[:n] = x
    scale = np.maximum(np.abs(b).max(axis=1) / 448.0, 2.0 ** -126)
    q = round_e4m3(b / scale[:, None])
    if root:
        q = np.where((b > 0) & (q == 0), 2.0 ** -9, q)
    return q.ravel()[:n], scale


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, wd, factor):
    """(p, m, v) after a step on the gradient g * factor."""
    g = g * factor
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p - lr * (m / (1 - beta1 ** step) / (np.sqrt(v / (1 - beta2 ** step)) + eps) + wd * p)
    return p, m, v
