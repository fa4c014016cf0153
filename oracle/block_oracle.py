"""fp64 definitions of the operators around the experts: norm, gate and linear.

Plain numpy on the CPU, one definition per function, sharing no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ---------------------------------------------------------------- norm
def norm_fwd(x, residual, weight, bias, kind, eps):
    """(y, h, mean, rstd) of y = (h - mean) rstd weight + bias, h = x + residual."""
    h = x if residual is None else x + residual
    mean = h.mean(axis=1) if kind == "layer" else np.zeros(len(h))
    rstd = 1.0 / np.sqrt(((h - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (h - mean[:, None]) * rstd[:, None] * weight
    return (y if bias is None else y + bias), h, mean, rstd


def norm_bwd(dy, dsum, h, weight, mean, rstd, kind):
    """(dx, dweight, dbias)."""
    xh = (h - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    dx = dx * rstd[:, None]
    return (dx if dsum is None else dx + dsum), (dy * xh).sum(axis=0), dy.sum(axis=0)


# ---------------------------------------------------------------- gate
def gate_scores(logits, score):
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    s = np.zeros_like(l)
    for t in range(len(l)):
        ok = l[t] > -np.inf
        if not ok.any():
            continue
        if score == "softmax":
            m = l[t].max()
            e = np.where(l[t] == m, 1.0, np.exp(np.where(ok, l[t], 0.0) - (m if np.isfinite(m) else 0.0)))
            if not np.isfinite(m):
                e = (l[t] == m).astype(np.float64)
            e = np.where(ok, e, 0.0)
            s[t] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s[t, ok] = 1.0 / (1.0 + np.exp(-l[t, ok]))
    return l, s


def gate_select(logits, bias, k, score, n_group=1, topk_group=1, group_take=1):
    """(idx, gap): the chosen experts and, per token, the smallest nonzero difference that the selection
    or the slot order rests on (differences of exactly zero are ties, which go to the lower index)."""
    l, s = gate_scores(logits, score)
    T, E = l.shape
    per = E // n_group
    idx = np.zeros((T, k), np.int64)
    gap = np.full(T, np.inf)

    def note(t, a, b):
        if np.isfinite(a) and np.isfinite(b) and a != b:
            gap[t] = min(gap[t], abs(a - b))

    for t in range(T):
        c = s[t] if bias is None else s[t] + bias
        c = np.where((l[t] == -np.inf) | np.isnan(c), -np.inf, c)
        groups = range(n_group)
        if topk_group < n_group:
            gs = []
            for g in range(n_group):
                top = sorted((v for v in c[g * per:(g + 1) * per] if v > -np.inf), reverse=True)[:group_take]
                gs.append(sum(top) if top else -np.inf)
            order = sorted(range(n_group), key=lambda g: (-gs[g], g))
            groups = order[:topk_group]
            note(t, gs[order[topk_group - 1]], gs[order[topk_group]])
        cand = [e for g in groups for e in range(g * per, (g + 1) * per)]
        cand.sort(key=lambda e: (-c[e], e))
        idx[t] = cand[:k]
        for j in range(min(k, len(cand) - 1)):
            note(t, c[cand[j]], c[cand[j + 1]])
    return idx, gap


def gate_weights(logits, idx, score, renorm, scale):
    l, s = gate_scores(logits, score)
    if renorm and score == "softmax":  # the softmax over the chosen logits
        s = np.stack([gate_scores(l[t:t + 1, idx[t]], score)[1][0] for t in range(len(l))])
        return s * scale
    w = np.take_along_axis(s, idx, axis=1)
    if renorm:
        S = w.sum(axis=1, keepdims=True)
        w = np.divide(w, S, out=np.zeros_like(w), where=S > 0)
    return w * scale


def gate_bwd(logits, idx, dw, score, renorm, scale):
    _, s = gate_scores(logits, score)
    dl = np.zeros_like(s)
    for t in range(len(s)):
        sj = s[t, idx[t]]
        d = dw[t] * scale
        if renorm:
            S = sj.sum()
            d = (d - (d * sj).sum() / S) / S if S > 0 else np.zeros_like(d)
        ds = np.zeros(s.shape[1])
        np.add.at(ds, idx[t], d)
        dl[t] = s[t] * (ds - (ds * s[t]).sum()) if score == "softmax" else ds * s[t] * (1.0 - s[t])
    return dl


# ---------------------------------------------------------------- linear
def act(name, z):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def act_grad(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        sg = 1.0 / (1.0 + np.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return np.ones_like(z)


def linear_fwd(x, w, bias, residual, name):
    z = x @ w
    if bias is not None:
        z = z + bias
    y = act(name, z)
    return (y if residual is None else y + residual), z


def linear_bwd(dy, x, w, pre, name):
    """(dx, dw, dbias, dz)."""
    dz = dy if name == "none" else dy * act_grad(name, pre)
    return dz @ w.T, x.T @ dz, dz.sum(axis=0), dz
