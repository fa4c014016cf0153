"""Runs of the balance, cross entropy, norm and AdamW operators beside their fp64 definitions, with error bounds.

Bounds are the operators' own arithmetic: one rounding of a result to its type (u = 2^-8 for bf16, 2^-24 for fp32),
the growth of an fp32 sum (2^-24 a step; 2^-23 for tensor-core products, whose adders may truncate), a few ulp of the
elementary functions, and the rounding of an exponent's argument (its size times 2^-24).
"""
from __future__ import annotations

import numpy as np
import torch

from expert_grouped_gemm_gb300 import _lib
from oracle import train_oracle as O
from tests.block_checks import DT, E32, U, close, f64, rand


def i64(t):
    return None if t is None else t.cpu().numpy().astype(np.int64)


def nan(*s, dtype=torch.float32):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


# ---------------------------------------------------------------- balance
def balance_case(T, E, k, start=None, score="softmax", z=0.0, dtype="f32", grad_dtype="f32", add=False, alpha=0.3, seed=0,
                 spread=2.0):
    r = rand(seed)
    g = torch.Generator().manual_seed(seed + 1)
    logits = r(T, E, scale=spread, dtype=DT[dtype])
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    return dict(T=T, E=E, k=k, S=0 if start is None else len(start) - 1, score=score, z=z, dtype=dtype,
                grad_dtype=grad_dtype, alpha=alpha, logits=logits, idx=idx,
                start=None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda"),
                add=r(T, E, scale=1e-3, dtype=DT[grad_dtype]) if add else None)


def balance_dims(c):
    return _lib.make_balance_dims(c["T"], c["E"], c["k"], c["S"], c["score"], c["alpha"], c["z"], c["dtype"], c["grad_dtype"])


def run_balance_fwd(c, stream=None, ws=None, prob=True):
    d = balance_dims(c)
    if ws is None:
        ws = _lib.alloc_balance_workspace(d)
        ws[256:].fill_(0xFF)
    S = max(c["S"], 1)
    loss, p = nan(2), nan(S, c["E"]) if prob else None
    count = torch.full((S, c["E"]), -7, dtype=torch.int32, device="cuda")
    _lib.moe_balance_fwd(d, ws, c["logits"], c["idx"], c["start"], loss, count, p, stream=stream)
    assert _lib.moe_read_status(ws, stream) == _lib.MOE_OK
    assert int(ws[:256].sum()) == 0, "the header of the workspace is left at zero"
    return loss, count, p


def finite_span(l):
    """The largest argument of an exponential that is not zero: e^-104 rounds to zero in fp32."""
    f = np.where(np.isfinite(l), l, 0.0)
    return np.minimum(np.abs(f).max(axis=1, keepdims=True), 104.0)


def check_balance_fwd(c, out):
    loss, count, prob = out
    l = f64(c["logits"])
    L, N, P = O.balance_fwd(l, i64(c["idx"]), i64(c["start"]), c["score"], c["alpha"], c["z"])
    assert np.array_equal(i64(count), N)
    span = finite_span(l).max()
    rel = (128 + 8 * span + c["T"] + c["E"]) * E32  # a score, then sums of terms of one sign
    if prob is not None:
        close(prob, P, rel * P + 1e-37, "prob")
    lse = O.balance_probs(l, c["score"])[1]
    big = np.abs(lse[O.z_rows(lse)]).max(initial=0.0)
    zerr = abs(c["z"]) * (2 * big * (128 + 8 * span) * E32 * (1 + big)) + rel * L[1]
    close(loss, L, np.array([2 * rel * abs(L[0]), abs(zerr)]) + 1e-37, "loss")


def run_balance_bwd(c, count, dloss=None, stream=None, out=None):
    dl = nan(c["T"], c["E"], dtype=DT[c["grad_dtype"]]) if out is None else out
    _lib.moe_balance_bwd(balance_dims(c), c["logits"], count, c["start"], dloss, c["add"], dl, stream=stream)
    return dl


def check_balance_bwd(c, count, dl, up=1.0, add=None):
    l = f64(c["logits"])
    n = i64(count).astype(np.float64)
    want = O.balance_bwd(l, n, i64(c["start"]), c["k"], c["score"], c["alpha"], c["z"], up)
    p, lse = O.balance_probs(l, c["score"])
    spans = O.balance_spans(c["T"], i64(c["start"]))
    N = max(1, spans[-1][1] - spans[0][0])
    mag = np.zeros_like(p)  # the terms that cancel
    for s, (a, b) in enumerate(spans):
        if b > a:
            co = c["alpha"] * c["E"] * n[s] / (c["k"] * N * (b - a))
            z = np.abs(2 * c["z"] * np.where(O.z_rows(lse[a:b]), lse[a:b], 0.0) / N)[:, None]
            mag[a:b] = p[a:b] * (co + (p[a:b] @ co)[:, None] + z)
    tol = (256 + 16 * finite_span(l) + c["E"]) * E32 * mag * abs(up)
    add = f64(c["add"]) if add is None else add
    if add is not None:
        want = want + add
        tol = tol + 2 * E32 * np.abs(add)
    close(dl, want, tol + U[c["grad_dtype"]] * np.abs(want) + 1e-37, "dlogits")


# ---------------------------------------------------------------- cross entropy
def xent_case(M, H, V, dtype="bf16", tied=False, z=0.0, seed=0, drop=0.2, peak=3.0):
    r = rand(seed)
    g = torch.Generator().manual_seed(seed + 1)
    dt = DT[dtype]
    w = r(V, H, scale=H ** -0.5)
    target = torch.randint(0, V, (M,), generator=g).int()
    x = r(M, H) + peak * w[target.long().cuda()]
    target[torch.rand(M, generator=g) < drop] = -100
    target[0] = V - 1
    w = w.to(dt)
    return dict(M=M, H=H, V=V, dtype=dtype, tied=tied, z=z, x=x.to(dt), w=w if tied else w.t().contiguous(),
                target=target.cuda(), dloss=r(M))


def xent_setup(c, backward=True):
    d = _lib.make_xent_dims(c["M"], c["H"], c["V"], c["dtype"], c["tied"], c["z"])
    ws = _lib.alloc_xent_workspace(d, backward=backward)
    ws[256:].fill_(0xFF)
    return d, ws


def run_xent_fwd(c, dws=None, stream=None, total=True, status=_lib.MOE_OK):
    d, ws = dws or xent_setup(c, backward=False)
    loss, lse, tot = nan(c["M"]), nan(c["M"]), nan(2) if total else None
    _lib.moe_xent_fwd(d, ws, c["x"], c["w"], c["target"], loss, lse, tot, stream=stream)
    assert _lib.moe_read_status(ws, stream) == status
    assert int(ws[:256].sum()) == 0, "the header of the workspace is left at zero"
    return loss, lse, tot


def xent_bounds(c):
    """(x, w[H,V], target, logits' errors, lse's errors) in 64 bits."""
    x, w = f64(c["x"]), f64(c["w"])
    w = w.T if c["tied"] else w
    le = (c["H"] + 32) * 2 * E32 * (np.abs(x) @ np.abs(w))
    loss, lse, total, l = O.xent_fwd(x, w, i64(c["target"]), c["z"])
    # p's shares of the logits' errors, the exponentials (2^-22 and the rounding of their arguments), their sum
    e_lse = le.max(1) + (c["V"] / 32 + 256 + 8 * (l.max(1) - l.min(1))) * E32 + 4 * E32 * np.abs(lse)
    return x, w, i64(c["target"]), l, le, loss, lse, total, e_lse


def check_xent_fwd(c, out):
    loss, lse, tot = out
    x, w, t, l, le, LOSS, LSE, TOT, e = xent_bounds(c)
    close(lse, LSE, e, "lse")
    at = np.clip(t, 0, c["V"] - 1)
    rows = np.arange(len(t))
    tol = e * (1 + 2 * abs(c["z"]) * np.abs(LSE)) + le[rows, at] + 8 * E32 * (np.abs(LSE) + np.abs(l[rows, at]) + abs(c["z"]) * LSE ** 2)
    tol = np.where((t >= 0) & (t < c["V"]), tol, 0.0)
    close(loss, LOSS, tol, "loss")
    if tot is not None:
        close(tot, TOT, np.array([tol.sum() + (c["M"] + 8) * E32 * np.abs(LOSS).sum(), 0.0]), "total")


def run_xent_bwd(c, lse, dloss=None, total=None, dws=None, stream=None, dx=True, dw=True, status=_lib.MOE_OK):
    d, ws = dws or xent_setup(c)
    dt = DT[c["dtype"]]
    gx = nan(c["M"], c["H"], dtype=dt) if dx else None
    gw = torch.full_like(c["w"], float("nan")) if dw else None
    _lib.moe_xent_bwd(d, ws, c["x"], c["w"], c["target"], lse, dloss, total, gx, gw, stream=stream)
    assert _lib.moe_read_status(ws, stream) == status
    assert int(ws[:256].sum()) == 0, "the header of the workspace is left at zero"
    return gx, gw


def check_xent_bwd(c, d, out):
    gx, gw = out
    x, w, t, l, le, _, lse, _, e = xent_bounds(c)
    u = U[c["dtype"]]
    DX, DW, DL = O.xent_bwd(x, w, t, c["z"], d)
    ok = (t >= 0) & (t < c["V"])
    dd = np.where(ok, np.abs(d), 0.0)[:, None]
    p = np.exp(l - lse[:, None])
    f = np.abs(1 + 2 * c["z"] * lse)[:, None]
    rel = le + e[:, None] + (64 + 8 * np.abs(l - lse[:, None])) * E32
    err = dd * p * (f * rel + 2 * abs(c["z"]) * e[:, None]) + 4 * E32 * dd * (p * f)
    hit = np.zeros_like(p)
    hit[np.arange(len(t))[ok], t[ok]] = 1.0
    err = err + 4 * E32 * dd * hit
    if c["dtype"] == "bf16":
        err = err + u * np.abs(DL)  # dl is rounded for the two products
        # Exponentials below the smallest normal float are zero there (the hardware's base-2 exponential flushes): p is
        # off by at most p < 2^-126, so dl = d f p by at most d f 2^-126 whatever p is, and that is multiplied by x and w.
        err = err + dd * f * 2.0 ** -126
    a = np.abs(DL) + err
    if gx is not None:
        close(gx, DX, u * np.abs(DX) + (c["V"] + 64) * 2 * E32 * (a @ np.abs(w).T) + err @ np.abs(w).T + 1e-37, "dx")
    if gw is not None:
        got = gw.t() if c["tied"] else gw
        close(got, DW, u * np.abs(DW) + (c["M"] + 64) * 2 * E32 * (np.abs(x).T @ a) + np.abs(x).T @ err + 1e-37, "dw")


# ---------------------------------------------------------------- AdamW
def adamw_case(sizes, param="f32", grad="f32", master=False, bits=32, seed=0, lr=0.01, beta1=0.9, beta2=0.99, eps=1e-8,
               step=7, wd=0.1, gscale=1.0):
    r = rand(seed)
    c = dict(sizes=sizes, bits=bits, lr=lr, beta1=beta1, beta2=beta2, eps=eps, step=step, wd=wd)
    c["master"] = [r(n, scale=0.1) if master else None for n in sizes]
    c["p"] = [(r(n, scale=0.1) if t is None else t).to(DT[param]) for n, t in zip(sizes, c["master"])]
    c["g"] = [r(n, scale=gscale).to(DT[grad]) for n in sizes]
    m, v = [r(n, scale=0.3 * gscale) for n in sizes], [(gscale * (0.2 + r(n).abs())) ** 2 for n in sizes]
    c["ms"] = c["vs"] = None
    if bits == 8:
        def pack(x, root):
            q, s = O.quantise(f64(x), root)
            return (torch.tensor(q, device="cuda").to(torch.float8_e4m3fn), torch.tensor(s, dtype=torch.float32, device="cuda"))
        (m, c["ms"]), (v, c["vs"]) = zip(*[pack(t, False) for t in m]), zip(*[pack(t.sqrt(), True) for t in v])
    c["m"], c["v"] = list(m), list(v)
    return c


def adamw_before(c):
    """(p, g, m, v) of each tensor in 64 bits."""
    out = []
    for i, n in enumerate(c["sizes"]):
        m, v = f64(c["m"][i]), f64(c["v"][i])
        if c["bits"] == 8:
            rep = lambda s: np.repeat(f64(s), 256)[:n]
            m, v = m * rep(c["ms"][i]), (v * rep(c["vs"][i])) ** 2
        out.append((f64(c["p"][i] if c["master"][i] is None else c["master"][i]), f64(c["g"][i]), m, v))
    return out


def run_adamw(c, max_norm=0.0, norm=None, grad_scale=1.0, lr=None, step=None, stream=None, lr_scale=1.0):
    t = _lib.make_adamw_tensors(c["p"], c["g"], c["m"], c["v"], c["master"], c["ms"], c["vs"], c["wd"], lr_scale)
    d = _lib.make_adamw_dims(c["lr"], c["beta1"], c["beta2"], c["eps"], c["step"], c["bits"], max_norm, grad_scale)
    _lib.moe_adamw_step(d, t, norm, lr, step, stream=stream)


def check_adamw(c, before, factor=1.0, lr=None, step=None):
    b1, b2, eps = c["beta1"], c["beta2"], float(np.float32(c["eps"]))
    lr, step = float(np.float32(c["lr"])) if lr is None else lr, c["step"] if step is None else step
    wds = c["wd"] if isinstance(c["wd"], list) else [c["wd"]] * len(c["sizes"])
    for i, (p, g, m, v) in enumerate(before):
        wd = float(np.float32(wds[i]))
        P, M, V = O.adamw(p, g, m, v, lr, b1, b2, eps, step, wd, factor)
        mm = b1 * np.abs(m) + (1 - b1) * np.abs(g * factor)  # what cancels in m
        bc1, bc2 = 1 - b1 ** step, 1 - b2 ** step
        den = np.sqrt(V / bc2) + eps
        # the float betas are off by 2^-25, their complements too; v's terms have one sign
        tm = 8 * E32 * mm + 1e-44
        tv = 16 * E32 * V + 1e-44
        tp = 4 * E32 * np.abs(p) + lr * (64 * E32 * mm / bc1 / den + 8 * E32 * wd * np.abs(p)) + lr * tm / bc1 / den
        at = f"tensor {i}: "
        out = c["p"][i] if c["master"][i] is None else c["master"][i]
        u = U["bf16"] if out.dtype == torch.bfloat16 else U["f32"]
        close(out, P, tp + u * np.abs(P), at + "weight")
        if c["master"][i] is not None:
            assert torch.equal(c["p"][i], c["master"][i].bfloat16())
        if c["bits"] == 32:
            close(c["m"][i], M, tm, at + "m")
            close(c["v"][i], V, tv, at + "v")
            continue
        n = len(p)
        for name, X, tol, root in (("m", M, tm, False), ("v", np.sqrt(V), 16 * E32 * np.sqrt(V) + 1e-37, True)):
            blocks = lambda x: np.pad(x, (0, -n % 256)).reshape(-1, 256)
            S = np.maximum(np.abs(blocks(X)).max(1) / 448, 2.0 ** -126)
            ts = blocks(tol).max(1) / 448 + 4 * E32 * S
            s = c[name + "s"][i]
            close(s, S, ts, at + name + " scale")
            # the stored code is a nearest one of the value over the stored scale, within what the value is off
            q, rep = f64(c[name][i]), np.repeat(f64(s), 256)[:n]
            U8 = X / rep
            off = np.abs(U8) * 4 * E32 + tol / rep
            lo, hi = O.round_e4m3(U8 - off), O.round_e4m3(U8 + off)
            if root:
                lo, hi = (np.where(X > 0, np.maximum(t, 2.0 ** -9), t) for t in (lo, hi))
            bad = (q < lo) | (q > hi)
            assert not bad.any(), f"{at}{name}: {int(bad.sum())} codes are not the nearest, {q[bad][:4]} for {U8[bad][:4]}"
