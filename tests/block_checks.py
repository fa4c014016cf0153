"""Runs of the norm, gate and linear operators beside their fp64 definitions, with error bounds.

Every bound is the operator's own arithmetic: one rounding of the result to its type (u = 2^-8 for bf16,
2^-24 for fp32), the growth of an fp32 sum (n 2^-24 of the sum of magnitudes; 2^-23 a step for tensor-core
products, whose adders may truncate), and a few ulp of the elementary functions.
"""
from __future__ import annotations

import numpy as np
import torch

from expert_grouped_gemm_gb300 import _lib
from oracle import block_oracle as B

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E32 = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    got = f64(got)
    assert np.isfinite(got).all() or not np.isfinite(want).all(), f"{what}: not finite"
    d = np.abs(got - want)
    bad = d > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, worst {np.max(d / (tol + 1e-300)):.2f} "
                           f"of it at {np.unravel_index(np.argmax(d - tol), d.shape)}")


def rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0, dtype=torch.float32: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()


# ---------------------------------------------------------------- norm
def norm_case(T, H, dtype, kind, residual, bias=True, seed=0, stats=True, shift=0.5, eps=1e-5):
    r = rand(seed)
    dt = DT[dtype]
    x = (r(T, H) * (1 + 10 * (torch.rand(H, generator=torch.Generator().manual_seed(seed)) < 0.02).float().cuda())
         + shift).to(dt)
    return dict(x=x, res=r(T, H, dtype=dt) if residual else None, w=(1 + 0.2 * r(H)).to(dt),
                b=r(H, scale=0.1, dtype=dt) if bias else None, dy=r(T, H, dtype=dt),
                dsum=r(T, H, dtype=dt) if residual else None, T=T, H=H, dtype=dtype, kind=kind, stats=stats, eps=eps)


def run_norm_fwd(c, stream=None):
    dt, T, H = DT[c["dtype"]], c["T"], c["H"]
    d = _lib.make_norm_dims(T, H, c["dtype"], c["kind"], c["eps"])
    nan = lambda *s, dtype=dt: torch.full(s, float("nan"), dtype=dtype, device="cuda")
    y = nan(T, H)
    s = nan(T, H) if c["res"] is not None else None
    mean = nan(T, dtype=torch.float32) if c["stats"] and c["kind"] == "layer" else None
    rstd = nan(T, dtype=torch.float32) if c["stats"] else None
    _lib.moe_norm_fwd(d, c["x"], c["res"], c["w"], c["b"], y, s, mean, rstd, stream=stream)
    return y, s, mean, rstd


def check_norm_fwd(c, out):
    y, s, mean, rstd = out
    u = U[c["dtype"]]
    Y, Hs, M, R = B.norm_fwd(f64(c["x"]), f64(c["res"]), f64(c["w"]), f64(c["b"]), c["kind"], c["eps"])
    n = 256 * E32
    big = np.abs(Hs).max(axis=1, keepdims=True)
    if c["res"] is not None:
        big = np.maximum(big, np.maximum(np.abs(f64(c["x"])), np.abs(f64(c["res"]))).max(axis=1, keepdims=True))
    w = np.abs(f64(c["w"]))
    # the deviation h - mean carries the rounding of values as large as `big`; the variance is that of such
    # deviations, so rstd is off by up to n (1 + big rstd)
    rel_r = n * (1 + big * R[:, None])
    tol = u * np.abs(Y) + n * (big * R[:, None] * w + (0 if c["b"] is None else np.abs(f64(c["b"])))) \
        + rel_r * np.abs(Hs - M[:, None]) * R[:, None] * w
    close(y, Y, tol, "y")
    if s is not None:
        close(s, Hs, u * np.abs(Hs) + 2 * E32 * big, "sum")
    if mean is not None:
        close(mean, M, n * big[:, 0], "mean")
    if rstd is not None:
        close(rstd, R, rel_r[:, 0] * R, "rstd")


def run_norm_bwd(c, stream=None, mean=None, rstd=None, dbias=True, dx=None):
    dt, T, H = DT[c["dtype"]], c["T"], c["H"]
    d = _lib.make_norm_dims(T, H, c["dtype"], c["kind"], c["eps"])
    ws = _lib.alloc_norm_workspace(d)
    ws.fill_(0xFF)
    nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
    dx = nan(T, H) if dx is None else dx
    dw, db = nan(H), nan(H) if dbias else None
    _lib.moe_norm_bwd(d, ws, c["dy"], c["dsum"], c["x"], c["w"], mean, rstd, dx, dw, db, stream=stream)
    return dx, dw, db


def norm_stats(c):
    """The statistics a forward of x would have saved (fp32)."""
    _, _, m, r = B.norm_fwd(f64(c["x"]), None, f64(c["w"]), None, c["kind"], c["eps"])
    t = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")
    return (t(m) if c["kind"] == "layer" else None), t(r)


def check_norm_bwd(c, mean, rstd, out, dy=None, dsum=None):
    dx, dw, db = out
    u = U[c["dtype"]]
    T, H = c["T"], c["H"]
    x, w = f64(c["x"]), f64(c["w"])
    dy = f64(c["dy"]) if dy is None else dy
    dsum = f64(c["dsum"]) if dsum is None else dsum
    m = f64(mean) if mean is not None else np.zeros(T)
    r = f64(rstd)
    DX, DW, DB = B.norm_bwd(dy, dsum, x, w, m, r, c["kind"])
    X = (np.abs(x) + np.abs(m)[:, None]) * r[:, None]  # bounds |xh| and, times an ulp, its rounding
    g = np.abs(dy * w)
    n = 256 * E32
    tol = u * np.abs(DX) + n * r[:, None] * (g + g.mean(1, keepdims=True) + X * (g * X).mean(1, keepdims=True))
    if dsum is not None:
        tol = tol + n * np.abs(dsum)
    close(dx, DX, tol, "dx")
    k = (T + 64) * E32
    close(dw, DW, u * np.abs(DW) + k * (np.abs(dy) * X).sum(0), "dweight")
    if db is not None:
        close(db, DB, u * np.abs(DB) + k * np.abs(dy).sum(0), "dbias")


# ---------------------------------------------------------------- gate
def run_gate(logits, bias, k, score, renorm, scale=1.0, n_group=1, topk_group=1, group_take=1, stream=None):
    T, E = logits.shape
    d = _lib.make_gate_dims(T, E, k, score, renorm, scale, n_group, topk_group, group_take,
                            "bf16" if logits.dtype == torch.bfloat16 else "f32")
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    cnt = torch.full((E,), -7, dtype=torch.int32, device="cuda")
    _lib.moe_gate_fwd(d, logits, bias, idx, w, cnt, stream=stream)
    return idx, w, cnt


def weight_tol(logits, want):
    l = f64(logits)
    span = np.abs(np.where(np.isfinite(l), l, 0.0)).max(axis=1, keepdims=True)
    return (64 + 4 * span) * E32 * np.abs(want) + 1e-38


def check_gate(logits, bias, k, score, renorm, scale, out, n_group=1, topk_group=1, group_take=1, min_decided=0.9):
    idx, w, cnt = (t.cpu().numpy() for t in out)
    want, gap = B.gate_select(f64(logits), f64(bias), k, score, n_group, topk_group, group_take)
    top = B.gate_scores(f64(logits), score)[1].max(axis=1) + (0.0 if bias is None else np.abs(f64(bias)[np.isfinite(f64(bias))]).max())
    decided = gap > 1e-6 * top  # elsewhere fp32 scores may order the experts either way
    assert decided.mean() >= min_decided
    assert np.array_equal(idx[decided], want[decided])
    assert ((idx >= 0) & (idx < logits.shape[1])).all()
    assert all(len(set(row)) == k for row in idx.tolist())
    assert np.array_equal(cnt, np.bincount(idx.ravel(), minlength=logits.shape[1]))
    W = B.gate_weights(f64(logits), idx.astype(np.int64), score, renorm, scale)
    close(out[1], W, weight_tol(logits, W), "topk_w")


def run_gate_bwd(logits, idx, dw, score, renorm, scale=1.0, grad_dtype="f32", stream=None):
    T, E = logits.shape
    d = _lib.make_gate_dims(T, E, idx.shape[1], score, renorm, scale, 1, 1, 1,
                            "bf16" if logits.dtype == torch.bfloat16 else "f32", grad_dtype)
    dl = torch.full((T, E), float("nan"), dtype=DT[grad_dtype], device="cuda")
    _lib.moe_gate_bwd(d, logits, idx, dw, dl, stream=stream)
    return dl


def check_gate_bwd(logits, idx, dw, score, renorm, scale, dl):
    u = U["bf16" if dl.dtype == torch.bfloat16 else "f32"]
    l, i, g = f64(logits), idx.cpu().numpy().astype(np.int64), f64(dw)
    want = B.gate_bwd(l, i, g, score, renorm, scale)
    # the terms of dl are products of scores of at most 1 with scale dw (over the chosen sum with renorm)
    _, s = B.gate_scores(l, score)
    sj = np.take_along_axis(s, i, 1)
    S = sj.sum(1, keepdims=True) if renorm else 1.0
    mag = np.abs(g).max(1, keepdims=True) * scale
    span = np.abs(np.where(np.isfinite(l), l, 0.0)).max(axis=1, keepdims=True)
    frac = np.divide(s, S, out=np.zeros_like(s), where=S > 0) if renorm else s
    tol = u * np.abs(want) + (64 + 4 * span) * 4 * E32 * mag * frac * (1 if renorm else i.shape[1]) + 1e-38
    close(dl, want, tol, "dlogits")


# ---------------------------------------------------------------- linear
def linear_case(M, K, N, dtype, act="none", bias=True, residual=False, out_f32=False, seed=0):
    r = rand(seed)
    dt = DT[dtype]
    return dict(M=M, K=K, N=N, dtype=dtype, act=act, out_f32=out_f32, x=r(M, K, dtype=dt),
                w=r(K, N, scale=K ** -0.5, dtype=dt), bias=r(N, scale=0.5, dtype=dt) if bias else None,
                res=r(M, N, dtype=dt) if residual else None, dy=r(M, N, dtype=dt))


def linear_ws(c):
    d = _lib.make_linear_dims(c["M"], c["K"], c["N"], c["dtype"], c["act"], c["out_f32"])
    ws = _lib.alloc_linear_workspace(d)
    ws[4096:].fill_(0xFF)
    return d, ws


def run_linear_fwd(c, save=True, stream=None, y=None, dws=None):
    d, ws = dws or linear_ws(c)
    dt = DT[c["dtype"]]
    if y is None:
        y = torch.full((c["M"], c["N"]), float("nan"), dtype=torch.float32 if c["out_f32"] else dt, device="cuda")
    pre = torch.full((c["M"], c["N"]), float("nan"), dtype=dt, device="cuda") if save else None
    _lib.moe_linear_fwd(d, ws, c["x"], c["w"], c["bias"], c["res"], y, pre, stream=stream)
    assert _lib.moe_read_status(ws, stream) == _lib.MOE_OK
    assert int(ws[:4096].sum()) == 0, "the header of the workspace is left at zero"
    return y, pre


def act_slack(dtype):
    return 4e-6 if dtype == "bf16" else 1e-6


def check_linear_fwd(c, out, res=None):
    y, pre = out
    u = U[c["dtype"]]
    x, w, b = f64(c["x"]), f64(c["w"]), f64(c["bias"])
    res = f64(c["res"]) if res is None else res
    Y, Z = B.linear_fwd(x, w, b, res, c["act"])
    z_err = (c["K"] + 32) * 2 * E32 * (np.abs(x) @ np.abs(w)) + 2 * E32 * np.abs(Z)
    if b is not None:
        z_err = z_err + 2 * E32 * np.abs(b)
    # no activation here is steeper than 1.13
    tol = (U["f32"] if c["out_f32"] else u) * np.abs(Y) + 1.13 * z_err + 2 * E32 * np.abs(Y)
    if c["act"] != "none":
        tol = tol + act_slack(c["dtype"]) * (1 + np.abs(Z))
    if res is not None:
        tol = tol + 2 * E32 * np.abs(res)
    close(y, Y, tol, "y")
    if pre is not None:
        close(pre, Z, u * np.abs(Z) + z_err, "pre")


def linear_pre(c):
    if c["act"] == "none":
        return None
    z = f64(c["x"]) @ f64(c["w"])
    return torch.tensor(z if c["bias"] is None else z + f64(c["bias"]), device="cuda").to(DT[c["dtype"]])


def run_linear_bwd(c, pre, stream=None, dx=True, dw=True, db=True, dws=None):
    d, ws = dws or linear_ws(c)
    dt = DT[c["dtype"]]
    nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
    gx = nan(c["M"], c["K"]) if dx else None
    gw = nan(c["K"], c["N"]) if dw else None
    gb = nan(c["N"]) if db else None
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], pre, gx, gw, gb, stream=stream)
    assert _lib.moe_read_status(ws, stream) == _lib.MOE_OK
    assert int(ws[:4096].sum()) == 0, "the header of the workspace is left at zero"
    return gx, gw, gb


def check_linear_bwd(c, pre, out):
    gx, gw, gb = out
    u = U[c["dtype"]]
    x, w, dy = f64(c["x"]), f64(c["w"]), f64(c["dy"])
    DX, DW, DB, DZ = B.linear_bwd(dy, x, w, f64(pre), c["act"])
    dz_act = np.zeros_like(DZ)
    dz_err = np.zeros_like(DZ)
    if c["act"] != "none":
        dz_act = act_slack(c["dtype"]) * np.abs(dy) * (2 + np.abs(f64(pre)))
        dz_err = dz_act + u * np.abs(DZ)  # dz is rounded for the two products
    a = np.abs(DZ) + dz_err
    if gx is not None:
        close(gx, DX, u * np.abs(DX) + (c["N"] + 32) * 2 * E32 * (a @ np.abs(w).T) + dz_err @ np.abs(w).T, "dx")
    if gw is not None:
        close(gw, DW, u * np.abs(DW) + (c["M"] + 32) * 2 * E32 * (np.abs(x).T @ a) + np.abs(x).T @ dz_err, "dw")
    if gb is not None:
        close(gb, DB, u * np.abs(DB) + (c["M"] + 64) * E32 * np.abs(DZ).sum(0) + dz_act.sum(0), "dbias")
