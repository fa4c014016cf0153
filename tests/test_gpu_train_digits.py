"""Digits that a rounding of a shared factor, of a sum near one or of a large sum would cost the training operators."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from tests import train_checks as C
from tests.block_checks import E32, U, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- AdamW
@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (1e-5, 0.01), (1e-4, 0.1)])
@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_adamw_small_decay(lr, wd, bits, master):
    """A decay of 2e-8 to 1e-5 of a weight beside an update of some lr: each weight is off by its one rounding alone, and
    what they move by on average is not off at all."""
    n = 1 << 20
    c = C.adamw_case([n], "bf16" if master else "f32", "f32", master, bits, seed=21, lr=lr, wd=wd)
    w = 0.5 + 1.5 * torch.rand(n, generator=torch.Generator().manual_seed(23)).cuda()
    if master:
        c["master"][0].copy_(w)
        c["p"][0].copy_(w)
    else:
        c["p"][0].copy_(w)
    before = C.adamw_before(c)
    C.run_adamw(c)
    p, g, m, v = before[0]
    lr32, wd32 = float(np.float32(lr)), float(np.float32(wd))
    want = C.O.adamw(p, g, m, v, lr32, 0.9, 0.99, float(np.float32(1e-8)), 7, wd32, 1.0)[0]
    # the update's own roundings, as in check_adamw, and those of the decay: all relative to a part of the change
    mm = (0.9 * np.abs(m) + 0.1 * np.abs(g)) / (1 - 0.9 ** 7)
    den = np.sqrt((0.99 * v + 0.01 * g * g) / (1 - 0.99 ** 7)) + 1e-8
    part = 72 * E32 * lr * mm / den + 8 * E32 * lr * wd * np.abs(p)
    ulp = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64)
    ulp = np.maximum(ulp, np.spacing(np.abs(p).astype(np.float32)))  # at a power of two
    err = f64(c["p"][0] if not master else c["master"][0]) - want
    assert (np.abs(err) <= 0.5 * ulp + part).all()
    # 2^20 roundings of at most half a step h either way: their mean passes 0.0053 h with a chance of
    # 2 e^{-2^20 0.0053^2 / 2} = 8e-7 (Hoeffding's bound). The smallest decay is a sixth of a step and more.
    assert abs(err.mean()) <= 0.5 * ulp.max() * 0.0053 + part.mean()


@pytest.mark.parametrize("wd", [0.0, 0.1])
@pytest.mark.parametrize("bits,param,master", [(32, "f32", False), (32, "bf16", True), (32, "bf16", False), (8, "f32", False),
                                               (8, "bf16", True)])
def test_adamw_infinite_weights_stay(wd, bits, param, master):
    """Entries that a program has masked with an infinite weight keep it, with and without a decay, and the weights beside
    them are those of a step without such entries."""
    n = 1500
    c, ref = (C.adamw_case([n], param, "f32", master, bits, seed=24, wd=wd) for _ in range(2))
    at = torch.tensor([0, 1, 2, 3, 130, 257, 1023, n - 1], device="cuda")
    value = torch.tensor([-1, 1, -1, -1, 1, -1, -1, 1], device="cuda") * float("inf")
    for k in ("p", "master"):
        if c[k][0] is not None:
            c[k][0][at] = value.to(c[k][0].dtype)
    C.run_adamw(c)
    C.run_adamw(ref)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[at] = False
    for k in ("p", "master"):
        if c[k][0] is not None:
            assert torch.equal(c[k][0][at].float(), value) and torch.equal(c[k][0][others], ref[k][0][others])
    raw = lambda x: x.view(torch.uint8) if bits == 8 else x
    assert torch.equal(raw(c["m"][0]), raw(ref["m"][0])) and torch.equal(raw(c["v"][0]), raw(ref["v"][0]))


# ---------------------------------------------------------------- cross entropy
def likely_case(M, V, tied, z, seed):
    """Rows whose one target has a probability of 1 - 1e-2 to 1 - 1e-5: products of one sign make its logit, and the
    other logits are of about one."""
    H = 2048
    r = C.rand(seed)
    x = r(M, H).abs()
    w = r(V, H, scale=0.9 * H ** -0.5)
    t = V // 2 + 3
    w[t] = r(H).abs()
    x, w = x.bfloat16(), w.bfloat16()
    rest = torch.logsumexp((x.double() @ w.double().t())[:, torch.arange(V) != t], 1)
    want = rest + torch.linspace(4.6, 11.5, M, dtype=torch.float64).cuda()
    # the other features keep their sums: only the target's row of w is scaled, the rows' x by what is left
    w[t] = (w[t].double() * float((want / (x.double() @ w[t].double())).mean())).bfloat16()
    x = (x.double() * (want / (x.double() @ w[t].double()))[:, None]).bfloat16()
    return dict(M=M, H=H, V=V, dtype="bf16", tied=tied, z=z, x=x, w=w if tied else w.t().contiguous(),
                target=torch.full((M,), t, dtype=torch.int32, device="cuda"), dloss=0.5 + r(M).abs())


@pytest.mark.parametrize("M,V", [(12, 1000), (300, 1000), (300, 999), (700, 9000)])
@pytest.mark.parametrize("tied,z", [(False, 0.0), (True, 0.0), (False, 1e-4)])
def test_xent_gradient_of_likely_targets(M, V, tied, z):
    """dl of a target is the small difference of its probability and one: p - 1 = -(the others' share), in which the
    target's own logit has to be the one that lse was made of."""
    c = likely_case(M, V, tied, z, seed=M + V)
    loss, lse, _ = C.run_xent_fwd(c)
    x, w, t, l, le, LOSS, LSE, _, _ = C.xent_bounds(c)
    rows = np.arange(M)
    d = f64(c["dloss"])
    DX, DW, DL = C.O.xent_bwd(x, w, t, z, d)
    p = np.exp(l - LSE[:, None])
    others = p.copy()
    others[rows, t] = 0.0
    # The others' share: their logits' errors and exponentials; the sum that they join holds the target's 1 as well, whose
    # exponential is off by 2^-22 (4 units) and which up to 16 terms of a chunk, then chunks, lanes and slots are added to
    # (28). The target's logit is an fp32 sum of products of one sign, 8 a lane and then trees (32 steps).
    e_other = le + (256 + 8 * np.abs(l - LSE[:, None])) * E32
    e_at = 32 * E32 * np.abs(l[rows, t])
    share = (others * e_other).sum(1) + others.sum(1) * e_at + 48 * E32 * p[rows, t]
    close = C.close
    close(loss, LOSS, share / p[rows, t] + 2 * abs(z) * LSE * (e_at + share) + 16 * E32 * (LOSS + abs(z) * LSE ** 2), "loss")
    half = np.spacing(LSE.astype(np.float32)) / 2.0  # lse is handed on as a float
    f = 1 + 2 * z * np.abs(LSE)
    err = d[:, None] * f[:, None] * p * (e_other + half[:, None] + (e_at + share)[:, None])
    own = share + half + 8 * E32 * others.sum(1)  # of p - 1
    err[rows, t] = d * (own + 2 * abs(z) * (LSE * own + (e_at + share + half) + 16 * E32 * LSE))
    err = err + U["bf16"] * (np.abs(DL) + err) + d[:, None] * f[:, None] * 2.0 ** -126
    a = np.abs(DL) + err
    for mean in (False, True):
        if mean:  # the same with one factor for all rows
            c["dloss"] = None
            total = torch.tensor([0.0, 2.0], device="cuda")
            DX, DW, DL2 = C.O.xent_bwd(x, w, t, z, np.full(M, 0.5))
            scale = (0.5 / d)[:, None]
            err, a = err * scale, a * scale
        gx, gw = C.run_xent_bwd(c, lse, c["dloss"], total if mean else None)
        u = U["bf16"]
        close(gx, DX, u * np.abs(DX) + (V + 64) * 2 * E32 * (a @ np.abs(w).T) + err @ np.abs(w).T + 1e-37, "dx")
        got = gw.t() if tied else gw
        close(got, DW, u * np.abs(DW) + (M + 64) * 2 * E32 * (np.abs(x).T @ a) + np.abs(x).T @ err + 1e-37, "dw")


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e7, 1e9])
def test_xent_large_logits_of_one_sign(M, size):
    """Logits of -1e3 to -1e9, and targets that are the largest of their row: losses are finite and not below zero, and
    within what the logits are off."""
    H, V = 2048, 900
    r = C.rand(M)
    x, w = r(M, H).abs(), -(1 + 0.2 * r(V, H)).abs()
    s = (size / (0.8 * H)) ** 0.5
    x, w = (x * s).bfloat16(), (w * s).bfloat16()
    for sign in (1, -1):
        l = sign * (x.double() @ w.double().t())
        c = dict(M=M, H=H, V=V, dtype="bf16", tied=True, z=0.0, x=x, w=sign * w, target=l.argmax(1).int(), dloss=r(M))
        out = C.run_xent_fwd(c)
        assert torch.isfinite(out[0]).all() and float(out[0].min()) >= 0.0
        C.check_xent_fwd(c, out)
        if size <= 1e7:  # where a float still has the logits' units
            for t in C.run_xent_bwd(c, out[1], c["dloss"]):
                assert torch.isfinite(t).all()


# ---------------------------------------------------------------- far elements and odd rows
@pytest.mark.parametrize("tied", [False, True])
def test_xent_weight_past_2_31_elements_by_its_values(tied):
    """Few features are not zero, so sums are short and their bounds tight, and the columns that make the softmax lie past
    element 2^31 of w in either layout: whatever else is read changes every output by far more than its bound."""
    M, H, V = 3, 17000, 131072
    g = torch.Generator().manual_seed(5)
    x, w = torch.zeros(M, H, device="cuda"), torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    w.normal_(0.0, 0.05, generator=torch.Generator(device="cuda").manual_seed(6))
    cols = torch.randint(126400, V, (M, 6), generator=g)  # 126400 * 17000 > 2^31
    cols[0, 0] = V - 1
    at = []
    for t in range(M):  # half of a row's features below row 16384 of [H, V], which begins at element 2^31, half behind
        h = torch.cat([torch.randperm(16384, generator=g)[:32], 16384 + torch.randperm(H - 16384, generator=g)[:32]])
        h[0], h[32] = (0, H - 1) if t == 0 else (h[0], h[32])
        x[t, h.cuda()] = torch.sign(torch.randn(64, generator=g)).cuda()
        at.append(h)
    x = x.bfloat16()
    for t in range(M):  # logits of 12 to 14.5, from either half alike
        for j, v in enumerate(cols[t].tolist()):
            w[v, at[t].cuda()] = (x[t, at[t].cuda()].float() * (12 + 0.5 * j) / 64).bfloat16()
    target = cols[:, 2].int().cuda()
    target[1] = 7  # one that the softmax does not expect
    if not tied:
        w = w.t().contiguous()
    d = _lib.make_xent_dims(M, H, V, "bf16", tied)
    ws = _lib.alloc_xent_workspace(d)
    loss, lse, total = C.nan(M), C.nan(M), C.nan(2)
    _lib.moe_xent_fwd(d, ws, x, w, target, loss, lse, total)
    dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    _lib.moe_xent_bwd(d, ws, x, w, target, lse, None, total, dx, dw)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    l, xa = torch.empty(M, V, dtype=torch.float64, device="cuda"), 0.0
    xd = x.double()
    part = lambda i: (w[i:i + 8192].double().t() if tied else w[:, i:i + 8192].double())
    for i in range(0, V, 8192):
        l[:, i:i + 8192] = xd @ part(i)
        xa = max(xa, float((xd.abs() @ part(i).abs()).max()))
    want = torch.logsumexp(l, 1)
    le = 96 * 2 * E32 * xa  # 64 products that are not zero
    e = le + (V / 32 + 512) * E32
    assert e < 2e-3 and float((lse.double() - want).abs().max()) < e
    t64 = target.long()
    assert float((loss.double() - want + l.gather(1, t64[:, None])[:, 0]).abs().max()) < e + le
    dl = torch.exp(l - want[:, None])
    dl[torch.arange(M, device="cuda"), t64] -= 1
    dl /= M
    err = (2.0 ** -8 + 2 * e) * (dl.abs() + torch.exp(l - want[:, None]) * 2 * e / M) + 2 * e * torch.exp(l - want[:, None]) / M
    DX, mag, slack = (torch.zeros(M, H, dtype=torch.float64, device="cuda") for _ in range(3))
    for i in range(0, V, 8192):
        wi = part(i).t()
        DX += dl[:, i:i + 8192] @ wi
        mag += dl[:, i:i + 8192].abs() @ wi.abs()
        slack += err[:, i:i + 8192] @ wi.abs()
        # dw of these columns: rows of features that no x has are zero
        ref, tol = xd.t() @ dl[:, i:i + 8192], xd.abs().t() @ err[:, i:i + 8192]
        got = dw[i:i + 8192].double().t() if tied else dw[:, i:i + 8192].double()
        assert float(((got - ref).abs() - 2.0 ** -8 * ref.abs() - 1.01 * tol).max()) < 1e-30
    tol = 2.0 ** -8 * DX.abs() + slack + (V + 64) * 2 * E32 * mag
    assert float(((dx.double() - DX).abs() - tol).max()) < 0
    assert float(DX.abs().max()) > 10 * float(tol.max())


@pytest.mark.parametrize("tied", [False, True])
def test_xent_bf16_odd_rows_in_a_graph(tied):
    """Copies of odd rows of x and w, forward and backward, within a graph whose workspace is overwritten before its
    replay."""
    c = C.xent_case(70, 33, 2051, "bf16", tied, z=1e-3, seed=2)
    d, ws = dws = C.xent_setup(c)
    fwd = C.run_xent_fwd(c, dws)
    ref = fwd + C.run_xent_bwd(c, fwd[1], c["dloss"], dws=dws)
    C.check_xent_bwd(c, f64(c["dloss"]), ref[3:])
    outs = [torch.empty_like(t) for t in ref]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _lib.moe_xent_fwd(d, ws, c["x"], c["w"], c["target"], *outs[:3])
        _lib.moe_xent_bwd(d, ws, c["x"], c["w"], c["target"], outs[1], c["dloss"], None, *outs[3:])
    for _ in range(2):
        ws[256:].fill_(0xFF)
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, outs):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- 8-bit codes
@pytest.mark.parametrize("first", [2.0 ** -12, 1.0, 2.0 ** 20])
def test_adamw8_codes_of_rounded_roots_and_quotients(first):
    """With both betas zero m is the gradient and v its rounded square: the codes are those of the rounded root and of the
    rounded quotients by the stored scales, for every mantissa, bit for bit."""
    n = 1 << 24
    g = (np.arange(n, dtype=np.uint32) & 0x7FFFFF | (np.arange(n, dtype=np.uint32) >> 23) + 127 << 23).view(np.float32)
    g = g[np.random.default_rng(3).permutation(n)]
    g *= np.float32(first) * np.exp2(np.random.default_rng(4).integers(-9, 1, n)).astype(np.float32)  # within e4m3's span
    g[::2] *= -1
    zeros = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt, device="cuda")
    f8 = lambda: zeros(n, torch.uint8).view(torch.float8_e4m3fn)
    p, m, v, ms, vs = zeros(n), f8(), f8(), zeros(n // 256), zeros(n // 256)
    t = _lib.make_adamw_tensors([p], [torch.from_numpy(g).cuda()], [m], [v], None, [ms], [vs])
    _lib.moe_adamw_step(_lib.make_adamw_dims(0.1, 0.0, 0.0, 1e-8, 1, 8), t)
    for name, code, scale, x in (("m", m, ms, g), ("r", v, vs, np.sqrt(g * g))):
        q = (x.reshape(-1, 256) / scale.cpu().numpy()[:, None]).astype(np.float64)  # fp32 quotients
        want = C.O.round_e4m3(q)
        if name == "r":
            want = np.maximum(want, 2.0 ** -9)
        assert np.array_equal(f64(code).reshape(-1, 256), want), name


def test_optimiser_with_another_default_type():
    """lr on the device is fp32 whatever torch's default type is."""
    from expert_grouped_gemm_gb300.optim import AdamW

    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float64)
    try:
        p, g = (torch.ones(100, dtype=torch.float32, device="cuda") for _ in range(2))
        opt = AdamW([p], [g], 0.5, weight_decay=0.0, max_norm=100.0, capturable=True)
        opt.step()
    finally:
        torch.set_default_dtype(old)
    assert torch.equal(p, torch.full_like(p, 0.5)) or float((p - 0.5).abs().max()) < 1e-6
