"""The norm, gate and linear operators where fp32 runs out: scores that are denormal numbers, rows whose mean is large
against their spread, the far tails of the activations. Bounds follow from the arithmetic, with no slack that covers the
value itself."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from oracle import block_oracle as B
from tests import block_checks as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- gate
@pytest.mark.parametrize("k", [1, 2, 8])
def test_gate_gradient_of_denormal_sigmoid_scores(k):
    """Logits of -85 to -88.7: sigmoid scores down to 2^-128, whose reciprocal is past fp32's range. The renormalised
    weights and their gradients are ordinary numbers all the same."""
    T, E = 200, 16
    g = torch.Generator().manual_seed(k)
    logits = (-88.7 + 3.7 * torch.rand(T, E, generator=g)).cuda()
    logits[0, :], logits[1, :] = -88.7, -87.0
    dw = (4 * torch.randn(T, k, generator=g)).cuda()
    idx, w, _ = C.run_gate(logits, None, k, "sigmoid", True, 2.5)
    dl = C.run_gate_bwd(logits, idx, dw, "sigmoid", True, 2.5)
    l, i = C.f64(logits), idx.cpu().numpy().astype(np.int64)
    # a score of 2^-128 or more is a multiple of 2^-149 (2^-22 of it, half of that its rounding) with a few ulp of exp
    # and of a division: 2^-21. w carries it twice and one division; dl = w (dw - sum w dw) (1 - s) carries w's three
    # times, and the sums' roundings.
    e = 2.0 ** -19
    W = B.gate_weights(l, i, "sigmoid", True, 2.5)
    C.close(w, W, e * W, "topk_w")
    want = B.gate_bwd(l, i, C.f64(dw), "sigmoid", True, 2.5)
    mag = 2.5 * np.abs(C.f64(dw)).max(1, keepdims=True)
    dense = np.zeros((T, E))
    np.put_along_axis(dense, i, W / 2.5, 1)
    C.close(dl, want, 4 * e * dense * mag, "dlogits")


# ---------------------------------------------------------------- activations
E24 = 2.0 ** -24
TINY = 2.0 ** -126  # below it neither type has normal numbers: a factor that small may be flushed to zero
CT, AT = np.sqrt(2 / np.pi), 0.044715
EXACT_SIGMOID = lambda v: np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def phi_cap(z):
    """The normal distribution function, its lower tail to full relative accuracy."""
    return 0.5 * torch.special.erfc(torch.tensor(-z) / np.sqrt(2.0)).numpy()


def act64(name, z):
    """(act, act', the sum of the magnitudes of the terms act' is added up from)."""
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(float), (z > 0).astype(float)
    if name == "gelu":
        p, q = phi_cap(z), z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        return z * p, p + q, p + np.abs(q)
    u, du = (2 * CT * z * (1 + AT * z * z), 2 * CT * (1 + 3 * AT * z * z)) if name == "gelu_tanh" else (z, 1.0)
    s, t = EXACT_SIGMOID(u), EXACT_SIGMOID(-u)
    q = z * s * t * du
    return z * s, s + q, s + np.abs(q)


def rel64(name, z, fast):
    """Relative error of the distribution function or sigmoid that an activation is made of, in units of 2^-24.

    fp32: exp 2 ulp, erfc 4 ulp, an addition, a division and a product; the rounding of the argument counts as often as
    it grows through the function: z^2 + 1 times for erfc (twice), |u| times for the exponential (6 roundings for the
    tanh form). bf16: approximate exponential and reciprocal (2^-22 and 2^-23), two roundings of the exponent."""
    u = np.abs(2 * CT * z * (1 + AT * z * z)) if name == "gelu_tanh" else np.abs(z)
    if name == "relu":
        return 0 * z
    if name == "gelu":
        return 16 + 2 * z * z if not fast else 4e-6 / E24 + 40 + 2 * z * z
    n = 6 if name == "gelu_tanh" else 0
    return 10 + n * u if not fast else 32 + (n + 4) * u


def run_act(name, z, dtype, out_f32, M, K=8):
    """act(z) by a product that gives z exactly."""
    dt, N = C.DT[dtype], z.numel()
    x = torch.zeros(M, K, dtype=dt, device="cuda")
    w = torch.zeros(K, N, dtype=dt, device="cuda")
    x[:, 0], w[0] = 1.0, z
    c = dict(M=M, K=K, N=N, dtype=dtype, act=name, out_f32=out_f32, x=x, w=w, bias=None, res=None)
    y, pre = C.run_linear_fwd(c, save=True)
    assert torch.equal(pre, z.expand(M, N)) and torch.equal(y, y[:1].expand(M, N))
    return y[0]


def run_act_grad(name, z, dtype):
    """act'(z): the bias gradient of one row with dy = 1."""
    d, ws = C.linear_ws(dict(M=1, K=8, N=z.numel(), dtype=dtype, act=name, out_f32=False))
    one = lambda *s: torch.ones(*s, dtype=z.dtype, device="cuda")
    db = torch.full_like(z, float("nan"))
    _lib.moe_linear_bwd(d, ws, one(1, z.numel()), one(1, 8), one(8, z.numel()), z[None], None, None, db)
    return db


def grid(dtype, lo=-12.0, hi=12.0):
    return torch.unique(torch.linspace(lo, hi, 4003).to(C.DT[dtype]))[:4000].contiguous().cuda()


ACTS = ["relu", "gelu", "gelu_tanh", "silu"]


def act_tol(name, z, Y, fast, unit):
    return (rel64(name, z, fast) * E24 + unit) * np.abs(Y) + TINY * np.abs(z)


def check_act_grad(name, dtype):
    z = grid(dtype)
    got, zf, fast = run_act_grad(name, z, dtype), C.f64(z), dtype == "bf16"
    _, G, terms = act64(name, zf)
    du = 2 * CT * (1 + 3 * AT * zf * zf) if name == "gelu_tanh" else 1.0
    tol = (rel64(name, zf, fast) + 4) * E24 * terms + C.U[dtype] * np.abs(G) + TINY * (1 + np.abs(zf) * du)
    if name in ("gelu_tanh", "silu"):  # 1 - s is off by the rounding of an s near 1, times what multiplies it
        tol = tol + 8 * E24 * np.abs(zf) * du * EXACT_SIGMOID(zf)
    C.close(got, G, tol, name)


@pytest.mark.parametrize("act", ACTS)
def test_f32_activation_is_accurate_in_its_tails(act):
    z = grid("f32")
    zf = C.f64(z)
    Y = act64(act, zf)[0]
    for M in (1, 700):
        C.close(run_act(act, z, "f32", False, M), Y, act_tol(act, zf, Y, False, E24), act)
    check_act_grad(act, "f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,odd", [(1, 8, 0), (1, 8, 1), (300, 8, 1), (2100, 8, 0), (2100, 8, 1), (4096, 512, 0), (4096, 512, 1)])
def test_f32_output_of_bf16_products_has_f32_activations(act, M, K, odd):
    """Split products, tiles and tiles of CTA pairs, rows that are and are not multiples of 16 bytes."""
    z = grid("bf16")
    z = z[:len(z) // 8 * 8 - odd].contiguous()
    zf = C.f64(z)
    Y = act64(act, zf)[0]
    C.close(run_act(act, z, "bf16", True, M, K), Y, act_tol(act, zf, Y, False, E24), act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,odd", [(1, 8, 0), (2100, 8, 1), (4096, 512, 0)])
def test_bf16_activation_is_within_its_rounding(act, M, K, odd):
    """One rounding to bf16 (2^-8 of the value) and the fast forms' own small errors, in the tails as well."""
    z = grid("bf16")
    z = z[:len(z) // 8 * 8 - odd].contiguous()
    zf = C.f64(z)
    Y = act64(act, zf)[0]
    C.close(run_act(act, z, "bf16", False, M, K), Y, act_tol(act, zf, Y, True, C.U["bf16"] * (1 + 2.0 ** -10)), act)
    check_act_grad(act, "bf16")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activation_of_huge_finite_values(act, dtype):
    """Past the square root of fp32's range the activations are 0 and z, their derivatives 0 and 1."""
    z = torch.tensor([-3e38, -1e30, -1e20, -1e19, 1e19, 1e20, 1e30, 3e38], device="cuda").to(C.DT[dtype])
    assert torch.equal(run_act(act, z, dtype, False, 1), z.clamp_min(0))
    assert torch.equal(run_act_grad(act, z, dtype), (z > 0).to(z.dtype))


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("T,H", [(4, 512), (5, 1024), (4, 1111), (3, 2048), (4, 4100), (3, 20000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_gradient_at_a_large_mean(T, H, dtype):
    """Rows whose mean is 1000 times their spread, and rows of one value: x - mean is exact there (the two are within a
    factor of two), so xh is off by one rounding, however large the mean is."""
    c = C.norm_case(T, H, dtype, "layer", False, seed=H, shift=1000.0)
    c["x"][0], c["x"][1] = 1000.0, 3.0
    mean, rstd = C.norm_stats(c)
    mean[0], mean[1] = 1000.0, 3.0
    dx, dw, db = C.run_norm_bwd(c, mean=mean, rstd=rstd)
    x, w, dy, m, r = C.f64(c["x"]), C.f64(c["w"]), C.f64(c["dy"]), C.f64(mean), C.f64(rstd)
    DX, DW, DB = B.norm_bwd(dy, None, x, w, m, r, "layer")
    X = np.abs((x - m[:, None]) * r[:, None])
    # a column of dweight: xh's rounding and at most T products and sums; bf16 rounds the result
    u = C.U[dtype]
    C.close(dw, DW, u * np.abs(DW) + (T + 8) * E24 * (np.abs(dy) * X).sum(0), "dweight")
    C.close(db, DB, u * np.abs(DB) + (T + 8) * E24 * np.abs(dy).sum(0), "dbias")
    # a row's two means: sums over 32 elements a thread at most (80 in the longest rows), 5 steps in a warp, 16 warps
    g, n = np.abs(dy * w), 128 * E24
    C.close(dx, DX, u * np.abs(DX) + n * r[:, None] * (g + g.mean(1, keepdims=True) + X * (g * X).mean(1, keepdims=True)),
            "dx")


@pytest.mark.parametrize("T,H", [(4, 512), (4, 1111), (40, 2048), (2440, 512), (2433, 4096), (3, 20000)])
def test_norm_statistics_at_a_large_mean(T, H):
    """The variance is taken of h - mean, which is exact here: an error of the mean enters it squared, nothing else grows
    with the mean (a one-pass variance would be off by 2^-24 of the mean's square)."""
    c = C.norm_case(T, H, "f32", "layer", False, seed=H, shift=1000.0)
    _, _, mean, rstd = C.run_norm_fwd(c)
    _, h, M, R = B.norm_fwd(C.f64(c["x"]), None, C.f64(c["w"]), C.f64(c["b"]), "layer", c["eps"])
    n = 128 * E24
    d = n * np.abs(h).max(1)
    C.close(mean, M, d, "mean")
    C.close(rstd, R, (n + 0.5 * (d * R) ** 2) * R, "rstd")


# ---------------------------------------------------------------- workspaces
def test_linear_workspace_is_ready_for_any_stream():
    """The header is zero when the allocation returns, also behind work that the allocating stream still has to do, so
    that a first call on another stream finds its counters at zero."""
    d = _lib.make_linear_dims(256, 64, 512, "bf16", "silu")
    _lib.alloc_linear_workspace(d).fill_(0xFF)  # what the next allocation of this size gets back
    c = C.linear_case(256, 64, 512, "bf16", "silu", seed=50)
    pre = C.linear_pre(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    ws = _lib.alloc_linear_workspace(d)
    with torch.cuda.stream(side):
        head = ws[:4096].clone()
        out = C.run_linear_bwd(c, pre, stream=side, dws=(d, ws))
    side.synchronize()
    assert int(head.sum()) == 0
    C.check_linear_bwd(c, pre, out)


@pytest.mark.parametrize("shift,spread,steps", [(0.0, 4.0, 100), (-30.0, 0.5, 0), (-60.0, 0.1, 0)])
def test_gate_selects_on_fp32_scores(shift, spread, steps):
    """Sigmoid scores with a bias order the experts as 64 bits do wherever two choice scores differ by more than fp32's
    own roundings: exp 2 ulp (2^-22 of e^-l, which moves s by s (1 - s) times that), an addition and a reciprocal of
    one ulp (2^-24 and 2^-23 of s), and the sum with the bias (2^-24). Scores of e^-30 and e^-60 among them, which a
    bias of zero leaves as they are."""
    T, E, k = 100_000, 64, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = shift + spread * torch.randn(T, E, generator=g, device="cuda")
    bias = torch.randint(-steps, steps + 1, (E,), generator=g, device="cuda").float() * 1e-3
    idx, _, _ = C.run_gate(logits, bias, k, "sigmoid", True)
    s = torch.sigmoid(logits.double())
    c = s + bias.double()
    err = s * (1 - s) * 2.0 ** -22 + s * (2.0 ** -23 + E24) + c.abs() * E24
    want = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k + 1]
    cw, ew = c.gather(1, want), err.gather(1, want)
    # equal scores go to the lower expert, which the stable sort keeps
    gap = cw[:, :-1] - cw[:, 1:]
    decided = ((gap > ew[:, :-1] + ew[:, 1:]) | (gap == 0)).all(1)
    assert float(decided.float().mean()) > 0.9
    wrong = (idx.long() != want[:, :k]).any(1) & decided
    assert int(wrong.sum()) == 0
