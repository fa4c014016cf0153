"""The norm, gate and linear operators on the GPU against their fp64 definitions."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from tests import block_checks as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- norm
NORM_SIZES = [(1, 1), (3, 2), (1, 2048), (5, 7), (33, 64), (130, 100), (40, 1111), (300, 2048), (37, 4096), (9, 8192),
              (65, 24), (3, 20000), (2, 65536), (700, 136), (2, 9999), (40, 12000)]


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,residual", [("layer", True), ("layer", False), ("rms", True), ("rms", False)])
def test_norm(T, H, dtype, kind, residual):
    c = C.norm_case(T, H, dtype, kind, residual, bias=kind == "layer", seed=T + H)
    C.check_norm_fwd(c, C.run_norm_fwd(c))
    mean, rstd = C.norm_stats(c)
    C.check_norm_bwd(c, mean, rstd, C.run_norm_bwd(c, mean=mean, rstd=rstd, dbias=kind == "layer"))


@pytest.mark.parametrize("T,H", [(2440, 64), (2500, 256), (2433, 504), (3000, 1000), (2432, 2048), (2600, 1544), (2450, 4096),
                                 (2435, 8192), (2441, 1023)])
@pytest.mark.parametrize("dtype,kind,residual", [("bf16", "layer", True), ("bf16", "rms", False), ("f32", "layer", False),
                                                 ("f32", "rms", True)])
def test_norm_several_rows_a_group(T, H, dtype, kind, residual):
    """Enough rows that every group of threads walks several, loads of later rows running ahead."""
    c = C.norm_case(T, H, dtype, kind, residual, bias=kind == "layer", seed=H)
    C.check_norm_fwd(c, C.run_norm_fwd(c))
    mean, rstd = C.norm_stats(c)
    C.check_norm_bwd(c, mean, rstd, C.run_norm_bwd(c, mean=mean, rstd=rstd, dbias=kind == "layer"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_many_rows(dtype):
    """More rows than any grid has blocks, narrow rows and the weight gradients over all of them."""
    c = C.norm_case(20011, 72, dtype, "layer", True, seed=1)
    C.check_norm_fwd(c, C.run_norm_fwd(c))
    mean, rstd = C.norm_stats(c)
    C.check_norm_bwd(c, mean, rstd, C.run_norm_bwd(c, mean=mean, rstd=rstd))


def test_norm_row_of_one_value_and_large_mean():
    """Rows without spread give the bias; a mean a thousand times the spread costs no digits of the variance."""
    c = C.norm_case(6, 512, "f32", "layer", False, seed=2, shift=1000.0)
    c["x"][0] = 3.0
    c["x"][1] = 0.0
    y, _, mean, rstd = C.run_norm_fwd(c)
    C.check_norm_fwd(c, (y, None, mean, rstd))
    assert torch.equal(y[1], c["b"])
    assert float(rstd[1]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)


@pytest.mark.parametrize("T,H", [(50, 2048), (50, 1111), (3, 20000), (2500, 2048), (2500, 512)])
def test_norm_in_place(T, H):
    """y over x and sum over residual; dx over dy, and over dsum."""
    c = C.norm_case(T, H, "bf16", "layer", True, seed=3)
    want = C.run_norm_fwd(c)
    d = _lib.make_norm_dims(T, H)
    x, r = c["x"].clone(), c["res"].clone()
    _lib.moe_norm_fwd(d, x, r, c["w"], c["b"], x, r, None, None)
    assert torch.equal(x, want[0]) and torch.equal(r, want[1])
    mean, rstd = C.norm_stats(c)
    dx, dw, db = C.run_norm_bwd(c, mean=mean, rstd=rstd)
    for name in ("dy", "dsum"):
        cc = dict(c, **{name: c[name].clone()})
        got = C.run_norm_bwd(cc, mean=mean, rstd=rstd, dx=cc[name])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_norm_gradient_is_the_difference_quotient():
    """The GPU backward against central differences of the GPU forward, in fp32."""
    c = C.norm_case(4, 96, "f32", "layer", True, seed=4, shift=0.0)
    y, s, mean, rstd = C.run_norm_fwd(c)
    dx, dw, db = C.run_norm_bwd(dict(c, x=s), mean=mean, rstd=rstd)
    r = C.rand(5)
    h = 2.0 ** -6  # the third derivative's h^2 and the rounding's 2^-24 / h are both near 1e-4 of the value

    def loss(**kw):
        yy, ss, _, _ = C.run_norm_fwd(dict(c, **kw))
        return float((yy.double() * c["dy"].double()).sum() + (ss.double() * c["dsum"].double()).sum())

    for name, g in (("x", dx), ("w", dw), ("b", db)):
        d = r(*c[name].shape)
        d = d / d.norm()
        q = (loss(**{name: c[name] + h * d}) - loss(**{name: c[name] - h * d})) / (2 * h)
        scale = float(g.double().norm())
        assert abs(q - float((g.double() * d.double()).sum())) < 2e-3 * scale, name


# ---------------------------------------------------------------- gate
GATES = [
    # T, E, k, groups, kept, take (tokens beside what one block and one cluster of blocks count: 32 x 8, 16 x 8, 8 x 8)
    (32, 128, 4, 1, 1, 1), (33, 128, 4, 1, 1, 1), (256, 64, 4, 1, 1, 1), (257, 64, 4, 1, 1, 1), (128, 256, 8, 8, 4, 2),
    (129, 256, 8, 8, 4, 2), (64, 1000, 8, 1, 1, 1), (65, 1000, 8, 1, 1, 1),
    (1, 1, 1, 1, 1, 1), (1, 128, 8, 1, 1, 1), (8, 128, 8, 1, 1, 1), (77, 8, 2, 1, 1, 1), (300, 160, 6, 8, 3, 1),
    (200, 256, 8, 8, 4, 2), (33, 33, 33 - 1, 1, 1, 1), (64, 512, 16, 4, 2, 2), (50, 60, 10, 4, 1, 2),
    (19, 1024, 32, 32, 5, 2), (100, 40, 5, 8, 1, 2), (40, 24, 7, 8, 4, 2), (513, 64, 4, 2, 2, 1), (9, 16, 16, 1, 1, 1),
    (21, 96, 3, 32, 2, 2), (30, 990, 9, 3, 2, 2), (40, 35, 4, 5, 2, 2), (70, 700, 12, 7, 3, 1), (25, 512, 16, 8, 1, 2),
]


@pytest.mark.parametrize("T,E,k,G,Kg,take", GATES)
@pytest.mark.parametrize("score,renorm,bias", [("softmax", True, False), ("softmax", False, True),
                                               ("sigmoid", True, True), ("sigmoid", False, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate(T, E, k, G, Kg, take, score, renorm, bias, dtype):
    r = C.rand(T + E + k)
    logits = r(T, E, scale=1.5, dtype=C.DT[dtype])
    b = torch.round(100 * r(E, scale=0.1)) * 1e-2 if bias else None
    out = C.run_gate(logits, b, k, score, renorm, 2.5, G, Kg, take)
    C.check_gate(logits, b, k, score, renorm, 2.5, out, G, Kg, take)
    dw = r(T, k)
    for gd in ("f32", "bf16"):
        dl = C.run_gate_bwd(logits, out[0], dw, score, renorm, 2.5, gd)
        C.check_gate_bwd(logits, out[0], dw, score, renorm, 2.5, dl)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_ties_go_to_the_lower_expert(score):
    """Logits of three values only: nearly every decision is a tie."""
    g = torch.Generator().manual_seed(1)
    logits = torch.randint(-1, 2, (200, 96), generator=g).float().cuda()
    for G, Kg in ((1, 1), (8, 3)):
        out = C.run_gate(logits, None, 8, score, True, 1.0, G, Kg, 2)
        C.check_gate(logits, None, 8, score, True, 1.0, out, G, Kg, 2, min_decided=1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_masks_infinities_and_nan(score, renorm):
    r = C.rand(8)
    logits = r(12, 64, scale=1.0)
    inf = float("inf")
    logits[0] = -inf                       # nothing left
    logits[1, 1:] = -inf                   # one expert left
    logits[2, 5:] = -inf                   # fewer than k left
    logits[3, ::2] = float("nan")          # half of them not numbers
    logits[4, 7] = inf
    logits[5, 7] = inf
    logits[5, 40] = inf
    logits[6] = torch.finfo(torch.float32).min
    logits[7, :60] = torch.finfo(torch.float32).min
    logits[8] = 1e4
    logits[9, :32] = -inf                  # whole groups masked
    b = torch.round(100 * r(64, scale=0.1)) * 1e-2
    b[3] = -inf
    for bias in (None, b):
        for G, Kg in ((1, 1), (8, 4)):
            out = C.run_gate(logits, bias, 8, score, renorm, 1.0, G, Kg, 2)
            C.check_gate(logits, bias, 8, score, renorm, 1.0, out, G, Kg, 2, min_decided=0.8)
            assert torch.isfinite(out[1]).all()
            dl = C.run_gate_bwd(logits, out[0], r(12, 8), score, renorm)
            assert torch.isfinite(dl).all()
            assert (dl[torch.isnan(logits) | (logits == -inf)] == 0).all()
            assert (dl[0] == 0).all()


def test_gate_bwd_skips_indices_out_of_range():
    r = C.rand(9)
    logits, dw = r(10, 32), r(10, 4)
    idx, _, _ = C.run_gate(logits, None, 4, "sigmoid", False)
    want = C.run_gate_bwd(logits, idx[:, :3].contiguous(), dw[:, :3].contiguous(), "sigmoid", False)
    for badv in (-1, 32, 2 ** 31 - 1, -2 ** 31):
        idx[:, 3] = badv
        assert torch.equal(C.run_gate_bwd(logits, idx, dw, "sigmoid", False), want)


# ---------------------------------------------------------------- linear
LINEAR_SIZES = [(1, 1, 1), (3, 1, 5), (1, 64, 64), (1, 2048, 768), (2, 100, 36), (4, 4096, 512), (5, 520, 129), (8, 768, 2048),
                (16, 264, 128), (17, 1001, 1111), (31, 128, 8), (33, 72, 200), (64, 512, 640), (65, 2048, 128),
                (128, 256, 512), (129, 130, 131), (256, 64, 1024), (257, 520, 264), (300, 768, 1000), (513, 16, 24),
                (777, 1001, 333), (1000, 136, 2056), (40, 3000, 7), (2, 8, 4104)]


@pytest.mark.parametrize("M,K,N", LINEAR_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act,bias,residual", [("none", True, True), ("gelu", True, False), ("silu", False, True)])
def test_linear(M, K, N, dtype, act, bias, residual):
    c = C.linear_case(M, K, N, dtype, act, bias, residual, seed=M + K + N)
    C.check_linear_fwd(c, C.run_linear_fwd(c, save=act != "none"))
    pre = C.linear_pre(c)
    C.check_linear_bwd(c, pre, C.run_linear_bwd(c, pre, db=bias))


@pytest.mark.parametrize("M,K,N,dtype,act", [(3, 8, 70001, "bf16", "silu"), (40, 16, 600008, "bf16", "none"),
                                             (17, 4, 70003, "f32", "relu")])
def test_linear_bias_gradient_of_many_columns(M, K, N, dtype, act):
    """More column blocks than there are counters."""
    c = C.linear_case(M, K, N, dtype, act, seed=17)
    pre = C.linear_pre(c)
    d, ws = C.linear_ws(c)
    for _ in range(2):  # the counters are back at zero after a call
        db = torch.full((N,), float("nan"), dtype=C.DT[dtype], device="cuda")
        _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], pre, None, None, db)
        C.check_linear_bwd(c, pre, (None, None, db))


@pytest.mark.parametrize("M,K,N", [(2048, 512, 2048), (2560, 256, 2048), (2300, 200, 4104), (1030, 520, 3001), (2100, 131, 2049)])
@pytest.mark.parametrize("act,bias,residual", [("gelu", True, True), ("none", False, False)])
def test_linear_many_tiles(M, K, N, act, bias, residual):
    """Outputs of several rounds of 256 x 256 tiles, ragged ones and a last round in half tiles among them."""
    c = C.linear_case(M, K, N, "bf16", act, bias, residual, seed=3)
    C.check_linear_fwd(c, C.run_linear_fwd(c, save=act != "none"))
    pre = C.linear_pre(c)
    C.check_linear_bwd(c, pre, C.run_linear_bwd(c, pre, db=bias))


@pytest.mark.parametrize("M,K,N,one", [(2080, 1096, 2312, True), (2048, 2048, 2048, True), (1024, 4096, 4096, True),
                                       (3000, 1800, 1032, False), (1288, 3400, 1600, True), (4096, 2048, 4096, False),
                                       (4096, 2048, 2048, True)])
def test_linear_both_products_in_one_launch(M, K, N, one):
    """dx and dw of middling products share a launch, the longer sum first whichever it is: the bits of two calls."""
    c = C.linear_case(M, K, N, "bf16", seed=5)
    add = C.rand(6)(M, K, dtype=torch.bfloat16)
    d, ws = C.linear_ws(c)
    new = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    dx, dw, dx1, dw1 = new(M, K), new(K, N), new(M, K), new(K, N)
    n = _lib.moe_kernel_launches()
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], None, dx, dw, dx_add=add)
    assert _lib.moe_kernel_launches() - n == (1 if one else 2)
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], None, dx1, dx_add=add)
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], None, None, dw1)
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    x, w, dy, r = (t.double() for t in (c["x"], c["w"], c["dy"], add))
    for got, want, mag, k in ((dx, dy @ w.T + r, dy.abs() @ w.abs().T + r.abs(), N),
                              (dw, x.T @ dy, x.abs().T @ dy.abs(), M)):
        tol = C.U["bf16"] * want.abs() + (k + 32) * 2 * C.E32 * mag
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("M,K,N", [(300, 768, 1000), (17, 256, 700), (333, 500, 257), (64, 1300, 70), (70, 65, 1300),
                                   (1, 512, 512), (1000, 64, 40)])
def test_linear_f32_gradients_of_unlike_products(M, K, N):
    """dx and dw in one launch, their tiles in different numbers of parts, the last cluster not full."""
    c = C.linear_case(M, K, N, "f32", "none", False, seed=9)
    n = _lib.moe_kernel_launches()
    out = C.run_linear_bwd(c, None, db=False)
    assert _lib.moe_kernel_launches() - n == 1
    C.check_linear_bwd(c, None, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N", [(2, 256, 320), (200, 96, 260), (384, 512, 256)])
def test_linear_other_activations_and_outputs(M, K, N, dtype, act):
    c = C.linear_case(M, K, N, dtype, act, True, True, seed=7)
    C.check_linear_fwd(c, C.run_linear_fwd(c, save=False))
    C.check_linear_fwd(c, C.run_linear_fwd(c, save=True))
    pre = C.linear_pre(c)
    full = C.run_linear_bwd(c, pre)
    C.check_linear_bwd(c, pre, full)
    for i in range(3):  # each gradient alone gives the same bits
        want = [i == j for j in range(3)]
        got = C.run_linear_bwd(c, pre, dx=want[0], dw=want[1], db=want[2])
        assert torch.equal(got[i], full[i]) and all(got[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("M,K,N", [(1, 2048, 128), (300, 256, 128), (4096, 2048, 128), (50, 333, 77), (256, 512, 1024)])
def test_linear_f32_output(M, K, N):
    """Router logits: bf16 products kept in fp32."""
    c = C.linear_case(M, K, N, "bf16", "none", False, False, out_f32=True, seed=11)
    C.check_linear_fwd(c, C.run_linear_fwd(c, save=False))


@pytest.mark.parametrize("M,K,N", [(3, 512, 384), (300, 264, 392), (130, 33, 77), (600, 512, 1024)])
def test_linear_result_over_the_residual(M, K, N):
    c = C.linear_case(M, K, N, "bf16", "silu", True, True, seed=12)
    want, _ = C.run_linear_fwd(c, save=False)
    res = C.f64(c["res"])
    y, _ = C.run_linear_fwd(c, save=False, y=c["res"])
    assert torch.equal(y, want)
    C.check_linear_fwd(c, (y, None), res=res)


@pytest.mark.parametrize("M,K,N,dtype", [(3, 512, 384, "bf16"), (1, 129, 64, "bf16"), (600, 520, 264, "bf16"),
                                         (500, 2048, 1000, "bf16"), (50, 60, 70, "f32")])
def test_linear_gradient_of_another_path(M, K, N, dtype):
    """dx_add joins dx before its one rounding, also where it is dx's own buffer."""
    c = C.linear_case(M, K, N, dtype, seed=15)
    add = C.rand(16)(M, K, dtype=C.DT[dtype])
    d, ws = C.linear_ws(c)
    dx = torch.full_like(add, float("nan"))
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], None, dx, dx_add=add)
    x, w, dy = (C.f64(c[n]) for n in ("x", "w", "dy"))
    want = dy @ w.T + C.f64(add)
    tol = C.U[dtype] * np.abs(want) + (N + 32) * 2 * C.E32 * (np.abs(dy) @ np.abs(w).T) + 2 * C.E32 * np.abs(C.f64(add))
    C.close(dx, want, tol, "dx")
    _lib.moe_linear_bwd(d, ws, c["dy"], c["x"], c["w"], None, add, dx_add=add)
    assert torch.equal(add, dx)


@pytest.mark.parametrize("M,K,N,dtype", [(3, 512, 384, "bf16"), (600, 520, 264, "bf16"), (300, 200, 100, "f32")])
def test_linear_gradient_is_the_difference_quotient(M, K, N, dtype):
    """<dy, y> moved along a direction, taken in 64 bits from the products of the inputs, against the gradients."""
    c = C.linear_case(M, K, N, dtype, "gelu", True, False, seed=13)
    pre = C.linear_pre(c)
    gx, gw, gb = C.run_linear_bwd(c, pre)
    from oracle import block_oracle as B
    x, w, b, dy = (C.f64(c[n]) for n in ("x", "w", "bias", "dy"))
    rng = np.random.default_rng(1)
    f = lambda x_, w_, b_: (B.linear_fwd(x_, w_, b_, None, "gelu")[0] * dy).sum()
    h = 1e-4
    for g, args in ((gx, 0), (gw, 1), (gb, 2)):
        base = [x, w, b]
        d = rng.normal(size=base[args].shape)
        hi, lo = list(base), list(base)
        hi[args], lo[args] = base[args] + h * d, base[args] - h * d
        q = (f(*hi) - f(*lo)) / (2 * h)
        G = C.f64(g)
        # independent roundings of every gradient entry (and of dz before it) add up like a random walk
        tol = 8 * (2 * C.U[dtype] + 1e-6) * np.sqrt(((G * d) ** 2).sum()) * (M ** 0.5) + 1e-4 * abs(q)
        assert abs(q - (G * d).sum()) < tol


@pytest.mark.parametrize("M,K,N", [(2, 512, 256), (700, 512, 768)])
def test_linear_infinities_and_nan_pass_through(M, K, N):
    """A NaN or infinity in one row of x reaches that row of y and no other."""
    c = C.linear_case(M, K, N, "bf16", "silu", True, False, seed=14)
    c["x"][1, 3] = float("nan")
    y, _ = C.run_linear_fwd(c, save=False)
    assert torch.isnan(y[1]).all()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.isfinite(y[keep]).all()


# ---------------------------------------------------------------- offsets past 32 bits
def _tail(t, n=3):
    return t[-n:].contiguous()


def test_norm_offsets_past_32_bits():
    T, H = 2_200_003, 1000  # 2.2e9 elements
    d = _lib.make_norm_dims(T, H)
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    w, b = C.rand(40)(H, dtype=torch.bfloat16), C.rand(41)(H, dtype=torch.bfloat16)
    y, m, r = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    _lib.moe_norm_fwd(d, x, None, w, b, y, None, m, r)
    c = dict(x=_tail(x), res=None, w=w, b=b, dtype="bf16", kind="layer", eps=1e-5)
    C.check_norm_fwd(c, (_tail(y), None, m[-3:], r[-3:]))
    dy = torch.zeros_like(x)
    dy[-3:] = C.rand(42)(3, H, dtype=torch.bfloat16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    _lib.moe_norm_bwd(d, _lib.alloc_norm_workspace(d), dy, None, x, w, m, r, dx, dw, db)
    c.update(T=3, H=H, dy=_tail(dy), dsum=None)
    C.check_norm_bwd(c, m[-3:], r[-3:], (_tail(dx), dw, db))
    assert float(dx[:-3].abs().max()) == 0.0


def test_gate_offsets_past_32_bits():
    T, E, k = 9_000_001, 248, 2  # 2.2e9 logits
    d = _lib.make_gate_dims(T, E, k, "softmax", True, grad_dtype="bf16")
    logits = torch.randn(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, cnt = torch.empty(T, k, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
    _lib.moe_gate_fwd(d, logits, None, idx, w, cnt)
    assert int(cnt.sum()) == T * k and torch.equal(cnt, torch.bincount(idx.flatten(), minlength=E).int())
    t, i = _tail(logits, 50), _tail(idx, 50)
    C.check_gate(t, None, k, "softmax", True, 1.0, (i, _tail(w, 50), torch.bincount(i.flatten(), minlength=E).int()))
    dw = torch.randn(T, k, device="cuda")
    dl = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    _lib.moe_gate_bwd(d, logits, idx, dw, dl)
    C.check_gate_bwd(t, i, _tail(dw, 50), "softmax", True, 1.0, _tail(dl, 50))


@pytest.mark.parametrize("N", [2048, 2050])
def test_linear_offsets_past_32_bits(N):
    M, K = 1_100_001, 64  # 2.25e9 outputs
    c = dict(M=3, K=K, N=N, dtype="bf16", act="relu", out_f32=False, x=torch.randn(M, K, device="cuda").bfloat16(),
             w=C.rand(43)(K, N, scale=0.1, dtype=torch.bfloat16), bias=C.rand(44)(N, dtype=torch.bfloat16),
             res=torch.randn(M, N, device="cuda", dtype=torch.bfloat16))
    d = _lib.make_linear_dims(M, K, N, "bf16", "relu")
    ws = _lib.alloc_linear_workspace(d)
    y, pre = torch.empty_like(c["res"]), torch.empty_like(c["res"])
    _lib.moe_linear_fwd(d, ws, c["x"], c["w"], c["bias"], c["res"], y, pre)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    t = dict(c, x=_tail(c["x"]), res=_tail(c["res"]))
    C.check_linear_fwd(t, (_tail(y), _tail(pre)))
    dy = torch.zeros_like(y)
    dy[-3:] = C.rand(45)(3, N, dtype=torch.bfloat16)
    dx, dw, db = torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["bias"])
    _lib.moe_linear_bwd(d, ws, dy, c["x"], c["w"], pre, dx, dw, db)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    C.check_linear_bwd(dict(t, dy=_tail(dy)), _tail(pre), (_tail(dx), dw, db))


# ---------------------------------------------------------------- all of them
def _everything(stream=None):
    n = C.norm_case(70, 512, "bf16", "layer", True, seed=20)
    l = C.linear_case(70, 512, 320, "bf16", "gelu", True, True, seed=21)
    s = C.linear_case(3, 1024, 640, "bf16", "none", True, True, seed=23)
    logits = C.rand(22)(70, 64)
    mean, rstd = C.norm_stats(n)
    pre = C.linear_pre(l)
    dw = C.rand(24)(70, 6)
    torch.cuda.synchronize()

    def go(st):
        out = list(C.run_norm_fwd(n, st)) + list(C.run_norm_bwd(n, st, mean, rstd))
        idx, w, cnt = C.run_gate(logits, None, 6, "sigmoid", True, 1.0, 8, 4, 2, stream=st)
        out += [idx, w, cnt, C.run_gate_bwd(logits, idx, dw, "sigmoid", True, stream=st)]
        out += list(C.run_linear_fwd(l, stream=st)) + list(C.run_linear_bwd(l, pre, stream=st))
        out += list(C.run_linear_fwd(s, save=False, stream=st))
        return [t for t in out if t is not None]

    return go


def test_same_bits_on_every_run_and_on_another_stream():
    go = _everything()
    a, b = go(None), go(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = go(side)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_cuda_graph_replay():
    """A forward and backward of each operator captured once and replayed on new inputs."""
    T, H, E, k, N = 96, 512, 64, 6, 384
    nd, ld = _lib.make_norm_dims(T, H), _lib.make_linear_dims(T, H, N, "bf16", "gelu")
    gd = _lib.make_gate_dims(T, E, k, "sigmoid", True, 1.0, 8, 4, 2)
    n = C.norm_case(T, H, "bf16", "layer", True, seed=30)
    l = C.linear_case(T, H, N, "bf16", "gelu", True, False, seed=31)
    logits = C.rand(32)(T, E)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    fl = lambda *s: torch.zeros(*s, device="cuda")
    it = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    nws, lws = _lib.alloc_norm_workspace(nd), _lib.alloc_linear_workspace(ld)
    o = dict(y=bf(T, H), s=bf(T, H), m=fl(T), r=fl(T), dx=bf(T, H), dw=bf(H), db=bf(H), z=bf(T, N), pre=bf(T, N),
             gx=bf(T, H), gw=bf(H, N), gb=bf(N), idx=it(T, k), w=fl(T, k), cnt=it(E), dl=fl(T, E))
    dy, dg = n["dy"], C.rand(33)(T, k)

    def step():
        _lib.moe_norm_fwd(nd, n["x"], n["res"], n["w"], n["b"], o["y"], o["s"], o["m"], o["r"])
        _lib.moe_linear_fwd(ld, lws, o["y"], l["w"], l["bias"], None, o["z"], o["pre"])
        _lib.moe_gate_fwd(gd, logits, None, o["idx"], o["w"], o["cnt"])
        _lib.moe_gate_bwd(gd, logits, o["idx"], dg, o["dl"])
        _lib.moe_linear_bwd(ld, lws, l["dy"], o["y"], l["w"], o["pre"], o["gx"], o["gw"], o["gb"])
        _lib.moe_norm_bwd(nd, nws, o["gx"], dy, o["s"], n["w"], o["m"], o["r"], o["dx"], o["dw"], o["db"])

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    n["x"].copy_(C.rand(34)(T, H))
    logits.copy_(C.rand(35)(T, E))
    g.replay()
    torch.cuda.synchronize()
    got = {a: b.clone() for a, b in o.items()}
    step()
    torch.cuda.synchronize()
    for a, b in o.items():
        assert torch.equal(got[a], b), a
    assert _lib.moe_read_status(lws) == _lib.MOE_OK
