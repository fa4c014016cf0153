"""The training operators at their largest sizes and where index arithmetic could run out."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from tests import train_checks as C
from tests.block_checks import E32, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def xent_on_gpu(M, H, V, tied, seed, dtype=torch.bfloat16):
    g = gen(seed)
    x = torch.randn(M, H, generator=g, device="cuda").to(dtype)
    w = torch.empty(V, H, dtype=dtype, device="cuda").normal_(0.0, H ** -0.5, generator=g)
    if not tied:
        w = w.t().contiguous()
    return x, w, torch.randint(0, V, (M,), generator=g, device="cuda").int()


def run_xent(x, w, target, tied, backward):
    M, H = x.shape
    V = w.shape[0] if tied else w.shape[1]
    d = _lib.make_xent_dims(M, H, V, "bf16" if x.dtype == torch.bfloat16 else "f32", tied)
    ws = _lib.alloc_xent_workspace(d, backward=backward)
    loss, lse, total = C.nan(M), C.nan(M), C.nan(2)
    _lib.moe_xent_fwd(d, ws, x, w, target, loss, lse, total)
    dx = dw = None
    if backward:
        dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
        _lib.moe_xent_bwd(d, ws, x, w, target, lse, None, total, dx, dw)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    return loss, lse, total, dx, dw


def check_rows(x, w, target, tied, loss, lse, dx, n, rows):
    """Some rows against 64 bits on the GPU: logits of about one, 2^-23 a step of the product and 2^-20 around it."""
    wd = w.double().t() if tied else w.double()
    xs = x[rows].double()
    l = xs @ wd
    want = torch.logsumexp(l, 1)
    H = x.shape[1]
    le = (H + 32) * 2 * E32 * float((xs.abs() @ wd.abs()).max())
    tol = le + (wd.shape[1] / 32 + 512) * E32 + 8 * E32 * float(want.abs().max())
    assert float((lse[rows].double() - want).abs().max()) < tol
    at = l.gather(1, target[rows].long()[:, None])[:, 0]
    assert float((loss[rows].double() - (want - at)).abs().max()) < 2 * tol
    if dx is not None:
        dl = torch.exp(l - want[:, None])
        dl[torch.arange(len(rows)), target[rows].long()] -= 1
        ref = dl @ wd.t() / n
        mag = (dl.abs() @ wd.abs().t()) / n
        err = (dx[rows].double() - ref).abs()
        # dl rounded to bf16 (2^-8 with its exponential's error), the sum over the vocabulary, the result rounded
        assert float((err - (2.0 ** -8 * ref.abs() + (1.1 * 2.0 ** -8 + 2 * tol + (wd.shape[1] + 64) * 2 * E32) * mag)).max()) < 0


@pytest.mark.parametrize("M,H,V,tied", [(270000, 16, 8300, True), (270000, 16, 8300, False), (70000, 8, 9, True),
                                        (70000, 8, 9, False), (20000, 64, 131072, False), (20000, 64, 131072, True)])
def test_xent_many_rows(M, H, V, tied):
    """Statistics of the vocabulary in several products, M V past 2^31, more rows than a grid's second axis holds."""
    x, w, target = xent_on_gpu(M, H, V, tied, M)
    loss, lse, total, dx, dw = run_xent(x, w, target, tied, True)
    rows = torch.cat([torch.arange(300), torch.randint(0, M, (300,)), torch.arange(M - 300, M)]).cuda()
    check_rows(x, w, target, tied, loss, lse, dx, M, rows)
    assert abs(float(total[0]) - float(loss.double().sum())) < 64 * E32 * float(loss.double().sum()) and float(total[1]) == M
    # columns of dw at the ends of the vocabulary and of pieces of it, from every row
    cols = [v for b in (0, 1024, 4096, 6656, V - 20) for v in range(max(0, b - 20), min(V, b + 20))]
    cols = torch.tensor(sorted(set(cols)), device="cuda")
    wc = (w[cols].t() if tied else w[:, cols]).double()
    dl = torch.exp(x.double() @ wc - lse.double()[:, None]) - (target[:, None] == cols[None, :]).double()
    ref, mag = x.double().t() @ dl / M, x.double().abs().t() @ dl.abs() / M
    got = (dw[cols].t() if tied else dw[:, cols]).double()
    # dl rounded to bf16 and off by its exponential's argument (10 x 2^-22), the sum over the rows, the result rounded
    assert float(((got - ref).abs() - 2.0 ** -8 * ref.abs() - (1.1 * 2.0 ** -8 + (M + 64) * 2 * E32) * mag).max()) < 1e-30
    # the columns of dw add up to sum_t x_t (sum_v dl_tv) = 0, each off by its rounding
    s = (dw.double().sum(0) if tied else dw.double().sum(1)).abs()
    mag = (dw.double().abs().sum(0) if tied else dw.double().abs().sum(1))
    assert float((s - 2.0 ** -7 * mag).max()) < 0 and torch.isfinite(dw).all()


@pytest.mark.parametrize("tied", [False, True])
def test_xent_weight_past_2_31_elements(tied):
    M, H, V = 3, 17000, 131072
    x, w, target = xent_on_gpu(M, H, V, tied, 1)
    target[0], target[1] = V - 1, 0
    loss, lse, total, dx, dw = run_xent(x, w, target, tied, True)
    l = torch.cat([x.double() @ (w[i:i + 8192].double().t() if tied else w[:, i:i + 8192].double())
                   for i in range(0, V, 8192)], 1)
    want = torch.logsumexp(l, 1)
    at = l.gather(1, target.long()[:, None])[:, 0]
    tol = (H + 32) * 2 * E32 * 4 * H ** 0.5 + 1e-3  # sums of 17000 products of one over its root
    assert float((lse.double() - want).abs().max()) < tol and float((loss.double() - want + at).abs().max()) < tol
    dl = torch.exp(l - want[:, None])
    dl[torch.arange(M), target.long()] -= 1
    dl /= M
    for lo in (0, V // 2, V - 1024):  # columns at both ends, past 2^31 elements in either layout
        ref = x.double().t() @ dl[:, lo:lo + 1024]
        mag = x.double().abs().t() @ dl[:, lo:lo + 1024].abs()
        got = dw[lo:lo + 1024].double().t() if tied else dw[:, lo:lo + 1024].double()
        assert float(((got - ref).abs() - 2.0 ** -8 * ref.abs() - (1.1 * 2.0 ** -8 + 2 * tol) * mag).max()) < 1e-30


def test_xent_f32_odd_in_a_graph():
    """Rows that are copied to a multiple of 16 bytes, their ends set to zero within the graph."""
    c = C.xent_case(70, 33, 2051, "f32", False, seed=2)
    d, ws = dws = C.xent_setup(c)
    fwd = C.run_xent_fwd(c, dws)
    ref = fwd + C.run_xent_bwd(c, fwd[1], c["dloss"], dws=dws)
    outs = [torch.empty_like(t) for t in ref]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _lib.moe_xent_fwd(d, ws, c["x"], c["w"], c["target"], *outs[:3])
        _lib.moe_xent_bwd(d, ws, c["x"], c["w"], c["target"], outs[1], c["dloss"], None, *outs[3:])
    ws[256:].fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, outs):
        assert torch.equal(a, b)


def test_balance_past_2_31_elements():
    T, E, k = 2_200_000, 1024, 2
    g = gen(3)
    logits = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    start = torch.tensor([0, 1_000_000, T], dtype=torch.int32, device="cuda")
    d = _lib.make_balance_dims(T, E, k, 2, "softmax", 0.5, 0.1, "bf16", "bf16")
    ws = _lib.alloc_balance_workspace(d)
    loss, count, prob = C.nan(2), torch.zeros(2, E, dtype=torch.int32, device="cuda"), C.nan(2, E)
    _lib.moe_balance_fwd(d, ws, logits, idx, start, loss, count, prob)
    dl = torch.full_like(logits, float("nan"))
    _lib.moe_balance_bwd(d, logits, count, start, None, None, dl)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK
    for s, (a, b) in enumerate(((0, 1_000_000), (1_000_000, T))):
        assert torch.equal(count[s].long(), torch.bincount(idx[a:b].flatten().long(), minlength=E))
        want = torch.zeros(E, dtype=torch.float64, device="cuda")
        for i in range(a, b, 100_000):
            want += torch.softmax(logits[i:min(b, i + 100_000)].double(), 1).sum(0)
        want /= b - a
        # 256 + 8 x 5 ulp of a score; a warp adds 460 or so of one sign, then trees
        assert float(((prob[s].double() - want).abs() / want).max()) < 1024 * E32
    rows = torch.arange(T - 64, T, device="cuda")
    p = torch.softmax(logits[rows].double(), 1)
    lse = torch.logsumexp(logits[rows].double(), 1, keepdim=True)
    co = 0.5 * E / (k * T) * count[1].double() / (T - 1_000_000)
    want = p * (co - p @ co[:, None] + 2 * 0.1 * lse / T)
    assert float(((dl[rows].double() - want).abs() - 2.0 ** -8 * want.abs() - 1024 * E32 * p * (2 * co.max() + 0.2 * lse.abs() / T)).max()) < 0


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_and_norm_past_2_31_elements(bits):
    n = 2 ** 31 + 1003
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    if bits == 8:
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        ms, vs = ([torch.zeros(-(-n // 256), device="cuda")] for _ in range(2))
    else:
        m, v, ms, vs = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), None, None
    at = torch.tensor([0, 255, 256, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, n - 2, n - 1], device="cuda")
    g[at] = torch.arange(1, 9, device="cuda").bfloat16()
    t = _lib.make_adamw_tensors([p], [g], [m], [v], None, ms, vs)
    norm = C.nan(1)
    _lib.moe_grad_norm(t, _lib.alloc_grad_norm_workspace(t), norm)
    assert abs(float(norm) - 204 ** 0.5) < 1e-5
    _lib.moe_adamw_step(_lib.make_adamw_dims(0.5, 0.9, 0.99, 1e-8, 1, bits), t)
    assert torch.equal(p[at], torch.full((8,), -0.5, dtype=torch.bfloat16, device="cuda"))  # a first step moves by lr
    p[at] = 0
    assert int(torch.count_nonzero(p)) == 0
    m = m.view(torch.uint8) if bits == 8 else m
    assert int(torch.count_nonzero(m[at])) == 8
    m[at] = 0
    assert int(torch.count_nonzero(m)) == 0
