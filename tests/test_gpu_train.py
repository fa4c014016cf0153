"""Balance loss, vocabulary cross entropy, gradient norm and AdamW on the GPU against their fp64 definitions."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from expert_grouped_gemm_gb300.optim import AdamW
from tests import train_checks as C
from tests.block_checks import DT, E32, f64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- balance
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 5, 2), (64, 128, 8), (65, 33, 3), (300, 256, 8), (1000, 64, 6),
                                   (37, 1024, 32), (2433, 100, 4), (5000, 8, 2)])
@pytest.mark.parametrize("score,z", [("softmax", 0.0), ("softmax", 0.01), ("sigmoid", 0.0)])
def test_balance(T, E, k, score, z):
    dt, gt = ("bf16", "f32") if T % 2 else ("f32", "bf16")
    c = C.balance_case(T, E, k, None, score, z, dt, gt, add=T % 3 == 0, seed=T + E)
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    C.check_balance_bwd(c, out[1], C.run_balance_bwd(c, out[1]))


@pytest.mark.parametrize("start", [[0, 100], [0, 0, 100], [3, 3, 40, 41, 41, 90], [10, 10], [0, 1, 2, 3, 50, 50, 100, 100],
                                   list(range(0, 101)), [100, 100, 100]])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_sequences(start, score):
    """Empty sequences, sequences of one token, tokens before the first and behind the last."""
    c = C.balance_case(100, 48, 3, start, score, 0.02 if score == "softmax" else 0.0, "f32", "f32", add=True, seed=len(start))
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    dl = C.run_balance_bwd(c, out[1])
    C.check_balance_bwd(c, out[1], dl)
    outside = torch.ones(100, dtype=torch.bool)
    outside[start[0]:start[-1]] = False
    assert torch.equal(dl[outside.cuda()], c["add"][outside.cuda()])


@pytest.mark.parametrize("S", [37, 3000])
def test_balance_many_sequences(S):
    g = torch.Generator().manual_seed(S)
    cut = torch.sort(torch.randint(0, 9001, (S - 1,), generator=g)).values.tolist()
    c = C.balance_case(9100, 24, 2, [0] + cut + [9000], "softmax", 0.0, "bf16", "bf16", seed=3)
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    C.check_balance_bwd(c, out[1], C.run_balance_bwd(c, out[1]))


@pytest.mark.parametrize("T,S", [(1, 1), (1, 2), (1, 3), (2, 3), (1, 5000), (7, 7), (17, 2), (17, 3), (64, 4), (64, 16),
                                 (64, 5000), (128, 3), (128, 40), (128, 128), (130, 300)])
def test_balance_few_tokens_in_sequences(T, S):
    """From one sequence to far more than tokens: runs of empty ones before, between and behind the others."""
    g = torch.Generator().manual_seed(T * 10007 + S)
    at = torch.randint(0, min(T, 9) + 1, (S - 1,), generator=g) * T // min(T, 9)
    c = C.balance_case(T, 40, 3, [0] + torch.sort(at).values.tolist() + [T], "softmax", 0.02, "f32", "f32", seed=S)
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    C.check_balance_bwd(c, out[1], C.run_balance_bwd(c, out[1]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_balance_masks_and_extremes(score, dtype):
    c = C.balance_case(40, 64, 4, None, score, 0.5 if score == "softmax" else 0.0, dtype, "f32", seed=5)
    l = c["logits"]
    l[0] = -INF
    l[1] = NAN
    l[2, ::2] = -INF
    l[3, 5:] = NAN
    l[4] = torch.finfo(l.dtype).min
    l[5, 1:] = torch.finfo(l.dtype).min
    l[6] = -100.0
    l[7] = -100.0 - torch.arange(64).cuda()
    l[8] = 90.0
    l[9, :2] = 80.0
    l[10] = -300.0
    c["idx"][11, 0] = -1
    c["idx"][12, 1] = 64
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    dl = C.run_balance_bwd(c, out[1])
    C.check_balance_bwd(c, out[1], dl)
    assert torch.all(dl[:2] == 0) and torch.all(dl[2, ::2] == 0) and torch.all(dl[3, 5:] == 0)


def test_balance_infinite_logits():
    c = C.balance_case(20, 16, 2, None, "softmax", 0.1, seed=6)
    c["logits"][3, 4] = INF
    c["logits"][4, 2:5] = INF
    out = C.run_balance_fwd(c)
    C.check_balance_fwd(c, out)
    assert torch.isfinite(out[0]).all() and torch.isfinite(C.run_balance_bwd(c, out[1])).all()


def test_balance_bad_offsets_are_reported():
    c = C.balance_case(50, 16, 2, [0, 30, 20, 50], seed=7)
    d = C.balance_dims(c)
    ws = _lib.alloc_balance_workspace(d)
    loss, count = C.nan(2), torch.zeros(3, 16, dtype=torch.int32, device="cuda")
    for start in ([0, 30, 20, 50], [-5, 10, 20, 50], [0, 10, 20, 51], [2 ** 31 - 1, -2 ** 31, 7, 2 ** 31 - 1]):
        st = torch.tensor(start, dtype=torch.int32, device="cuda")
        _lib.moe_balance_fwd(d, ws, c["logits"], c["idx"], st, loss, count)
        assert _lib.moe_read_status(ws) == _lib.MOE_ERR_DEVICE_ARG
        _lib.moe_balance_bwd(d, c["logits"], count, st, None, None, torch.empty_like(c["logits"]))
    torch.cuda.synchronize()


def test_balance_gradient_scale_place_and_differences():
    c = C.balance_case(60, 32, 4, [0, 25, 60], "softmax", 0.05, seed=8)
    out = C.run_balance_fwd(c)
    up = torch.tensor([-2.5], device="cuda")
    C.check_balance_bwd(c, out[1], C.run_balance_bwd(c, out[1], up), up=-2.5)
    # into the buffer of the gradient it is added to
    c["add"] = torch.randn(60, 32, device="cuda") * 1e-3
    add = f64(c["add"])
    C.check_balance_bwd(c, out[1], C.run_balance_bwd(c, out[1], None, out=c["add"]), add=add)
    c["add"] = None
    dl = f64(C.run_balance_bwd(c, out[1]))
    # a difference of the operator's own losses along a direction
    v = torch.randn(60, 32, device="cuda")
    h = 2.0 ** -6
    base = c["logits"]
    ends = []
    for s in (h, -h):
        c["logits"] = base + s * v
        ends.append(f64(C.run_balance_fwd(c)[0]).sum())
    want = (dl * f64(v)).sum()
    # losses of about 0.6 and 2 to 2^-18, and the third derivative's h^2
    assert abs((ends[0] - ends[1]) / (2 * h) - want) < 1e-3 * max(1.0, abs(want))


def test_balance_graphs_streams_and_bits():
    c = C.balance_case(4000, 128, 8, [0, 1000, 1001, 4000], "softmax", 0.01, seed=9)
    ref = C.run_balance_fwd(c)
    for _ in range(3):
        for a, b in zip(ref, C.run_balance_fwd(c)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for a, b in zip(ref, C.run_balance_fwd(c, stream=side)):
        assert torch.equal(a, b)
    d = C.balance_dims(c)
    ws = _lib.alloc_balance_workspace(d)
    outs = [[torch.empty_like(t) for t in ref] for _ in range(2)]
    graphs = []
    for o in outs:  # two graphs that share a workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.moe_balance_fwd(d, ws, c["logits"], c["idx"], c["start"], *o)
        graphs.append(g)
    for _ in range(3):
        for o, g in zip(outs, graphs):
            for t in o:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(ref, o):
                assert torch.equal(a, b)
    a, b, e = (C.run_balance_bwd(c, ref[1]) for _ in range(3))
    assert torch.equal(a, b) and torch.equal(a, e)
    assert C.run_balance_fwd(c, prob=False)[2] is None


# ---------------------------------------------------------------- cross entropy
SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 7), (1, 64, 1000), (8, 256, 4096), (17, 72, 999), (64, 128, 129), (65, 33, 2050),
         (130, 200, 1001), (200, 320, 5000), (300, 64, 257), (513, 136, 776), (40, 1024, 12345)]


@pytest.mark.parametrize("M,H,V", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tied", [False, True])
def test_xent(M, H, V, dtype, tied):
    c = C.xent_case(M, H, V, dtype, tied, z=0.01 if (M + H + V) % 2 else 0.0, seed=M + V)
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    C.check_xent_bwd(c, f64(c["dloss"]), C.run_xent_bwd(c, out[1], c["dloss"]))
    mean = np.full(M, 1.0 / f64(out[2])[1])
    C.check_xent_bwd(c, mean, C.run_xent_bwd(c, out[1], None, out[2]))


@pytest.mark.parametrize("M,V", [(600, 70000), (2100, 20000), (5000, 9000), (16, 140000)])
@pytest.mark.parametrize("tied", [False, True])
def test_xent_many_columns(M, V, tied):
    """Many tiles of the vocabulary, ragged last ones, K in parts (pieces of it: test_gpu_train_edges.py)."""
    c = C.xent_case(M, 40, V, "bf16", tied, z=1e-3, seed=M)
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    C.check_xent_bwd(c, f64(c["dloss"]), C.run_xent_bwd(c, out[1], c["dloss"]))


@pytest.mark.parametrize("tied", [False, True])
def test_xent_several_pieces_f32(tied):
    c = C.xent_case(5000, 24, 8000, "f32", tied, seed=4)
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    C.check_xent_bwd(c, f64(c["dloss"]), C.run_xent_bwd(c, out[1], c["dloss"]))


@pytest.mark.parametrize("M,H,V", [(1, 64, 50257), (17, 100, 30001), (300, 24, 70001), (3, 5, 9000)])
@pytest.mark.parametrize("tied", [False, True])
def test_xent_f32_few_tiles_of_a_long_vocabulary(M, H, V, tied):
    """dx in parts of the vocabulary, in one piece and (300 rows) in two of different lengths."""
    c = C.xent_case(M, H, V, "f32", tied, seed=11)
    out = C.run_xent_fwd(c)
    both = C.run_xent_bwd(c, out[1], c["dloss"])
    C.check_xent_bwd(c, f64(c["dloss"]), both)
    assert torch.equal(C.run_xent_bwd(c, out[1], c["dloss"], dw=False)[0], both[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_one_output_only(dtype):
    c = C.xent_case(70, 96, 700, dtype, seed=5)
    out = C.run_xent_fwd(c)
    both = C.run_xent_bwd(c, out[1], c["dloss"])
    gx, none = C.run_xent_bwd(c, out[1], c["dloss"], dw=False)
    assert none is None and torch.equal(gx, both[0])
    none, gw = C.run_xent_bwd(c, out[1], c["dloss"], dx=False)
    assert none is None and torch.equal(gw, both[1])
    assert C.run_xent_fwd(c, total=False)[2] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_rows_that_are_not_counted(dtype):
    c = C.xent_case(50, 64, 300, dtype, seed=6)
    c["target"][:] = -1
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    for t in C.run_xent_bwd(c, out[1], None, out[2]):
        assert torch.all(t == 0)
    # a target past the vocabulary is reported and not counted
    c["target"][3], c["target"][4], c["target"][5] = 300, 2 ** 31 - 1, 7
    out = C.run_xent_fwd(c, status=_lib.MOE_ERR_DEVICE_ARG)
    C.check_xent_fwd(c, out)
    assert f64(out[2])[1] == 1
    C.check_xent_bwd(c, np.where(np.arange(50) == 5, 1.0, 0.0), C.run_xent_bwd(c, out[1], None, out[2]))
    # rows without weight stay at zero whatever their logits are
    c["target"][:] = 5
    c["x"][7] = INF
    lse = C.run_xent_fwd(c)[1]
    c["dloss"][7] = 0.0
    gx, _ = C.run_xent_bwd(c, lse, c["dloss"])
    assert torch.all(gx[7] == 0)


def test_xent_nan_and_infinite_rows_stay_alone():
    c = C.xent_case(40, 64, 500, "bf16", seed=7, drop=0.0)
    ref = C.run_xent_fwd(c)
    c["x"][11, 3] = NAN
    got = C.run_xent_fwd(c)
    others = torch.arange(40, device="cuda") != 11
    assert torch.isnan(got[0][11]) and torch.isnan(got[1][11])
    assert torch.equal(got[0][others], ref[0][others]) and torch.equal(got[1][others], ref[1][others])


def test_xent_large_logits():
    """Logits of a few hundred: exponentials of their differences to the largest alone, lse as exact as they are."""
    c = C.xent_case(60, 128, 2000, "bf16", seed=8)
    c["x"].mul_(64)
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    C.check_xent_bwd(c, f64(c["dloss"]), C.run_xent_bwd(c, out[1], c["dloss"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_same_target_in_every_row(dtype):
    c = C.xent_case(300, 72, 900, dtype, seed=9)
    c["target"][:] = 899
    out = C.run_xent_fwd(c)
    C.check_xent_fwd(c, out)
    C.check_xent_bwd(c, f64(c["dloss"]), C.run_xent_bwd(c, out[1], c["dloss"]))


def test_xent_gradient_by_differences():
    c = C.xent_case(20, 24, 150, "f32", z=0.02, seed=10)
    out = C.run_xent_fwd(c)
    gx, gw = C.run_xent_bwd(c, out[1], c["dloss"])
    base = {n: c[n] for n in ("x", "w")}
    for name, g in (("x", gx), ("w", gw)):
        v = torch.randn_like(base[name])
        h = 2.0 ** -8
        ends = []
        for s in (h, -h):
            c[name] = base[name] + s * v
            ends.append((f64(C.run_xent_fwd(c)[0]) * f64(c["dloss"])).sum())
        c[name] = base[name]
        want = (f64(g) * f64(v)).sum()
        assert abs((ends[0] - ends[1]) / (2 * h) - want) < 4e-3 * max(1.0, np.abs(f64(g) * f64(v)).sum())


def test_xent_graphs_streams_and_bits():
    c = C.xent_case(300, 256, 6000, "bf16", seed=11)
    d, ws = dws = C.xent_setup(c)
    ref = C.run_xent_fwd(c, dws) + C.run_xent_bwd(c, C.run_xent_fwd(c, dws)[1], c["dloss"], dws=dws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    fwd = C.run_xent_fwd(c, dws, stream=side)
    for a, b in zip(ref, fwd + C.run_xent_bwd(c, fwd[1], c["dloss"], dws=dws, stream=side)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    outs = [[torch.empty_like(t) for t in ref] for _ in range(2)]
    graphs = []
    for loss, lse, tot, gx, gw in outs:  # two graphs that share a workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.moe_xent_fwd(d, ws, c["x"], c["w"], c["target"], loss, lse, tot)
            _lib.moe_xent_bwd(d, ws, c["x"], c["w"], c["target"], lse, c["dloss"], None, gx, gw)
        graphs.append(g)
    for _ in range(2):
        for o, g in zip(outs, graphs):
            for t in o:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(ref, o):
                assert torch.equal(a, b)
    assert _lib.moe_read_status(ws) == _lib.MOE_OK


def test_calls_at_once_on_two_streams():
    """The same calls on two streams with workspaces of their own, nothing waited for in between."""
    c = C.xent_case(130, 256, 5000, "bf16", seed=12)
    b = C.balance_case(3000, 64, 4, [0, 700, 3000], "softmax", 0.1, seed=13)
    grads = [torch.randn(70001, device="cuda") for _ in range(3)]
    t = _lib.make_grad_tensors(grads)
    runs = []
    for _ in range(2):
        d, ws = C.xent_setup(c)
        bd = C.balance_dims(b)
        runs.append(dict(stream=torch.cuda.Stream(), d=d, ws=ws, bd=bd, bws=_lib.alloc_balance_workspace(bd),
                         nws=_lib.alloc_grad_norm_workspace(t), x=[C.nan(130), C.nan(130), C.nan(2)],
                         g=[torch.empty_like(c["x"]), torch.empty_like(c["w"])], norm=C.nan(1),
                         b=[C.nan(2), torch.zeros(2, 64, dtype=torch.int32, device="cuda"), C.nan(2, 64)]))
    torch.cuda.synchronize()
    for _ in range(5):
        for r in runs:
            st = r["stream"]
            _lib.moe_balance_fwd(r["bd"], r["bws"], b["logits"], b["idx"], b["start"], *r["b"], stream=st)
            _lib.moe_xent_fwd(r["d"], r["ws"], c["x"], c["w"], c["target"], *r["x"], stream=st)
            _lib.moe_xent_bwd(r["d"], r["ws"], c["x"], c["w"], c["target"], r["x"][1], None, r["x"][2], *r["g"], stream=st)
            _lib.moe_grad_norm(t, r["nws"], r["norm"], stream=st)
    torch.cuda.synchronize()
    for x, y in zip(*([*r["x"], *r["g"], *r["b"], r["norm"]] for r in runs)):
        assert torch.equal(x, y)
    C.check_xent_fwd(c, runs[0]["x"])
    C.check_balance_fwd(b, runs[1]["b"])


# ---------------------------------------------------------------- gradient norm
@pytest.mark.parametrize("sizes", [[1], [0, 3], [255, 256, 257], [8192, 1, 40000], [7] * 30, list(range(1, 401)), [300000] * 3,
                                   [5] * 1250 + [0] * 3, [0] * 2 + [9000] * 1300 + [0]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_norm(sizes, dtype):
    g = torch.Generator().manual_seed(len(sizes))
    grads = [torch.randn(n, generator=g).to(DT[dtype]).cuda() for n in sizes]
    t = _lib.make_grad_tensors(grads)
    ws = _lib.alloc_grad_norm_workspace(t)
    ws[256:].fill_(0xFF)
    norm = C.nan(1)
    want = np.sqrt(sum((f64(x) ** 2).sum() for x in grads))
    for scale in (1.0, -0.25):
        _lib.moe_grad_norm(t, ws, norm, scale)
        # a thread adds some 32 squares for each of its steps, then trees
        assert abs(float(norm) - abs(scale) * want) <= 256 * E32 * want * abs(scale)
        assert int(ws[:256].sum()) == 0


def test_grad_norm_of_nothing_and_of_nan():
    norm = C.nan(1)
    for grads in ([], [torch.zeros(0, device="cuda")], [torch.zeros(500, device="cuda")]):
        t = _lib.make_grad_tensors(grads)
        _lib.moe_grad_norm(t, _lib.alloc_grad_norm_workspace(t), norm)
        assert float(norm) == 0.0
    for bad in (NAN, INF):
        x = torch.zeros(3000, device="cuda")
        x[2999] = bad
        t = _lib.make_grad_tensors([torch.zeros(10, device="cuda"), x])
        _lib.moe_grad_norm(t, _lib.alloc_grad_norm_workspace(t), norm)
        assert not np.isfinite(float(norm))


# ---------------------------------------------------------------- AdamW
TENSORS = [[1], [3, 0, 5], [255, 256, 257, 4095, 4096, 4097], [1000] * 30, [100003], list(range(1, 420)),
           [5000] * 400 + [0]]


@pytest.mark.parametrize("sizes", TENSORS)
@pytest.mark.parametrize("param,grad,master,bits", [("f32", "f32", False, 32), ("bf16", "bf16", True, 32),
                                                    ("bf16", "f32", False, 32), ("f32", "bf16", False, 8),
                                                    ("bf16", "bf16", True, 8), ("bf16", "f32", False, 8)])
def test_adamw(sizes, param, grad, master, bits):
    c = C.adamw_case(sizes, param, grad, master, bits, seed=len(sizes))
    before = C.adamw_before(c)
    C.run_adamw(c)
    C.check_adamw(c, before)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [dict(step=1), dict(step=100000), dict(beta1=0.0, beta2=0.0), dict(beta2=0.9999), dict(eps=1.0),
                                dict(wd=0.0), dict(gscale=1e-6), dict(gscale=1e6), dict(lr=0.0)])
def test_adamw_settings(bits, kw):
    c = C.adamw_case([3000, 77], bits=bits, seed=2, **kw)
    before = C.adamw_before(c)
    C.run_adamw(c)
    C.check_adamw(c, before)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_clips_scales_and_skips(bits):
    norm = torch.tensor([8.0], device="cuda")
    c = C.adamw_case([5000, 3], "bf16", "bf16", True, bits, seed=3)
    before = C.adamw_before(c)
    C.run_adamw(c, max_norm=2.0, norm=norm, grad_scale=0.5)
    C.check_adamw(c, before, factor=0.125)
    before = C.adamw_before(c)
    C.run_adamw(c, max_norm=20.0, norm=norm)  # below the limit
    C.check_adamw(c, before)
    before = C.adamw_before(c)
    C.run_adamw(c, norm=norm)  # no limit
    C.check_adamw(c, before)
    kept = [t.clone() for k in ("p", "master", "m", "v") for t in c[k]]
    for bad in (NAN, INF):
        norm.fill_(bad)
        C.run_adamw(c, max_norm=2.0, norm=norm)
        C.run_adamw(c, norm=norm)
    raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    for a, b in zip(kept, [t for k in ("p", "master", "m", "v") for t in c[k]]):
        assert torch.equal(raw(a), raw(b))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_limit_of_infinity_clips_nothing(bits):
    """A limit that is there for the norm, and for steps that it leaves out."""
    c = C.adamw_case([700], bits=bits, seed=12)
    before = C.adamw_before(c)
    norm = torch.tensor([8.0], device="cuda")
    C.run_adamw(c, max_norm=INF, norm=norm)
    C.check_adamw(c, before)
    kept = c["p"][0].clone()
    norm.fill_(INF)
    C.run_adamw(c, max_norm=INF, norm=norm)
    assert torch.equal(kept, c["p"][0])


def test_adamw_factors_of_each_tensor():
    c = C.adamw_case([600, 600, 1], seed=4, wd=[0.0, 0.5, 0.25])
    before = C.adamw_before(c)
    C.run_adamw(c, lr_scale=[1.0, 0.0, 1.0])
    assert np.array_equal(f64(c["p"][1]), before[1][0])  # lr of zero
    c["p"][1].copy_(torch.tensor(before[1][0] * (1 - 0.01 * 0.5), device="cuda"))
    P, M, V = C.O.adamw(*before[1], 0.01, 0.9, 0.99, 1e-8, 7, 0.5, 1.0)
    C.close(c["m"][1], M, 8 * E32 * (np.abs(M) + np.abs(before[1][1]) + np.abs(before[1][2])), "m")
    for i in (0, 2):
        one = dict(c, sizes=[c["sizes"][i]], wd=[c["wd"][i]], **{k: [c[k][i]] for k in ("p", "g", "m", "v", "master")})
        C.check_adamw(one, [before[i]])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_values_that_are_not_finite_stay_alone(bits):
    c = C.adamw_case([1024], bits=bits, seed=5)
    ref = C.adamw_case([1024], bits=bits, seed=5)
    before = C.adamw_before(ref)
    C.run_adamw(ref)
    C.check_adamw(ref, before)
    c["g"][0][300] = NAN
    c["g"][0][301] = INF
    C.run_adamw(c)
    ok = torch.ones(1024, dtype=torch.bool, device="cuda")
    ok[300:302] = False
    for k in ("p", "m", "v"):
        a, b = c[k][0].float(), ref[k][0].float()
        if k == "p" or bits == 32:
            assert torch.equal(a[ok], b[ok])
        else:  # the block's largest may have been one of the two
            other = torch.ones(1024, dtype=torch.bool, device="cuda")
            other[256:512] = False
            assert torch.equal(a[other], b[other]) and torch.isfinite(a[ok]).all() and torch.isnan(a[300:302]).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [1e-21, 3e-20, 2e-19, 1e20])
def test_adamw_squares_that_leave_fp32(bits, size):
    """Gradients whose squares are denormal, zero or infinite in fp32 (all of a tensor, so that 8-bit scales are as
    small): roots and weights are what that arithmetic gives, and nothing is NaN."""
    c = C.adamw_case([600], bits=bits, seed=9, step=3, eps=1e-30 if size < 1 else 1e-8, wd=0.0)
    for k in ("m", "v"):
        (c[k][0].view(torch.uint8) if bits == 8 else c[k][0]).zero_()
    c["g"][0].copy_(torch.sign(c["g"][0]) * size * (0.5 + torch.rand(600, device="cuda")))
    p0 = f64(c["p"][0])
    g = f64(c["g"][0]).astype(np.float32)
    C.run_adamw(c)
    with np.errstate(over="ignore", under="ignore"):
        v = np.float32(1 - 0.99) * (g * g)
    m = np.float32(1 - 0.9) * g
    r = np.sqrt(v.astype(np.float64))
    want = p0 - np.float32(0.01) * (m / (1 - 0.9 ** 3)) / (r / np.sqrt(1 - 0.99 ** 3) + np.float32(c["eps"]))
    got = f64(c["p"][0])
    assert np.isfinite(got).all()
    # v is off by a denormal's last place and half, r by half of that of itself
    slack = 1e-5 + 2.0 ** -149 / np.maximum(v.astype(np.float64), 2.0 ** -149)
    assert (np.abs(got - want) <= 2 * E32 * np.abs(p0) + slack * np.abs(want - p0)).all()


def test_adamw8_small_roots_stay_above_zero():
    """In a block with one large gradient, states far below it: a root becomes at least the smallest code, so later
    steps do not divide by eps alone."""
    n = 256
    c = C.adamw_case([n], bits=8, seed=6, step=1)
    for k in ("m", "v"):
        c[k][0].view(torch.uint8).zero_()
    c["g"][0].fill_(1e-6)
    c["g"][0][0] = 1e3
    before = C.adamw_before(c)
    C.run_adamw(c)
    C.check_adamw(c, before)
    assert float(c["v"][0].float()[1:].min()) == 2.0 ** -9
    c["g"][0].zero_()
    p = c["p"][0].clone()
    c["step"] = 2
    C.run_adamw(c)
    assert float((c["p"][0] - p).abs().max()) < 0.1


def test_adamw_device_lr_and_step_in_a_graph():
    lr, step = torch.tensor([0.02], device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda")
    c = C.adamw_case([3000, 5], "bf16", "f32", True, 32, seed=7)
    for k in ("m", "v"):
        for t in c[k]:
            t.zero_()
    t = _lib.make_adamw_tensors(c["p"], c["g"], c["m"], c["v"], c["master"], weight_decay=0.1)
    d = _lib.make_adamw_dims(9.0, 0.9, 0.99, 1e-8, 999)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.add_(1)
        _lib.moe_adamw_step(d, t, None, lr, step)
    for i in range(1, 5):
        before = C.adamw_before(c)
        lr.fill_(0.01 * i)
        g.replay()
        torch.cuda.synchronize()
        C.check_adamw(c, before, lr=float(np.float32(0.01 * i)), step=i)


def test_adamw_refusals():
    f = lambda n=8: torch.zeros(n, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        p = f()
        _lib.make_adamw_tensors([p, p], [f(), f()], [f(), f()], [f(), f()])
    with pytest.raises(ValueError, match="overlap"):  # a state in the gradient's buffer
        g = f()
        _lib.make_adamw_tensors([f()], [g], [g], [f()])
    with pytest.raises(ValueError, match="overlap"):  # part of a buffer
        b = f(16)
        _lib.make_adamw_tensors([b[:8], b[4:12]], [f(), f()], [f(), f()], [f(), f()])
    shared = f()  # two weights with one gradient
    _lib.make_adamw_tensors([f(), f()], [shared, shared], [f(), f()], [f(), f()])
    with pytest.raises(ValueError, match="m.0. must have 8 values"):
        _lib.make_adamw_tensors([f()], [f()], [f(9)], [f()])
    with pytest.raises(TypeError, match="v.0. must be"):
        _lib.make_adamw_tensors([f()], [f()], [f()], [f().bfloat16()])
    with pytest.raises(ValueError, match="contiguous"):
        _lib.make_adamw_tensors([f()], [f(16)[::2]], [f()], [f()])
    with pytest.raises(ValueError, match="scale"):
        _lib.make_adamw_tensors([f()], [f()], [f()], [f()], m_scale=[f(1)], v_scale=[f(1)])
    t = _lib.make_adamw_tensors([f()], [f()], [f()], [f()])
    with pytest.raises(ValueError, match="bits"):
        _lib.moe_adamw_step(_lib.make_adamw_dims(0.1, state_bits=8), t)
    with pytest.raises(_lib.MoeError, match="misaligned"):
        _lib.moe_adamw_step(_lib.make_adamw_dims(0.1), _lib.make_adamw_tensors([f(9)[1:]], [f()], [f()], [f()]))
    with pytest.raises(ValueError, match="shape"):
        _lib.moe_adamw_step(_lib.make_adamw_dims(0.1), t, norm=f(2))


@pytest.mark.parametrize("bits", [32, 8])
def test_optimiser_over_several_steps(bits):
    """The class against the definition, step after step from zero states, with clipping."""
    g = torch.Generator().manual_seed(8)
    sizes = [1000, 17, 513]
    params = [(torch.randn(n, generator=g) * 0.1).bfloat16().cuda() for n in sizes]
    grads = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
    opt = AdamW(params, grads, 0.01, 0.9, 0.95, weight_decay=[0.1, 0.0, 0.1], state_bits=bits, max_norm=1.0)
    for step in range(1, 5):
        for t in grads:
            t.copy_(torch.randn(t.numel(), generator=g) * 0.2)
        want = np.sqrt(sum((f64(t) ** 2).sum() for t in grads))
        c = dict(sizes=sizes, bits=bits, p=params, g=grads, m=opt.m, v=opt.v, ms=opt.m_scale, vs=opt.v_scale,
                 master=opt.master, lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, step=step, wd=[0.1, 0.0, 0.1])
        before = C.adamw_before(c)
        opt.step()
        assert abs(float(opt.norm) - want) < 256 * E32 * want
        C.check_adamw(c, before, factor=1.0 / max(1.0, float(opt.norm)))
