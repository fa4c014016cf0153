"""The experts on a caller's routing (moe_fwd_routed, moe_bwd_routed) and MoEBlock, which runs the norm, linear
and gate operators with them, against fp64 autograd."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from expert_grouped_gemm_gb300.block import MoEBlock
from expert_grouped_gemm_gb300.inputs import custom, make_inputs
from expert_grouped_gemm_gb300.layer import MoELayer
from tests.parity import TOL, rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- fp64 reference
def experts64(n, idx, w, p):
    """sum_j w_j swiglu_{e_j}(n) + shared(n), in whatever precision the tensors have."""
    sw = lambda v, g, u, d: (torch.nn.functional.silu(v @ g) * (v @ u)) @ d
    y = torch.zeros_like(n)
    for e in range(p["w_gate"].shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            y = y.index_add(0, t, w[t, j, None] * sw(n[t], p["w_gate"][e], p["w_up"][e], p["w_down"][e]))
    if p.get("ws_gate") is not None:
        y = y + sw(n, p["ws_gate"], p["ws_up"], p["ws_down"])
    return y


def leaf(t):
    return None if t is None else t.detach().double().cpu().requires_grad_(True)


def routing(w, seed):
    """Different experts per token, weights of either sign."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(w.E, generator=g)[:w.k] for _ in range(w.T)]).int()
    return idx, torch.randn(w.T, w.k, generator=g)


def run_routed(w, inp, idx, tw, use_retained=False, quota=None, recompute=False):
    layer = MoELayer(w, inp, recompute=recompute)
    d, ws, p = layer.dims, layer.ws, layer.p
    x, dy = inp["x"].cuda(), inp["dy"].cuda()
    idx, tw = idx.cuda(), tw.cuda()
    dtw = torch.full((w.T, w.k), float("nan"), device="cuda")
    off = torch.empty(w.E + 1, dtype=torch.int32, device="cuda")
    _lib.moe_fwd_routed(d, ws, x, idx, tw, p["w_gate"], p["w_up"], p["w_down"], p["ws_gate"], p["ws_up"], p["ws_down"],
                        layer.y, off)
    if quota is not None:
        _lib.moe_select_retained(d, ws, dy, quota.cuda())
    g = {n: t for n, t in layer.grads.items() if n != "dw_router"}
    _lib.moe_bwd_routed(d, ws, dy, x, use_retained, layer.dx, dtw, *(g.get(n) for n in (
        "dw_gate", "dw_up", "dw_down", "dws_gate", "dws_up", "dws_down")))
    return layer, off, dtw, g, _lib.moe_read_status(ws)


@pytest.mark.parametrize("kw", [
    dict(T=200, H=128, F=192, E=16, k=4, F_shared=64), dict(T=1, H=128, F=128, E=16, k=2),
    dict(T=77, H=192, F=128, E=32, k=12), dict(T=45, H=40, F=24, E=5, k=3, dtype="f32", F_shared=8),
    dict(T=60, H=128, F=64, E=16, k=16), dict(T=64, H=128, F=128, E=16, k=2, frozen=True)])
@pytest.mark.parametrize("recompute", [False, True])
def test_routed_against_autograd(kw, recompute):
    w = custom("routed", **kw)
    inp = make_inputs(w, seed=1)
    idx, tw = routing(w, 2)
    layer, off, dtw, g, status = run_routed(w, inp, idx, tw, recompute=recompute)
    assert status == _lib.MOE_OK
    assert np.array_equal(np.diff(off.cpu().numpy()), np.bincount(idx.numpy().ravel(), minlength=w.E))
    x, tw64 = leaf(inp["x"]), leaf(tw)
    p = {n: leaf(inp[n]) for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")}
    y = experts64(x, idx.long(), tw64, p)
    (y * inp["dy"].double()).sum().backward()
    tol = TOL[w.dtype]
    f = lambda t: t.detach().double().cpu().numpy()
    assert rel_fro(f(layer.y), f(y)) < tol
    assert rel_fro(f(layer.dx), x.grad.numpy()) < tol
    assert rel_fro(f(dtw), tw64.grad.numpy()) < tol
    for n, t in g.items():
        assert rel_fro(f(t), p[n[1:]].grad.numpy()) < tol, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_routed_with_the_routers_choice_is_moe_fwd(dtype):
    """Given the experts and weights moe_fwd chose, the same bits come out; dtopk_w is what its router gradient is
    made of."""
    w = custom("same", T=300, H=128, F=128, E=16, k=4, zipf_s=1.0, F_shared=64, dtype=dtype, quota_factor=0.5)
    inp = make_inputs(w, seed=3)
    for quota in (None, inp["quota"]):
        ref = MoELayer(w, inp, record_routing=True)
        x, dy = inp["x"].cuda(), inp["dy"].cuda()
        ref.forward(x)
        if quota is not None:
            ref.select(dy, quota.cuda())
        ref.backward(dy, x, quota is not None)
        got, off, dtw, g, status = run_routed(w, inp, ref.topk_idx.cpu(), ref.topk_w.cpu(), quota is not None, quota)
        assert status == _lib.MOE_OK
        assert torch.equal(got.y, ref.y) and torch.equal(off, ref.offsets)
        for n, t in g.items():
            assert torch.equal(t, ref.grads[n]), n
        tw = ref.topk_w
        dl = tw * (dtw - (tw * dtw).sum(1, keepdim=True))
        dense = torch.zeros(w.T, w.E, device="cuda").scatter_(1, ref.topk_idx.long(), dl)
        dwr = inp["x"].double().T @ dense.double().cpu()
        assert rel_fro(ref.grads["dw_router"].double().cpu().numpy(), dwr.numpy()) < TOL[dtype]


@pytest.mark.parametrize("T", [40, 100])
def test_routed_call_order_and_bad_indices(T):
    w = custom("order", T=T, H=128, F=128, E=16, k=3)
    inp = make_inputs(w, seed=4)
    idx, tw = routing(w, 5)
    layer, _, _, g, _ = run_routed(w, inp, idx, tw)
    x, dy = inp["x"].cuda(), inp["dy"].cuda()
    with pytest.raises(_lib.MoeError) as e:
        layer.backward(dy, x, False)          # moe_bwd after moe_fwd_routed
    assert e.value.code == _lib.MOE_ERR_STATE
    layer.forward(x)
    with pytest.raises(_lib.MoeError) as e:   # moe_bwd_routed after moe_fwd
        _lib.moe_bwd_routed(layer.dims, layer.ws, dy, x, False, layer.dx, torch.empty(w.T, w.k, device="cuda"),
                            g["dw_gate"], g["dw_up"], g["dw_down"])
    assert e.value.code == _lib.MOE_ERR_STATE
    with pytest.raises(ValueError, match="topk_w"):
        _lib.moe_fwd_routed(layer.dims, layer.ws, x, idx.cuda(), None, *([layer.p["w_gate"]] * 3), None, None, None, layer.y)
    # an index out of range and a repeated one: reported, weight 0, everything else as without them
    bad, zeroed = idx.clone(), tw.clone()
    bad[3, 1], bad[7, 0], bad[9, 2], bad[11, 2] = 16, -1, bad[9, 0], 2 ** 31 - 1
    for t, j in ((3, 1), (7, 0), (9, 2), (11, 2)):
        zeroed[t, j] = 0.0
    want, _, _, _, status = run_routed(w, inp, idx, zeroed)
    assert status == _lib.MOE_OK
    got, off, dtw, _, status = run_routed(w, inp, bad, tw)
    assert status == _lib.MOE_ERR_DEVICE_ARG
    assert int(off[-1]) == w.T * w.k and torch.isfinite(dtw).all()
    f = lambda t: t.double().cpu().numpy()
    assert rel_fro(f(got.y), f(want.y)) < 1e-2


# ---------------------------------------------------------------- the block
def block_params(w, A, seed, norm_b):
    inp = make_inputs(w, seed)
    g = torch.Generator().manual_seed(seed + 100)
    r = lambda *s, scale: (torch.randn(*s, generator=g) * scale).to(inp["x"].dtype)
    p = {n: inp[n] for n in ("w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")}
    p["w_router"] = r(w.H, w.E, scale=0.1)
    p.update(w_o=r(A, w.H, scale=A ** -0.5), b_o=r(w.H, scale=0.1), norm_w=1 + r(w.H, scale=0.2),
             norm_b=r(w.H, scale=0.1) if norm_b else None,
             balance_bias=torch.round(100 * torch.randn(w.E, generator=g) * 0.05) * 1e-2)
    return p, r(w.T, A, scale=1.0), r(w.T, w.H, scale=1.0), r(w.T, w.H, scale=1.0), r(w.T, w.H, scale=1.0)


BLOCKS = [
    (dict(T=300, H=256, F=192, E=32, k=4, F_shared=64), 320, dict(norm="layer", score="sigmoid", renorm=True, scale=2.5,
                                                                  n_group=8, topk_group=4, group_take=2)),
    (dict(T=1, H=256, F=128, E=16, k=2), 256, dict(norm="rms", score="softmax", renorm=True)),
    (dict(T=5, H=128, F=128, E=16, k=3, F_shared=64), 100, dict(norm="rms", score="softmax", renorm=False, scale=4.0)),
    (dict(T=50, H=48, F=24, E=10, k=3, F_shared=8, dtype="f32"), 33, dict(norm="layer", score="sigmoid", renorm=False)),
    (dict(T=512, H=2048, F=768, E=128, k=8), 4096, dict(norm="rms", score="softmax", renorm=True)),
]


@pytest.mark.parametrize("kw,A,opt", BLOCKS)
def test_block_against_autograd(kw, A, opt):
    w = custom("block", **kw)
    params, attn, res, dy, dh = block_params(w, A, 7, opt["norm"] == "layer")
    blk = MoEBlock(w, params, **opt)
    c = lambda t: t.cuda()
    y, h = blk.forward(c(attn), c(res))
    dattn, dres, g = blk.backward(c(attn), c(dy), c(dh))
    assert blk.status() == _lib.MOE_OK
    idx = blk.topk_idx.cpu().long()
    assert torch.equal(blk.expert_count.cpu(), torch.bincount(idx.flatten(), minlength=w.E).int())
    # fp64, the choice of experts taken from the GPU
    P = {n: leaf(t) for n, t in params.items() if n != "balance_bias"}
    a64, r64 = leaf(attn), leaf(res)
    h64 = r64 + a64 @ P["w_o"] + P["b_o"]
    m = h64.mean(1, keepdim=True) if opt["norm"] == "layer" else 0.0
    n64 = (h64 - m) * torch.rsqrt(((h64 - m) ** 2).mean(1, keepdim=True) + 1e-5) * P["norm_w"]
    if P["norm_b"] is not None:
        n64 = n64 + P["norm_b"]
    l64 = n64 @ P["w_router"]
    s = torch.softmax(l64, 1) if opt["score"] == "softmax" else torch.sigmoid(l64)
    tw = s.gather(1, idx)
    if opt["renorm"]:
        tw = tw / tw.sum(1, keepdim=True)
    tw = tw * opt.get("scale", 1.0)
    y64 = experts64(n64, idx, tw, P)
    ((y64 * dy.double()).sum() + (h64 * dh.double()).sum()).backward()
    tol = TOL[w.dtype]
    f = lambda t: t.detach().double().cpu().numpy()
    errs = dict(y=rel_fro(f(y), f(y64)), h=rel_fro(f(h), f(h64)), w=rel_fro(f(blk.topk_w), f(tw)),
                dattn=rel_fro(f(dattn), a64.grad.numpy()), dres=rel_fro(f(dres), r64.grad.numpy()))
    for n, t in g.items():
        errs[n] = rel_fro(f(t), P[n].grad.numpy())
    print(errs)
    assert all(v < tol for v in errs.values()), errs


def test_block_in_a_graph_and_on_a_stream():
    w = custom("block", T=64, H=256, F=128, E=16, k=2)
    params, attn, res, dy, dh = block_params(w, 256, 9, False)
    blk = MoEBlock(w, params)
    attn, res, dy, dh = attn.cuda(), res.cuda(), dy.cuda(), dh.cuda()

    def step():
        blk.forward(attn, res)
        blk.backward(attn, dy, dh)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (blk.y, blk.h, blk.dattn, blk.dh, *blk.grads.values())]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (blk.y, blk.h, blk.dattn, blk.dh, *blk.grads.values()):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (blk.y, blk.h, blk.dattn, blk.dh, *blk.grads.values())):
        assert torch.equal(a, b)
    assert blk.status() == _lib.MOE_OK
