"""MoEBlock with retention quotas and with recomputed activations."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from expert_grouped_gemm_gb300.block import MoEBlock
from expert_grouped_gemm_gb300.inputs import custom, make_inputs
from tests.parity import TOL, rel_fro
from tests.test_gpu_moe_block import block_params, leaf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


BLOCKS = [
    (dict(T=300, H=256, F=192, E=32, k=4, F_shared=64, quota_factor=0.5), 320,
     dict(norm="layer", score="sigmoid", renorm=True, scale=2.5, n_group=8, topk_group=4, group_take=2)),
    (dict(T=50, H=48, F=24, E=10, k=3, F_shared=8, dtype="f32", quota_factor=0.4), 33, dict(norm="rms", score="softmax",
                                                                                          renorm=False)),
]


def run(kw, A, opt, recompute, quota):
    """A forward and backward; quota None: every pair, else the experts' part over the pairs within it."""
    w = custom("block", **kw)
    params, attn, res, dy, dh = block_params(w, A, 7, opt["norm"] == "layer")
    blk = MoEBlock(w, params, recompute=recompute, **opt)
    attn, res, dy, dh = (t.cuda() for t in (attn, res, dy, dh))
    blk.forward(attn, res)
    if quota is not None:
        blk.select(dy, quota.cuda())
    blk.backward(attn, dy, dh, use_retained=quota is not None)
    assert blk.status() == _lib.MOE_OK
    return w, params, blk, attn, dy


def outputs(blk):
    return dict(y=blk.y, h=blk.h, dattn=blk.dattn, dh=blk.dh, dtopk_w=blk.dtopk_w, **blk.grads)


@pytest.mark.parametrize("kw,A,opt", BLOCKS)
def test_recomputed_activations_give_the_same_bits(kw, A, opt):
    want, got = (outputs(run(kw, A, opt, r, None)[2]) for r in (False, True))
    for n, t in want.items():
        assert torch.equal(got[n], t), n


@pytest.mark.parametrize("kw,A,opt", BLOCKS)
@pytest.mark.parametrize("recompute", [False, True])
def test_retention_in_the_block(kw, A, opt, recompute):
    """Under quotas the experts' gradients, dn's expert part among them, are those of the kept pairs; quotas that keep
    every pair give the bits of the full backward."""
    w = custom("block", **kw)
    full = outputs(run(kw, A, opt, recompute, None)[2])
    every = torch.full((w.E,), w.T, dtype=torch.int32)
    for n, t in outputs(run(kw, A, opt, recompute, every)[2]).items():
        assert torch.equal(t, full[n]), n
    quota = make_inputs(w, 7)["quota"]
    _, params, blk, attn, dy = run(kw, A, opt, recompute, quota)
    assert torch.equal(blk.dtopk_w, full["dtopk_w"]) and torch.equal(blk.y, full["y"])
    # the kept pairs, from the selection's own list
    off = torch.empty(w.E + 1, dtype=torch.int32, device="cuda")
    rows = torch.full((w.T * w.k,), -1, dtype=torch.int32, device="cuda")
    _lib.moe_select_retained(blk.moe, blk.ws_moe, dy, quota.cuda(), off, rows)
    counts = np.bincount(blk.topk_idx.cpu().numpy().ravel(), minlength=w.E)
    assert np.array_equal(np.diff(off.cpu().numpy()), np.minimum(quota.numpy(), counts))
    row_of_pair = _lib.ws_view(blk.ws_moe, blk.moe, "row_of_pair", torch.int32, (w.T, w.k))
    kept = torch.isin(row_of_pair, rows[:int(off[-1])]).cpu()
    assert 0 < int(kept.sum()) < w.T * w.k
    # the experts alone in 64 bits, on the block's own n and routing: gradients through the kept pairs and the shared expert
    P = {n: leaf(params[n]) for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")}
    n64, idx, tw = leaf(blk.n), blk.topk_idx.cpu().long(), blk.topk_w.double().cpu()
    sw = lambda v, a, b, c: (torch.nn.functional.silu(v @ a) * (v @ b)) @ c
    y = sw(n64, P["ws_gate"], P["ws_up"], P["ws_down"])
    for e in range(w.E):
        t, j = torch.nonzero((idx == e) & kept, as_tuple=True)
        if len(t):
            y = y.index_add(0, t, tw[t, j, None] * sw(n64[t], P["w_gate"][e], P["w_up"][e], P["w_down"][e]))
    (y * dy.double().cpu()).sum().backward()
    f = lambda t: t.detach().double().cpu().numpy()
    for n in P:
        assert rel_fro(f(blk.grads[n]), P[n].grad.numpy()) < TOL[w.dtype], n
    # dn = that part and the router's, which reads every pair's dtopk_w
    dn = n64.grad + blk.dlogits.double().cpu() @ params["w_router"].double().T
    assert rel_fro(f(blk.dn), dn.numpy()) < TOL[w.dtype]
