"""A training step of the MoE block as it is used: experts with their balance loss, a vocabulary loss on the output,
gradients back through both, clipping and AdamW; against fp64 autograd."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from expert_grouped_gemm_gb300.block import MoEBlock
from expert_grouped_gemm_gb300.inputs import custom
from expert_grouped_gemm_gb300.optim import AdamW
from oracle import train_oracle as O
from tests.parity import TOL, rel_fro
from tests.test_gpu_moe_block import block_params, experts64, leaf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def reference(w, P, attn, res, idx, opt, start):
    """(y, h, losses) of the block in fp64, the choice of experts given."""
    h = res + attn @ P["w_o"] + P["b_o"]
    n = h * torch.rsqrt((h ** 2).mean(1, keepdim=True) + 1e-5) * P["norm_w"]
    l = n @ P["w_router"]
    s = torch.softmax(l, 1) if opt["score"] == "softmax" else torch.sigmoid(l)
    tw = s.gather(1, idx)
    tw = tw / tw.sum(1, keepdim=True)
    y = experts64(n, idx, tw, P)
    p = s / s.sum(1, keepdim=True)
    N = start[-1] - start[0]
    bal = 0.0
    for a, b in zip(start[:-1], start[1:]):
        if b > a:
            count = torch.bincount(idx[a:b].flatten(), minlength=w.E).double()
            bal = bal + opt["balance"] * w.E / (w.k * N) * (count * p[a:b].mean(0)).sum()
    z = opt.get("z_coef", 0.0) * (torch.logsumexp(l[start[0]:start[-1]], 1) ** 2).sum() / N
    return y, h, bal, z


CASES = [
    (dict(T=200, H=128, F=64, E=16, k=3, F_shared=64), 96, dict(score="softmax", balance=0.5, z_coef=0.02), [0, 60, 60, 190], 1.5),
    (dict(T=70, H=48, F=24, E=10, k=2, dtype="f32"), 33, dict(score="sigmoid", balance=0.3), [0, 70], None),
    (dict(T=300, H=256, F=128, E=32, k=4), 128, dict(score="sigmoid", balance=2.0), [5, 100, 300], -0.5),
]


@pytest.mark.parametrize("kw,A,opt,start,up", CASES)
def test_block_with_balance_loss_against_autograd(kw, A, opt, start, up):
    w = custom("block", **kw)
    params, attn, res, dy, dh = block_params(w, A, 11, False)
    blk = MoEBlock(w, params, sequences=len(start) - 1, **opt)
    c = lambda t: t.cuda()
    dev = torch.tensor(start, dtype=torch.int32, device="cuda")
    blk.forward(c(attn), c(res), seq_start=dev)
    dloss = None if up is None else torch.tensor([up], device="cuda")
    dattn, dres, g = blk.backward(c(attn), c(dy), c(dh), dloss=dloss)
    assert blk.status() == _lib.MOE_OK
    P = {n: leaf(t) for n, t in params.items() if n != "balance_bias"}
    a64, r64 = leaf(attn), leaf(res)
    idx = blk.topk_idx.cpu().long()
    y, h, bal, z = reference(w, P, a64, r64, idx, opt, start)
    ((y * dy.double()).sum() + (h * dh.double()).sum() + (bal + z) * (1.0 if up is None else up)).backward()
    tol = TOL[w.dtype]
    errs = dict(loss=rel_fro(f64(blk.loss), np.array([float(bal), float(z)])),
                dattn=rel_fro(f64(dattn), a64.grad.numpy()), dres=rel_fro(f64(dres), r64.grad.numpy()))
    errs.update({n: rel_fro(f64(t), P[n].grad.numpy()) for n, t in g.items()})
    assert all(v < tol for v in errs.values()), errs
    for s, (a, b) in enumerate(zip(start[:-1], start[1:])):
        assert torch.equal(blk.seq_count[s].cpu(), torch.bincount(idx[a:b].flatten(), minlength=w.E).int())


def test_block_without_balance_is_unchanged():
    """The balance loss reads the routing; without a factor nothing of it runs, with a factor of zero nothing changes."""
    w = custom("block", T=64, H=128, F=64, E=16, k=2)
    params, attn, res, dy, dh = (t.cuda() if isinstance(t, torch.Tensor) else t for t in block_params(w, 64, 3, False))
    outs = []
    for kw in ({}, dict(balance=0.0)):
        blk = MoEBlock(w, params, **kw)
        y, h = blk.forward(attn, res)
        a, r, g = blk.backward(attn, dy, dh)
        outs.append([t.clone() for t in (y, h, a, r, *g.values())])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="seq_start"):
        MoEBlock(w, params).forward(attn, res, seq_start=torch.zeros(2, dtype=torch.int32, device="cuda"))


class Trainer:
    """A block with a vocabulary head on y + h, and an optimiser over both; every step in the library's kernels but
    the sum of y and h."""

    def __init__(self, w, A, V, bits, seed=5, tied=True, capturable=False):
        params, self.attn, self.res, _, _ = block_params(w, A, seed, False)
        g = torch.Generator().manual_seed(seed)
        dt = params["w_o"].dtype
        self.w, self.V = w, V
        self.blk = MoEBlock(w, params, balance=0.1, z_coef=0.001)
        self.head = (torch.randn(V, w.H, generator=g) * w.H ** -0.5).to(dt).cuda()
        self.target = torch.randint(-1, V, (w.T,), generator=g).int().cuda()
        self.dims = _lib.make_xent_dims(w.T, w.H, V, w.dtype, tied)
        self.ws = _lib.alloc_xent_workspace(self.dims)
        f = lambda *s: torch.empty(*s, device="cuda")
        self.loss, self.lse, self.total = f(w.T), f(w.T), f(2)
        self.dout, self.dhead = torch.empty(w.T, w.H, dtype=dt, device="cuda"), torch.empty_like(self.head)
        self.attn, self.res = self.attn.cuda(), self.res.cuda()
        names = list(self.blk.grads)
        self.names = names + ["head"]
        self.params = [self.blk.p[n] for n in names] + [self.head]
        self.grads = [self.blk.grads[n] for n in names] + [self.dhead]
        self.opt = AdamW(self.params, self.grads, 1e-3, weight_decay=[0.0 if p.dim() == 1 else 0.1 for p in self.params],
                         state_bits=bits, max_norm=0.5, capturable=capturable)

    def step(self):
        y, h = self.blk.forward(self.attn, self.res)
        self.out = y + h
        _lib.moe_xent_fwd(self.dims, self.ws, self.out, self.head, self.target, self.loss, self.lse, self.total)
        _lib.moe_xent_bwd(self.dims, self.ws, self.out, self.head, self.target, self.lse, None, self.total, self.dout, self.dhead)
        self.blk.backward(self.attn, self.dout, self.dout)
        self.opt.step()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_against_autograd(dtype, bits):
    kw = dict(T=96, H=64, F=64, E=16, k=2) if dtype == "bf16" else dict(T=50, H=40, F=24, E=10, k=3, dtype="f32")
    w = custom("train", **kw)
    t = Trainer(w, 48, 501, bits)
    for step in (1, 2):
        before = {n: (p.clone() if m is None else m.clone()) for n, p, m in zip(t.names, t.params, t.opt.master)}
        rounded = {n: p.clone() for n, p in zip(t.names, t.params)}
        states = []
        for i, p in enumerate(t.params):
            m, v = f64(t.opt.m[i].float()), f64(t.opt.v[i].float())
            if bits == 8:
                rep = lambda s: np.repeat(f64(s), 256)[:p.numel()]
                m, v = m * rep(t.opt.m_scale[i]), (v * rep(t.opt.v_scale[i])) ** 2
            states.append((m, v))
        t.step()
        assert t.blk.status() == _lib.MOE_OK and _lib.moe_read_status(t.ws) == _lib.MOE_OK
        # the forward and backward of the weights as they were
        P = {n: leaf(rounded[n].cpu()) for n in t.names}
        P["b_o"] = P.get("b_o", leaf(t.blk.p["b_o"].cpu()))
        opt = dict(score="softmax", balance=0.1, z_coef=0.001)
        y, h, bal, z = reference(w, P, t.attn.cpu().double(), t.res.cpu().double(), t.blk.topk_idx.cpu().long(), opt, [0, w.T])
        tgt = t.target.cpu().long()
        ce = torch.nn.functional.cross_entropy((y + h) @ P["head"].t(), tgt, ignore_index=-1)
        (ce + bal + z).backward()
        tol = TOL[dtype]
        total = f64(t.total)
        assert abs(total[0] / total[1] - float(ce)) < tol * float(ce) and total[1] == int((tgt >= 0).sum())
        errs = {n: rel_fro(f64(g), P[n].grad.numpy().reshape(g.shape)) for n, g in zip(t.names, t.grads)}
        assert all(e < tol for e in errs.values()), errs
        # the step on the gradients that were computed
        norm = np.sqrt(sum((f64(g) ** 2).sum() for g in t.grads))
        assert abs(float(t.opt.norm) - norm) < 1e-5 * norm
        factor = min(1.0, 0.5 / float(t.opt.norm))
        for i, n in enumerate(t.names):
            wd = 0.0 if t.params[i].dim() == 1 else 0.1
            want, _, _ = O.adamw(f64(before[n]).ravel(), f64(t.grads[i]).ravel(), *states[i], 1e-3, 0.9, 0.999, 1e-8, step, wd, factor)
            got = t.params[i] if t.opt.master[i] is None else t.opt.master[i]
            # a step moves a weight by about lr: 1e-3 of that, and the rounding of the weight
            assert np.abs(f64(got).ravel() - want).max() < 1e-6 + 2.0 ** -23 * np.abs(want).max(), n
            if t.opt.master[i] is not None:
                assert torch.equal(t.params[i], t.opt.master[i].bfloat16().view_as(t.params[i]))


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_in_a_graph(bits):
    """Captured and replayed steps move on as eager ones do, bit for bit, an eager run of the same program alive beside."""
    w = custom("train", T=64, H=64, F=64, E=16, k=2)
    eager = Trainer(w, 48, 300, bits, capturable=True)
    graph = Trainer(w, 48, 300, bits, capturable=True)
    for t in (eager, graph):
        t.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for _ in range(3):
        eager.step()
        g.replay()
    torch.cuda.synchronize()
    assert int(eager.opt.t) == int(graph.opt.t) == 4
    for a, b in zip(eager.params + [eager.loss], graph.params + [graph.loss]):
        assert torch.equal(a, b)
