"""The operators of a training step around the MoE layer, as cases to be timed and compared.

* balance: counts, mean probabilities, the balance loss and the z loss of router logits; their gradient.
* xent:    softmax cross entropy of x W over a large vocabulary; the loss alone, or with the gradients of x and W.
* norm:    the global norm of many gradient tensors.
* adamw:   one AdamW step over many tensors, with states in 32 bits or in 8 (e4m3 over a scale for 256 values;
           the second moment as its square root).

``run`` computes a case either in its plain form (elementary torch operations in 32 bits, rounded once at the
end) or, with ``own`` set, through the library's entry points. ``exact`` evaluates the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_F8 = torch.float8_e4m3fn
_BLOCK = 256          # values that share a scale of the 8-bit states
_TINY = 2.0 ** -126
_B1, _B2, _EPS, _LR, _WD, _STEP = 0.9, 0.95, 1e-8, 3e-4, 0.1, 100


# ---------------------------------------------------------------- cases
def listed() -> list[dict]:
    return [
        # the routing of a small batch: latency is all that counts
        dict(name="balance_fwd_t64", op="balance_fwd", T=64, E=128, k=8, S=0, tail=0, score="softmax", z=1e-3,
             dtype="f32", grad_dtype="f32", add=False),
        # a training step's router, packed sequences of uneven length with padding behind them, sigmoid scores
        dict(name="balance_fwd_t16384_seqs", op="balance_fwd", T=16384, E=256, k=8, S=37, tail=300, score="sigmoid",
             z=0.0, dtype="f32", grad_dtype="f32", add=False),
        # the gradient joining the gate's, in the type the router's products read
        dict(name="balance_bwd_t8192", op="balance_bwd", T=8192, E=128, k=8, S=0, tail=0, score="softmax", z=1e-3,
             dtype="f32", grad_dtype="bf16", add=True),
        # the loss of eight tokens: a stream of the head's weight
        dict(name="xent_fwd_m8", op="xent_fwd", M=8, H=2048, V=65536, dtype="bf16", tied=False, z=0.0),
        # the loss of a training step with both gradients, a large vocabulary
        dict(name="xent_train_m4096", op="xent_train", M=4096, H=2048, V=131072, dtype="bf16", tied=False, z=0.0),
        # an embedding table as the head, sizes that no tile divides, z loss
        dict(name="xent_train_tied_odd", op="xent_train", M=777, H=1000, V=50001, dtype="bf16", tied=True, z=1e-4),
        # 32-bit weights and activations
        dict(name="xent_train_f32", op="xent_train", M=500, H=768, V=10007, dtype="f32", tied=False, z=0.0),
        # every gradient of one layer (128 experts of 2048 x 768, projection, router, norm)
        dict(name="norm_layer", op="norm", set="layer", H=2048, F=768, E=128, A=4096, grad="bf16"),
        # many odd tensors: norms, biases, small projections
        dict(name="norm_many", op="norm", set="many", count=150, lo=1, hi=50000, sizes=1, grad="f32"),
        # the optimiser step of that layer: bf16 weights with 32-bit copies, clipped
        dict(name="adamw32_layer", op="adamw", set="layer", H=2048, F=768, E=128, A=4096, param="bf16", grad="bf16",
             master=True, bits=32, clip=True),
        # the same with the states in 8 bits and no 32-bit copy: memory counts
        dict(name="adamw8_layer", op="adamw", set="layer", H=2048, F=768, E=128, A=4096, param="bf16", grad="bf16",
             master=False, bits=8, clip=True),
        # many odd 32-bit tensors
        dict(name="adamw32_many", op="adamw", set="many", count=150, lo=1, hi=50000, sizes=2, param="f32", grad="f32",
             master=False, bits=32, clip=False),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _size(rng, lo: int, hi: int, step: int) -> int:
    """A size spread over the logarithm of the range: three quarters multiples of `step`, else any number."""
    v = _log_int(rng, lo, hi)
    if rng.random() < 0.75:
        v = min(hi, max(step, v // step * step))
    return v


def draw(rng) -> dict:
    op = rng.choice(["balance_fwd", "balance_bwd", "xent_fwd", "xent_train", "norm", "adamw", "adamw"])
    if op.startswith("balance"):
        T = _log_int(rng, 1, 32768)
        E = _size(rng, 8, 512, 8)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(16, E)), S=rng.choice([0, 0, _log_int(rng, 1, 64)]),
                    tail=rng.choice([0, 0, T // 7]), score=score,
                    z=1e-3 if score == "softmax" and rng.random() < 0.5 else 0.0, dtype=rng.choice(["f32", "f32", "bf16"]),
                    grad_dtype=rng.choice(["f32", "bf16"]), add=rng.random() < 0.5)
    if op.startswith("xent"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H = _size(rng, 32, 4096, 64)
        V = _size(rng, 500, 131072, 64)
        M = max(1, min(_log_int(rng, 1, 8192), (1_000_000_000_000 if dtype == "bf16" else 20_000_000_000) // (H * V)))
        return dict(op=op, M=M, H=H, V=V, dtype=dtype, tied=rng.random() < 0.5, z=rng.choice([0.0, 0.0, 1e-4]))
    if rng.random() < 0.4:
        H = 64 * _log_int(rng, 2, 32)
        size = dict(set="layer", H=H, F=64 * _log_int(rng, 1, 12), E=16 * _log_int(rng, 1, 8), A=H)
    else:
        hi = _log_int(rng, 10, 1_000_000)
        size = dict(set="many", count=_log_int(rng, 1, 300), lo=rng.randint(1, min(hi, 1000)), hi=hi,
                    sizes=rng.randint(0, 10 ** 6))
    if op == "norm":
        return dict(op=op, grad=rng.choice(["bf16", "f32"]), **size)
    param = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, param=param, grad=rng.choice(["f32", param]), master=param == "bf16" and rng.random() < 0.6,
                bits=rng.choice([8, 32]), clip=rng.random() < 0.5, **size)


# ---------------------------------------------------------------- inputs
def _gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _prepare_balance(case, g, st):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    pop = 0.7 * _randn(g, 1, E)  # experts differ in popularity
    st["logits"] = (1.3 * _randn(g, T, E) + pop).to(_DT[case["dtype"]])
    st["idx"] = st["logits"].float().topk(k, dim=1).indices.int().contiguous()
    st["start"] = None
    if S:  # sequences of uneven length, some of them empty, and rows of padding behind the last
        cut = torch.sort((_rand(g, S - 1) * (T - case["tail"] + 1)).int()).values
        end = torch.tensor([T - case["tail"]], dtype=torch.int32, device="cuda")
        st["start"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cut, end])
    if case["op"] == "balance_bwd":
        st["count"] = _balance_counts(st)
        st["dloss"] = torch.full((1,), 1.5, device="cuda")
        st["dadd"] = (1e-6 * _randn(g, T, E)).to(_DT[case["grad_dtype"]]) if case["add"] else None


def _prepare_xent(case, g, st):
    M, H, V = case["M"], case["H"], case["V"]
    dt = _DT[case["dtype"]]
    w = 0.9 / math.sqrt(H) * _randn(g, V, H)
    # targets as frequent as words are, some of them not to be counted
    target = (torch.exp(_rand(g, M) * math.log(V)) - 1.0).int().clamp(0, V - 1)
    x = _randn(g, M, H)
    if M > 1:
        target[1:][_rand(g, M - 1) < 0.1] = -100
    # what a model has learned: a target's logit stands out by up to what it takes to be likely
    known = _rand(g, M, 1) * (1.2 * math.log(V) / 0.81)
    x = x + known * w[target.clamp(min=0).long()] * (target >= 0)[:, None]
    st["x"], st["target"] = x.to(dt), target
    st["w"] = w.to(dt) if case["tied"] else w.to(dt).t().contiguous()


def _tensor_sizes(case):
    if case["set"] == "layer":
        H, F, E, A = case["H"], case["F"], case["E"], case["A"]
        return [A * H, H, H * E, E * H * F, E * H * F, E * F * H]
    r = random.Random(case["sizes"])
    return [_log_int(r, case["lo"], case["hi"]) for _ in range(case["count"])]


def _prepare_tensors(case, g, st):
    sizes = _tensor_sizes(case)
    # the tensors lie one behind another, each beginning at a multiple of 256 values, zeros between them
    at, n = [], 0
    for s in sizes:
        at.append(n)
        n += -(-s // _BLOCK) * _BLOCK
    st["at"], st["sizes"] = at, sizes
    gaps = [(a + s, -(-s // _BLOCK) * _BLOCK - s) for a, s in zip(at, sizes) if s % _BLOCK]

    def flat(t, dtype):
        t = t.to(dtype)
        for a, m in gaps:
            t[a:a + m] = 0
        return t

    scale = 1e-3 * torch.exp(1.5 * _randn(g, n // _BLOCK, 1))  # gradients differ from row to row
    st["g"] = flat((scale * _randn(g, n // _BLOCK, _BLOCK)).view(-1), _DT[case["grad"]])
    if case["op"] == "norm":
        return
    p = flat(0.02 * _randn(g, n), torch.float32)
    m = flat((0.3 * scale * _randn(g, n // _BLOCK, _BLOCK)).view(-1), torch.float32)
    v = flat((scale * (0.3 + _rand(g, n // _BLOCK, _BLOCK))).view(-1), torch.float32).square_()
    st["master"] = p if case["master"] else None
    st["p"] = p.to(_DT[case["param"]]) if case["param"] == "bf16" else p
    st["m"], st["v"], st["ms"], st["vs"] = m, v, None, None
    if case["bits"] == 8:
        st["m"], st["ms"] = _to8(m)
        st["v"], st["vs"] = _to8(torch.sqrt(v), True)
    st["norm"] = st["g"].float().square().sum(dtype=torch.float64).sqrt().float().view(1) if case["clip"] else None


def prepare(case: dict, seed: int) -> dict:
    st = dict(case=case)
    g = _gen(seed)
    op = case["op"]
    if op.startswith("balance"):
        _prepare_balance(case, g, st)
    elif op.startswith("xent"):
        _prepare_xent(case, g, st)
    else:
        _prepare_tensors(case, g, st)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """Output buffers, workspaces and descriptions, as a program that calls the library keeps them."""
    from expert_grouped_gemm_gb300 import _lib

    c = st["case"]
    op = c["op"]
    new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")
    if op.startswith("balance"):
        T, E, S = c["T"], c["E"], c["S"]
        d = st["dims"] = _lib.make_balance_dims(T, E, c["k"], S, c["score"], 0.01, c["z"], c["dtype"], c["grad_dtype"])
        if op == "balance_fwd":
            st["ws"] = _lib.alloc_balance_workspace(d)
            st["out"] = [new(2), new(max(S, 1), E, dtype=torch.int32), new(max(S, 1), E)]
        else:
            st["out"] = [new(T, E, dtype=_DT[c["grad_dtype"]])]
    elif op.startswith("xent"):
        M, H, V = c["M"], c["H"], c["V"]
        d = st["dims"] = _lib.make_xent_dims(M, H, V, c["dtype"], c["tied"], c["z"])
        st["ws"] = _lib.alloc_xent_workspace(d, backward=op == "xent_train")
        st["out"] = [new(M), new(M), new(2)]
        if op == "xent_train":
            st["out"] += [new(M, H, dtype=_DT[c["dtype"]]), torch.empty_like(st["w"])]
    else:
        cut = lambda t, k=1: None if t is None else [t[a // k:(a + s + k - 1) // k] for a, s in zip(st["at"], st["sizes"])]
        if op == "norm":
            st["tensors"] = _lib.make_grad_tensors(cut(st["g"]))
            st["out"] = [new(1)]
            st["ws"] = _lib.alloc_grad_norm_workspace(st["tensors"])
        else:
            st["tensors"] = _lib.make_adamw_tensors(
                cut(st["p"]), cut(st["g"]), cut(st["m"]), cut(st["v"]), master=cut(st["master"]),
                m_scale=cut(st["ms"], _BLOCK), v_scale=cut(st["vs"], _BLOCK), weight_decay=_WD)
            st["dims"] = _lib.make_adamw_dims(lr=_LR, beta1=_B1, beta2=_B2, eps=_EPS, step=_STEP, state_bits=c["bits"],
                                              max_norm=1.0 if c["clip"] else 0.0)


# ---------------------------------------------------------------- one pass
def run(state: dict):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"balance_fwd": _balance_fwd, "balance_bwd": _balance_bwd, "xent_fwd": _xent, "xent_train": _xent,
            "norm": _norm, "adamw": _adamw}[op](state)


def _run_own(st, op):
    from expert_grouped_gemm_gb300 import _lib

    if op == "balance_fwd":
        loss, count, prob = st["out"]
        _lib.moe_balance_fwd(st["dims"], st["ws"], st["logits"], st["idx"], st["start"], loss, count, prob)
        return st["out"]
    if op == "balance_bwd":
        _lib.moe_balance_bwd(st["dims"], st["logits"], st["count"], st["start"], st["dloss"], st["dadd"], st["out"][0])
        return st["out"]
    if op.startswith("xent"):
        o = st["out"]
        _lib.moe_xent_fwd(st["dims"], st["ws"], st["x"], st["w"], st["target"], o[0], o[1], o[2])
        if op == "xent_train":  # of the mean loss
            _lib.moe_xent_bwd(st["dims"], st["ws"], st["x"], st["w"], st["target"], o[1], None, o[2], o[3], o[4])
        return o
    if op == "norm":
        _lib.moe_grad_norm(st["tensors"], st["ws"], st["out"][0])
        return st["out"]
    _lib.moe_adamw_step(st["dims"], st["tensors"], st["norm"])
    return [st[n] for n in ("p", "master", "m", "v", "ms", "vs") if st[n] is not None]


def _probs(c, l):
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    s = 1.0 / (1.0 + torch.exp(-l))
    return s / s.sum(1, keepdim=True)


def _members(st):
    """[S, T]: which tokens are in which sequence, as 0 and 1."""
    T = st["case"]["T"]
    if st["start"] is None:
        return torch.ones(1, T, device="cuda")
    t = torch.arange(T, device="cuda")
    return ((t >= st["start"][:-1, None]) & (t < st["start"][1:, None])).float()


def _balance_counts(st):
    c = st["case"]
    hit = torch.zeros(c["T"], c["E"], device="cuda").scatter_(1, st["idx"].long(), 1.0)
    return (_members(st) @ hit).int()


def _balance_fwd(st):
    c = st["case"]
    E, k, alpha = c["E"], c["k"], 0.01
    l = st["logits"].float()
    inside = _members(st)
    n = inside.sum(1, keepdim=True)
    N = n.sum().clamp_min(1.0)
    count = _balance_counts(st)
    prob = inside @ _probs(c, l) / n.clamp_min(1.0)
    balance = alpha * (count.float() * prob).sum() * (E / k) / N
    mx = l.amax(1, keepdim=True)
    lse = torch.log(torch.exp(l - mx).sum(1)) + mx[:, 0]
    zloss = c["z"] * (lse * lse * inside.sum(0)).sum() / N
    return [torch.stack([balance, zloss]), count, prob]


def _balance_bwd(st):
    c = st["case"]
    E, k, alpha = c["E"], c["k"], 0.01
    l = st["logits"].float()
    inside = _members(st)
    n = inside.sum(1, keepdim=True)
    N = n.sum().clamp_min(1.0)
    p = _probs(c, l)
    co = inside.t() @ (st["count"].float() / n.clamp_min(1.0)) * (alpha * E / k / N) * st["dloss"]
    dl = p * (co - (p * co).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        dl = dl * (1.0 - 1.0 / (1.0 + torch.exp(-l)))
    if c["z"]:
        mx = l.amax(1, keepdim=True)
        lse = torch.log(torch.exp(l - mx).sum(1, keepdim=True)) + mx
        dl = dl + p * lse * (2.0 * c["z"] / N * st["dloss"]) * inside.sum(0)[:, None]
    if st["dadd"] is not None:
        dl = dl + st["dadd"].float()
    return [dl.to(_DT[c["grad_dtype"]])]


def _xent(st):
    c = st["case"]
    z = c["z"]
    x, w = st["x"].float(), st["w"].float()
    if c["tied"]:
        w = w.t()
    l = x @ w
    mx = l.amax(1, keepdim=True)
    e = torch.exp(l - mx)
    s = e.sum(1, keepdim=True)
    lse = (torch.log(s) + mx)[:, 0]
    counted = st["target"] >= 0
    at = st["target"].clamp(min=0).long()[:, None]
    loss = torch.where(counted, lse - l.gather(1, at)[:, 0] + z * lse * lse, 0.0)
    n = counted.float().sum()
    outs = [loss, lse, torch.stack([loss.sum(), n])]
    if c["op"] == "xent_fwd":
        return outs
    d = (counted.float() / n)[:, None]
    dl = e.mul_((1.0 + 2.0 * z * lse[:, None]) * d / s)
    dl.scatter_add_(1, at, -d)
    dt = _DT[c["dtype"]]
    dw = dl.t() @ x if c["tied"] else x.t() @ dl
    return outs + [(dl @ w.t()).to(dt), dw.to(dt)]


def _norm(st):
    return [st["g"].float().square().sum(dtype=torch.float64).sqrt().float().view(1)]


def _to8(x, positive=False):
    """Values in blocks of 256 as e4m3 over a scale each; where `positive`, what is not zero stays so."""
    b = x.view(-1, _BLOCK)
    scale = (b.abs().amax(1) / 448.0).clamp_min(_TINY)
    u = b / scale[:, None]
    if positive:
        u = torch.where(b > 0, u.clamp_min(2.0 ** -9), u)
    return u.to(_F8).view(-1), scale


def _from8(q, scale):
    return (q.float().view(-1, _BLOCK) * scale[:, None]).view(-1)


def _adamw(st):
    c = st["case"]
    g = st["g"].float()
    if c["clip"]:
        g = g * (1.0 / st["norm"].clamp_min(1.0))
    m, v = st["m"], st["v"]
    if c["bits"] == 8:
        m, v = _from8(m, st["ms"]), _from8(v, st["vs"]).square_()
    m.mul_(_B1).add_(g, alpha=1.0 - _B1)
    v.mul_(_B2).addcmul_(g, g, value=1.0 - _B2)
    r = torch.sqrt(v)
    u = (m / (1.0 - _B1 ** _STEP)) / (r / math.sqrt(1.0 - _B2 ** _STEP) + _EPS)
    if c["bits"] == 8:
        for name, x, positive in (("m", m, False), ("v", r, True)):
            q, scale = _to8(x, positive)
            st[name].copy_(q)
            st[name + "s"].copy_(scale)
    p = st["p"].float() if st["master"] is None else st["master"]
    u.add_(p, alpha=_WD)
    if c["param"] == "f32" or st["master"] is not None:
        p.add_(u, alpha=-_LR)
        if st["master"] is not None:
            st["p"].copy_(p)
    else:
        st["p"].copy_(p.add_(u, alpha=-_LR))
    return [st[n] for n in ("p", "master", "m", "v", "ms", "vs") if st[n] is not None]


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_balance(c, st):
    T, E, k = c["T"], c["E"], c["k"]
    l = st["logits"].double().requires_grad_(True)
    p = torch.softmax(l, 1)
    if c["score"] == "sigmoid":
        p = torch.special.expit(l)
        p = p / p.sum(1, keepdim=True)
    cuts = [0, T] if st["start"] is None else st["start"].tolist()
    N = max(1, cuts[-1] - cuts[0])
    total, counts, probs = 0.0, [], []
    for a, b in zip(cuts[:-1], cuts[1:]):
        hits = torch.bincount(st["idx"][a:b].flatten().long(), minlength=E).double()
        mean = p[a:b].sum(0) / max(1, b - a)
        total = total + 0.01 * E / k / N * torch.dot(hits, mean)
        counts.append(hits)
        probs.append(mean)
    zl = c["z"] / N * torch.logsumexp(l[cuts[0]:cuts[-1]], 1).square().sum()
    if c["op"] == "balance_fwd":
        return [torch.stack([total, zl]).detach(), torch.stack(counts).int(), torch.stack(probs).detach()]
    (dl,) = torch.autograd.grad((total + zl) * 1.5, l)
    return [dl + (0.0 if st["dadd"] is None else st["dadd"].double())]


def _exact_xent(c, st):
    train = c["op"] == "xent_train"
    x, w = st["x"].double().requires_grad_(train), st["w"].double().requires_grad_(train)
    l = torch.nn.functional.linear(x, w if c["tied"] else w.t())
    lse = torch.logsumexp(l, 1)
    counted = (st["target"] >= 0).double()
    own_logit = torch.take_along_dim(l, st["target"].clamp(min=0).long()[:, None], 1)[:, 0]
    loss = (lse - own_logit + c["z"] * lse ** 2) * counted
    outs = [loss.detach(), lse.detach(), torch.stack([loss.sum(), counted.sum()]).detach()]
    return outs + (list(torch.autograd.grad(loss.sum() / counted.sum(), (x, w))) if train else [])


def _exact8(x, positive):
    """(codes as their values, scales) on the grid of 4 exponent and 3 mantissa bits."""
    b = x.view(-1, _BLOCK)
    s = torch.maximum(b.abs().amax(1) / 448, torch.tensor(_TINY, dtype=torch.float64, device=x.device))
    u = b / s[:, None]
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))).clamp_max(8.0) - 3)
    q = torch.round(u / step) * step
    if positive:
        q = torch.where((b > 0) & (q == 0), 2.0 ** -9, q)
    return q.view(-1), s


def _exact_adamw(c, st):
    g = st["g"].double()
    if c["clip"]:
        g = g / max(1.0, float(st["norm"].double()))
    m, v = st["m"].double(), st["v"].double()
    if c["bits"] == 8:
        m = m * st["ms"].double().repeat_interleave(_BLOCK)
        v = (v * st["vs"].double().repeat_interleave(_BLOCK)) ** 2
    m = torch.lerp(g, m, _B1)
    v = torch.lerp(g * g, v, _B2)
    p = (st["p"] if st["master"] is None else st["master"]).double()
    p = p * (1 - _LR * _WD) - _LR / (1 - _B1 ** _STEP) * m / (torch.sqrt(v / (1 - _B2 ** _STEP)) + _EPS)
    outs = [p] + ([p] if st["master"] is not None else [])
    if c["bits"] == 32:
        return outs + [m, v]
    m8, ms = _exact8(m, False)
    v8, vs = _exact8(torch.sqrt(v), True)
    return outs + [m8, v8, ms, vs]


def exact(case: dict, seed: int):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"].startswith("balance"):
        return _exact_balance(case, st)
    if case["op"].startswith("xent"):
        return _exact_xent(case, st)
    if case["op"] == "norm":
        return [torch.linalg.vector_norm(st["g"].double()).view(1)]
    return _exact_adamw(case, st)


# ---------------------------------------------------------------- unavoidable work
def work(case: dict) -> dict:
    op = case["op"]
    if op.startswith("balance"):
        T, E, S = case["T"], case["E"], max(1, case["S"])
        es, gs = _ES[case["dtype"]], _ES[case["grad_dtype"]]
        if op == "balance_fwd":
            return dict(bytes=T * E * es + T * case["k"] * 4 + S * E * 8, flops=6 * T * E)
        return dict(bytes=T * E * (es + gs * (2 if case["add"] else 1)) + S * E * 4, flops=8 * T * E)
    if op.startswith("xent"):
        M, H, V = case["M"], case["H"], case["V"]
        n = 2 if op == "xent_train" else 1
        return dict(bytes=(M * H + H * V) * _ES[case["dtype"]] * n + 12 * M, flops=2 * M * H * V * (3 if n == 2 else 1))
    n = sum(_tensor_sizes(case))
    gs = _ES[case["grad"]]
    if op == "norm":
        return dict(bytes=n * gs, flops=2 * n)
    ps = _ES[case["param"]]
    weight = ps + 8 if case["master"] else 2 * ps
    return dict(bytes=n * (weight + gs + 4 * (case["bits"] // 8)), flops=14 * n)
