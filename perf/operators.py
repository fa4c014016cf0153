"""The operators around the experts of one transformer layer, as cases to be timed and compared.

Three operators, each forward and backward:

* norm:   h = x + residual; layer norm or RMS norm of h; backward with the weight's and bias's gradients.
* gate:   routing scores (softmax or sigmoid), a balance bias that only selects, groups of experts, top-k,
          renormalised and scaled weights; backward to the router logits.
* linear: y = act(x W + bias) + residual; backward to x, W and the bias.

``run`` computes a case either in its plain form (elementary torch operations in 32 bits, rounded once at the
end) or, with ``own`` set, through the library's entry points. ``exact`` evaluates the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed() -> list[dict]:
    return [
        # one token of a decoding step entering a layer: latency is all that counts
        dict(name="norm_fwd_one_token", op="norm_fwd", T=1, H=2048, dtype="bf16", kind="rms", residual=True),
        # the norm before the experts of a training step
        dict(name="norm_fwd_t4096", op="norm_fwd", T=4096, H=2048, dtype="bf16", kind="layer", residual=True),
        # its backward at the wide layer, the gradient of the residual stream joining in
        dict(name="norm_bwd_t8192", op="norm_bwd", T=8192, H=4096, dtype="bf16", kind="layer", residual=True),
        # 32-bit values and a width no vector divides
        dict(name="norm_bwd_f32_odd", op="norm_bwd", T=1001, H=1111, dtype="f32", kind="layer", residual=False),
        # routing of a small decoding batch
        dict(name="gate_fwd_t8", op="gate_fwd", T=8, E=128, k=8, n_group=1, topk_group=1, group_take=1,
             score="softmax", renorm=True, scale=1.0, bias=False, dtype="f32", grad_dtype="f32"),
        # routing of a training step: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="gate_fwd_t8192_groups", op="gate_fwd", T=8192, E=256, k=8, n_group=8, topk_group=4, group_take=2,
             score="sigmoid", renorm=True, scale=2.5, bias=True, dtype="f32", grad_dtype="f32"),
        # backward without renormalisation: every logit gets a gradient; bf16 logits, ragged sizes
        dict(name="gate_bwd_t4097_dense", op="gate_bwd", T=4097, E=160, k=6, n_group=8, topk_group=3, group_take=1,
             score="softmax", renorm=False, scale=16.0, bias=False, dtype="bf16", grad_dtype="bf16"),
        # output projection of a small decoding batch, back onto the residual stream: a stream of the weight
        dict(name="linear_fwd_m4", op="linear_fwd", M=4, K=4096, N=4096, dtype="bf16", act="none", bias=True,
             residual=True, save=False, out_f32=False),
        # first half of a dense MLP in training (the value before the activation is kept)
        dict(name="linear_fwd_m4096_gelu", op="linear_fwd", M=4096, K=2048, N=8192, dtype="bf16", act="gelu",
             bias=True, residual=False, save=True, out_f32=False),
        # backward of a wide projection
        dict(name="linear_bwd_m8192_silu", op="linear_bwd", M=8192, K=4096, N=4096, dtype="bf16", act="silu",
             bias=True),
        # sizes that no tile and no 16-byte row divides
        dict(name="linear_fwd_odd", op="linear_fwd", M=777, K=1001, N=1111, dtype="bf16", act="relu", bias=True,
             residual=True, save=False, out_f32=False),
        # 32-bit weights and activations
        dict(name="linear_bwd_f32", op="linear_bwd", M=300, K=768, N=1000, dtype="f32", act="gelu_tanh", bias=True),
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
    op = rng.choice(["norm_fwd", "norm_bwd", "gate_fwd", "gate_bwd", "linear_fwd", "linear_bwd"])
    if op.startswith("norm"):
        H = _size(rng, 64, 8192, 64)
        T = _log_int(rng, 1, min(16384, (1 << 25) // H))
        return dict(op=op, T=T, H=H, dtype=rng.choice(["bf16", "bf16", "f32"]), kind=rng.choice(["layer", "rms"]),
                    residual=rng.random() < 0.5)
    if op.startswith("gate"):
        G = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, max(2, 8 // G), 512 // G)
        E = G * per
        Kg = rng.randint(max(1, G // 4), G)
        k = rng.randint(1, min(16, Kg * per))
        renorm = rng.random() < 0.6 and (op == "gate_fwd" or k > 1)  # one renormalised weight has no gradient
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, n_group=G, topk_group=Kg,
                    group_take=rng.randint(1, 2), score=rng.choice(["softmax", "sigmoid"]), renorm=renorm,
                    scale=rng.choice([1.0, 2.5]), bias=rng.random() < 0.5, dtype=rng.choice(["f32", "f32", "bf16"]),
                    grad_dtype=rng.choice(["f32", "bf16"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    K = _size(rng, 32, 4096, 64)
    if dtype == "bf16":
        N = _size(rng, 32, 8192 if op == "linear_fwd" else 4096, 64)
        M = _log_int(rng, 1, 8192)
    else:
        N = _size(rng, 32, 4096, 64)
        M = max(1, min(_log_int(rng, 1, 4096), 8_000_000_000 // (K * N)))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    case = dict(op=op, M=M, K=K, N=N, dtype=dtype, act=act, bias=rng.random() < 0.7)
    if op == "linear_fwd":
        out_f32 = rng.random() < 0.15
        case.update(residual=not out_f32 and rng.random() < 0.5, save=not out_f32 and act != "none" and rng.random() < 0.5,
                    out_f32=out_f32)
    return case


# ---------------------------------------------------------------- inputs
def _gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hidden(g, T, H):
    """A residual stream: unit noise, a common shift and a few channels that are much larger than the rest."""
    x = _randn(g, T, H)
    col = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.004).float()
    return x * col + 0.1 * _randn(g, 1, H) + 0.05


def _choice64(case, logits, bias):
    """Choice scores, group scores and the selectable choice scores of the definition, in 64 bits."""
    l = logits.double()
    if case["score"] == "softmax":
        s = torch.softmax(l, 1)
    else:
        s = torch.special.expit(l)
    c = s if bias is None else s + bias.double()
    T, E = c.shape
    G = case["n_group"]
    top = c.view(T, G, E // G).topk(min(case["group_take"], E // G), dim=2).values
    gs = top.sum(2)
    gi = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
    keep = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, gi, True)
    sel = c.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    return s, gs, sel


def _undecided(case, logits, bias):
    """Rows whose selection or slot order rests on a difference that 32-bit rounding can turn over."""
    _, gs, sel = _choice64(case, logits, bias)
    k, Kg = case["k"], case["topk_group"]

    def close(v, n):  # among the n + 1 largest (n large ones and the first that is left out)
        v = torch.sort(v, dim=1, descending=True).values[:, :n + 1]
        a, b = v[:, :-1], v[:, 1:]
        d = a - b
        tol = 4e-6 * torch.maximum(a.abs(), b.abs()).clamp_min(0.1 if bias is not None else 1e-30)
        return ((d > 0) & (d < tol)).any(1)

    bad = close(sel, min(k, sel.shape[1] - 1)) if sel.shape[1] > 1 else torch.zeros(len(sel), dtype=torch.bool,
                                                                                     device=sel.device)
    if case["n_group"] > Kg:
        v = torch.sort(gs, dim=1, descending=True).values[:, Kg - 1:Kg + 1]
        d = v[:, 0] - v[:, 1]
        bad |= (d > 0) & (d < 4e-6 * v.abs().amax(1).clamp_min(0.1 if bias is not None else 1e-30))
    return bad


def _gate_inputs(case, g):
    T, E = case["T"], case["E"]
    pop = 0.5 * _randn(g, 1, E)  # experts differ in popularity
    dt = _DT[case["dtype"]]
    bias = None
    if case["bias"]:  # what an update of fixed step leaves: multiples of 0.001
        bias = torch.randint(-100, 101, (E,), generator=g, device="cuda").float() * 1e-3
    logits = (1.3 * _randn(g, T, E) + pop).to(dt)
    for _ in range(30):  # indices are compared as whole numbers: rows that rounding would decide are drawn again
        bad = _undecided(case, logits, bias)
        n = int(bad.sum())
        if n == 0:
            break
        logits[bad] = (1.3 * _randn(g, n, E) + pop).to(dt)
    return logits, bias


def prepare(case: dict, seed: int) -> dict:
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    dt = _DT[case["dtype"]]
    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        x = _hidden(g, T, H).to(dt)
        st["weight"] = (1.0 + 0.2 * _randn(g, H)).to(dt)
        layer = case["kind"] == "layer"
        if op == "norm_fwd":
            st["x"] = x
            st["bias"] = (0.1 * _randn(g, H)).to(dt) if layer else None
            st["residual"] = _hidden(g, T, H).to(dt) if case["residual"] else None
        else:
            st["x"] = x
            xf = x.float()
            st["mean"] = xf.mean(1) if layer else None
            v = xf.var(1, unbiased=False) if layer else xf.square().mean(1)
            st["rstd"] = torch.rsqrt(v + _EPS)
            st["dy"] = _randn(g, T, H).to(dt)
            st["dsum"] = _randn(g, T, H).to(dt) if case["residual"] else None
    elif op.startswith("gate"):
        st["logits"], st["bias"] = _gate_inputs(case, g)
        if op == "gate_bwd":
            _, _, sel = _choice64(case, st["logits"], st["bias"])
            st["idx"] = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :case["k"]].int().contiguous()
            st["dw"] = _randn(g, case["T"], case["k"])
    else:
        M, K, N = case["M"], case["K"], case["N"]
        st["x"] = _randn(g, M, K).to(dt)
        st["w"] = (0.02 * _randn(g, K, N)).to(dt)
        st["bias"] = (0.1 * _randn(g, N)).to(dt) if case["bias"] else None
        if op == "linear_fwd":
            st["residual"] = _randn(g, M, N).to(dt) if case["residual"] else None
        else:
            st["dy"] = _randn(g, M, N).to(dt)
            st["pre"] = None
            if case["act"] != "none":
                z = st["x"].float() @ st["w"].float()
                st["pre"] = (z if st["bias"] is None else z + st["bias"].float()).to(dt)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """Output buffers, workspace and problem description, as a program that calls the library keeps them."""
    from expert_grouped_gemm_gb300 import _lib

    c = st["case"]
    op = c["op"]
    dt = _DT[c["dtype"]]
    new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device="cuda")
    if op.startswith("norm"):
        T, H = c["T"], c["H"]
        d = st["dims"] = _lib.make_norm_dims(T, H, c["dtype"], c["kind"], _EPS)
        layer = c["kind"] == "layer"
        if op == "norm_fwd":
            st["out"] = dict(y=new(T, H), sum=new(T, H) if c["residual"] else None,
                             mean=new(T, dtype=torch.float32) if layer else None, rstd=new(T, dtype=torch.float32))
        else:
            st["out"] = dict(dx=new(T, H), dweight=new(H), dbias=new(H) if layer else None)
            st["ws"] = _lib.alloc_norm_workspace(d)
    elif op.startswith("gate"):
        T, E, k = c["T"], c["E"], c["k"]
        st["dims"] = _lib.make_gate_dims(T, E, k, c["score"], c["renorm"], c["scale"], c["n_group"], c["topk_group"],
                                         c["group_take"], c["dtype"], c["grad_dtype"])
        if op == "gate_fwd":
            st["out"] = dict(idx=new(T, k, dtype=torch.int32), w=new(T, k, dtype=torch.float32),
                             count=new(E, dtype=torch.int32))
        else:
            st["out"] = dict(dlogits=new(T, E, dtype=_DT[c["grad_dtype"]]))
    else:
        M, K, N = c["M"], c["K"], c["N"]
        d = st["dims"] = _lib.make_linear_dims(M, K, N, c["dtype"], c["act"], c.get("out_f32", False))
        st["ws"] = _lib.alloc_linear_workspace(d)
        if op == "linear_fwd":
            st["out"] = dict(y=new(M, N, dtype=torch.float32 if c["out_f32"] else dt), pre=new(M, N) if c["save"] else None)
        else:
            st["out"] = dict(dx=new(M, K), dw=new(K, N), dbias=new(N) if c["bias"] else None)


# ---------------------------------------------------------------- one pass
def run(state: dict):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "gate_fwd": _gate_fwd, "gate_bwd": _gate_bwd,
            "linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd}[op](state)


def _run_own(st, op):
    from expert_grouped_gemm_gb300 import _lib

    d, o = st["dims"], st["out"]
    if op == "norm_fwd":
        _lib.moe_norm_fwd(d, st["x"], st["residual"], st["weight"], st["bias"], o["y"], o["sum"], o["mean"], o["rstd"])
        return [t for t in (o["y"], o["sum"], o["mean"], o["rstd"]) if t is not None]
    if op == "norm_bwd":
        _lib.moe_norm_bwd(d, st["ws"], st["dy"], st["dsum"], st["x"], st["weight"], st["mean"], st["rstd"], o["dx"],
                          o["dweight"], o["dbias"])
        return [t for t in (o["dx"], o["dweight"], o["dbias"]) if t is not None]
    if op == "gate_fwd":
        _lib.moe_gate_fwd(d, st["logits"], st["bias"], o["idx"], o["w"], o["count"])
        return [o["idx"], o["w"], o["count"]]
    if op == "gate_bwd":
        _lib.moe_gate_bwd(d, st["logits"], st["idx"], st["dw"], o["dlogits"])
        return [o["dlogits"]]
    if op == "linear_fwd":
        _lib.moe_linear_fwd(d, st["ws"], st["x"], st["w"], st["bias"], st["residual"], o["y"], o["pre"])
        return [t for t in (o["y"], o["pre"]) if t is not None]
    _lib.moe_linear_bwd(d, st["ws"], st["dy"], st["x"], st["w"], st["pre"], o["dx"], o["dw"], o["dbias"])
    return [t for t in (o["dx"], o["dw"], o["dbias"]) if t is not None]


def _norm_fwd(st):
    c = st["case"]
    dt = _DT[c["dtype"]]
    h = st["x"].float()
    if c["residual"]:
        h = h + st["residual"].float()
    outs = []
    if c["kind"] == "layer":
        mean = h.sum(1, keepdim=True) / c["H"]
        d = h - mean
    else:
        mean, d = None, h
    rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / c["H"] + _EPS)
    y = d * rstd * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    outs.append(y.to(dt))
    if c["residual"]:
        outs.append(h.to(dt))
    if mean is not None:
        outs.append(mean[:, 0])
    outs.append(rstd[:, 0])
    return outs


def _norm_bwd(st):
    c = st["case"]
    dt = _DT[c["dtype"]]
    dy, x, rstd = st["dy"].float(), st["x"].float(), st["rstd"][:, None]
    layer = c["kind"] == "layer"
    xh = (x - st["mean"][:, None]) * rstd if layer else x * rstd
    gy = dy * st["weight"].float()
    dx = gy - xh * ((gy * xh).sum(1, keepdim=True) / c["H"])
    if layer:
        dx = dx - gy.sum(1, keepdim=True) / c["H"]
    dx = dx * rstd
    if c["residual"]:
        dx = dx + st["dsum"].float()
    outs = [dx.to(dt), (dy * xh).sum(0).to(dt)]
    if layer:
        outs.append(dy.sum(0).to(dt))
    return outs


def _scores(c, l):
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-l))


def _gate_fwd(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    s = _scores(c, st["logits"].float())
    choice = s if st["bias"] is None else s + st["bias"]
    if G > 1:
        per = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        gs = per[:, :, :c["group_take"]].sum(2)
        gi = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = (gi[:, :, None] == torch.arange(G, device=gi.device)).any(1)
        choice = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), choice, -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    count = torch.zeros(E, dtype=torch.int32, device=w.device)
    count.index_add_(0, idx.reshape(-1), torch.ones(T * k, dtype=torch.int32, device=w.device))
    return [idx.int(), w, count]


def _gate_bwd(st):
    c = st["case"]
    s = _scores(c, st["logits"].float())
    idx = st["idx"].long()
    ws = s.gather(1, idx)
    dw = st["dw"] * c["scale"]
    if c["renorm"]:
        S = ws.sum(1, keepdim=True)
        dw = (dw - (dw * ws).sum(1, keepdim=True) / S) / S
    ds = torch.zeros_like(s).scatter_(1, idx, dw)
    if c["score"] == "softmax":
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    else:
        dl = ds * s * (1.0 - s)
    return [dl.to(_DT[c["grad_dtype"]])]


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _dact(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _linear_fwd(st):
    c = st["case"]
    dt = _DT[c["dtype"]]
    z = st["x"].float() @ st["w"].float()
    if c["bias"]:
        z = z + st["bias"].float()
    y = _act(c["act"], z)
    if c["residual"]:
        y = y + st["residual"].float()
    outs = [y if c["out_f32"] else y.to(dt)]
    if c["save"]:
        outs.append(z.to(dt))
    return outs


def _linear_bwd(st):
    c = st["case"]
    dt = _DT[c["dtype"]]
    dz = st["dy"].float()
    if c["act"] != "none":
        dz = dz * _dact(c["act"], st["pre"].float())
    outs = [(dz @ st["w"].float().t()).to(dt), (st["x"].float().t() @ dz).to(dt)]
    if c["bias"]:
        outs.append(dz.sum(0).to(dt))
    return outs


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_act(name, z):
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.special.expit(z)
    return z


def exact(case: dict, seed: int):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    D = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "norm_fwd":
        h = D["x"] + D["residual"] if case["residual"] else D["x"]
        layer = case["kind"] == "layer"
        mean = h.mean(1)
        var = h.var(1, unbiased=False) if layer else h.square().mean(1)
        rstd = (var + _EPS).rsqrt()
        hh = torch.addcmul(-mean[:, None] * rstd[:, None], h, rstd[:, None]) if layer else h * rstd[:, None]
        y = hh * D["weight"] + (D["bias"] if layer else 0.0)
        return [y] + ([h] if case["residual"] else []) + ([mean] if layer else []) + [rstd]
    if op == "norm_bwd":
        x, dy, w, r = D["x"], D["dy"], D["weight"], D["rstd"]
        n = case["H"]
        layer = case["kind"] == "layer"
        xh = torch.einsum("th,t->th", x - D["mean"][:, None] if layer else x, r)
        a = torch.einsum("th,h,th->t", dy, w, xh) / n
        b = torch.einsum("th,h->t", dy, w) / n if layer else torch.zeros_like(a)
        dx = torch.einsum("th,h,t->th", dy, w, r) - (xh * a[:, None] + b[:, None]) * r[:, None]
        if case["residual"]:
            dx = dx + D["dsum"]
        return [dx, torch.einsum("th,th->h", dy, xh)] + ([dy.sum(0)] if layer else [])
    if op == "gate_fwd":
        s, _, sel = _choice64(case, st["logits"], st["bias"])
        idx = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        w = torch.take_along_dim(s, idx, 1)
        if case["renorm"]:
            w = torch.nn.functional.normalize(w, p=1.0, dim=1, eps=0.0)
        count = torch.bincount(idx.flatten(), minlength=case["E"])
        return [idx.int(), w * case["scale"], count.int()]
    if op == "gate_bwd":
        l = D["logits"].requires_grad_(True)
        s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.special.expit(l)
        w = torch.take_along_dim(s, st["idx"].long(), 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (dl,) = torch.autograd.grad((w * case["scale"] * D["dw"]).sum(), l)
        return [dl]
    if op == "linear_fwd":
        z = torch.matmul(D["x"], D["w"])
        if case["bias"]:
            z += D["bias"]
        y = _exact_act(case["act"], z)
        if case["residual"]:
            y = y + D["residual"]
        return [y] + ([z] if case["save"] else [])
    dz = D["dy"]
    if case["act"] != "none":
        z = D["pre"].requires_grad_(True)
        (dz,) = torch.autograd.grad(_exact_act(case["act"], z), z, D["dy"])
    return [torch.matmul(dz, D["w"].t()), torch.matmul(D["x"].t(), dz)] + ([dz.sum(0)] if case["bias"] else [])


# ---------------------------------------------------------------- unavoidable work
def work(case: dict) -> dict:
    op = case["op"]
    es = _ES[case["dtype"]]
    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        r = 1 if case["residual"] else 0
        layer = case["kind"] == "layer"
        stat = 4 * T * (2 if layer else 1)
        if op == "norm_fwd":
            return dict(bytes=T * H * es * (2 + 2 * r) + H * es * (2 if layer else 1) + stat, flops=8 * T * H)
        return dict(bytes=T * H * es * (3 + r) + H * es * (3 if layer else 2) + stat, flops=14 * T * H)
    if op.startswith("gate"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "gate_fwd":
            return dict(bytes=T * E * es + T * k * 8 + E * (8 if case["bias"] else 4), flops=6 * T * E)
        return dict(bytes=T * E * (es + _ES[case["grad_dtype"]]) + T * k * 8, flops=8 * T * E)
    M, K, N = case["M"], case["K"], case["N"]
    if op == "linear_fwd":
        oe = 4 if case["out_f32"] else es
        b = (M * K + K * N) * es + M * N * (oe + es * (int(case["residual"]) + int(case["save"])))
        return dict(bytes=b + (N * es if case["bias"] else 0), flops=2 * M * K * N)
    pre = 1 if case["act"] != "none" else 0
    b = (M * N * (1 + pre) + 2 * M * K + 2 * K * N) * es + (N * es if case["bias"] else 0)
    return dict(bytes=b, flops=4 * M * K * N)
