"""Refusals of the balance, cross entropy, norm and AdamW entry points that need no GPU."""
import ctypes

import pytest
import torch

from expert_grouped_gemm_gb300 import _lib, build
from expert_grouped_gemm_gb300.optim import AdamW

INV, UNS, WSP = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
FAKE, ODD = 0x10000, 0x10002  # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def balance(**kw):
    d = dict(T=4, E=64, k=4, S=0, score=0, dtype=1, grad_dtype=1, alpha=0.01, z_coef=0.0)
    d.update(kw)
    return _lib.BalanceDims(**d)


def xent(**kw):
    d = dict(M=4, H=64, V=1000, dtype=0, tied=0, z_coef=0.0)
    d.update(kw)
    return _lib.XentDims(**d)


BAD_BALANCE = [(dict(T=0), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(S=-1), INV), (dict(T=1 << 26), UNS),
               (dict(E=1025), UNS), (dict(k=33), UNS), (dict(S=(1 << 20) + 1), UNS), (dict(score=2), INV),
               (dict(dtype=2), INV), (dict(grad_dtype=-1), INV), (dict(alpha=NAN), INV), (dict(z_coef=INF), INV),
               (dict(score=1, z_coef=0.1), INV)]


@pytest.mark.parametrize("kw,code", BAD_BALANCE)
def test_balance_dims(lib, kw, code):
    d, n = balance(**kw), ctypes.c_size_t(0)
    assert lib.moe_balance_workspace_size(d, n) == code and _lib.moe_last_error()
    assert lib.moe_balance_fwd(d, FAKE, 1 << 40, None, FAKE, FAKE, FAKE if d.S else None, FAKE, FAKE, None) == code
    assert lib.moe_balance_bwd(d, None, FAKE, FAKE, FAKE if d.S else None, None, None, FAKE) == code


def test_balance_arguments(lib):
    def fwd(d, ws=FAKE, size=1 << 30, l=FAKE, i=FAKE, s=None, loss=FAKE, c=FAKE, p=None):
        return lib.moe_balance_fwd(d, ws, size, None, l, i, s, loss, c, p)

    def bwd(d, l=FAKE, c=FAKE, s=None, u=None, add=None, dl=FAKE):
        return lib.moe_balance_bwd(d, None, l, c, s, u, add, dl)

    d = balance()
    assert fwd(d, ws=None) == WSP and fwd(d, size=256) == WSP and fwd(d, ws=0x10010) == WSP
    for k in ("l", "i", "loss", "c"):
        assert fwd(d, **{k: None}) == INV and fwd(d, **{k: 0x10001}) == INV
    assert fwd(d, p=0x10001) == INV and fwd(d, s=FAKE) == INV and fwd(balance(S=2)) == INV
    assert bwd(d, l=None) == INV and bwd(d, c=None) == INV and bwd(d, dl=None) == INV and bwd(d, dl=ODD) == INV
    assert bwd(d, s=FAKE) == INV and bwd(balance(S=2)) == INV and bwd(d, u=ODD) == INV and bwd(d, add=ODD) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), INV), (dict(H=0), INV), (dict(V=0), INV), (dict(M=2 ** 31), UNS), (dict(H=1 << 24), UNS),
    (dict(V=1 << 24), UNS), (dict(dtype=5), INV), (dict(tied=2), INV), (dict(z_coef=NAN), INV)])
def test_xent_dims(lib, kw, code):
    d, n = xent(**kw), ctypes.c_size_t(0)
    assert lib.moe_xent_workspace_size(d, 1, n) == code and _lib.moe_last_error()
    assert lib.moe_xent_fwd(d, FAKE, 1 << 40, None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    assert lib.moe_xent_bwd(d, FAKE, 1 << 40, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == code


def test_xent_arguments(lib):
    d, n = xent(), ctypes.c_size_t(0)
    sizes = []
    for back in (0, 1):
        assert lib.moe_xent_workspace_size(d, back, n) == 0
        sizes.append(n.value)
    assert 256 <= sizes[0] <= sizes[1]

    def fwd(ws=FAKE, size=1 << 40, x=FAKE, w=FAKE, t=FAKE, loss=FAKE, lse=0x20000, total=None):
        return lib.moe_xent_fwd(d, ws, size, None, x, w, t, loss, lse, total)

    def bwd(ws=FAKE, size=1 << 40, x=FAKE, w=FAKE, t=FAKE, lse=FAKE, dl=FAKE, total=None, dx=0x30000, dw=0x40000):
        return lib.moe_xent_bwd(d, ws, size, None, x, w, t, lse, dl, total, dx, dw)

    assert fwd(ws=None) == WSP and fwd(size=sizes[0] - 1) == WSP and fwd(ws=0x10010) == WSP
    assert bwd(ws=None) == WSP and bwd(size=sizes[1] - 1) == WSP
    for k in ("x", "w", "t", "loss", "lse"):
        assert fwd(**{k: None}) == INV and fwd(**{k: 0x10001}) == INV
    for k in ("x", "w", "t", "lse"):
        assert bwd(**{k: None}) == INV and bwd(**{k: 0x10001}) == INV
    assert fwd(total=ODD) == INV and bwd(dx=ODD) == INV and bwd(dw=ODD) == INV
    assert fwd(lse=FAKE) == INV and fwd(total=FAKE) == INV and bwd(dx=FAKE) == INV and bwd(dw=FAKE) == INV
    assert bwd(dx=0x40000) == INV
    assert bwd(dl=None) == INV and bwd(total=FAKE) == INV and bwd(dx=None, dw=None) == INV


def test_xent_workspace_does_not_hold_the_logits(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_xent_workspace_size(xent(M=16384, H=4096, V=1 << 20), 1, n) == 0
    assert n.value < 16384 * (1 << 20) * 2 / 16


def entry(**kw):
    d = dict(param=FAKE, grad=FAKE, master=None, m=FAKE, v=FAKE, m_scale=None, v_scale=None, n=10, dtype=0, grad_dtype=0,
             lr_scale=1.0, weight_decay=0.0)
    d.update(kw)
    return _lib.AdamWTensor(**d)


def adamw_dims(**kw):
    d = dict(beta1=0.9, beta2=0.99, step=1, lr=0.1, eps=1e-8, grad_scale=1.0, max_norm=0.0, state_bits=32)
    d.update(kw)
    return _lib.AdamWDims(**d)


@pytest.mark.parametrize("kw", [
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=NAN), dict(step=0), dict(lr=INF), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=INF), dict(grad_scale=NAN), dict(max_norm=NAN), dict(state_bits=16)])
def test_adamw_dims(lib, kw):
    assert lib.moe_adamw_step(adamw_dims(**kw), entry(), 1, None, None, None, None) == INV and _lib.moe_last_error()


@pytest.mark.parametrize("kw", [
    dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=ODD), dict(grad=ODD), dict(m=ODD),
    dict(v=ODD), dict(master=ODD), dict(n=-1), dict(n=(1 << 40) + 1), dict(dtype=2), dict(grad_dtype=3),
    dict(lr_scale=INF), dict(weight_decay=NAN), dict(dtype=1, master=FAKE), dict(m_scale=FAKE)])
def test_adamw_tensors(lib, kw):
    e = (_lib.AdamWTensor * 2)(entry(), entry(**kw))
    assert lib.moe_adamw_step(adamw_dims(), e, 2, None, None, None, None) == INV
    assert "tensor 1" in _lib.moe_last_error()


def test_adamw_and_norm_arguments(lib):
    e = entry()
    assert lib.moe_adamw_step(None, e, 1, None, None, None, None) == INV
    assert lib.moe_adamw_step(adamw_dims(), e, -1, None, None, None, None) == INV
    assert lib.moe_adamw_step(adamw_dims(), None, 1, None, None, None, None) == INV
    for i in range(3):
        p = [None] * 3
        p[i] = ODD
        assert lib.moe_adamw_step(adamw_dims(), e, 1, None, *p) == INV
    assert lib.moe_adamw_step(adamw_dims(state_bits=8), e, 1, None, None, None, None) == INV  # no scales
    assert lib.moe_adamw_step(adamw_dims(), None, 0, None, None, None, None) == 0             # nothing to do
    n = ctypes.c_size_t(0)
    assert lib.moe_grad_norm_workspace_size(e, 1, n) == 0 and n.value > 256
    norm = lambda t=e, ws=FAKE, size=1 << 30, scale=1.0, out=FAKE: lib.moe_grad_norm(t, 1, ws, size, None, scale, out)
    assert norm(ws=None) == WSP and norm(size=256) == WSP and norm(scale=INF) == INV and norm(out=None) == INV
    assert norm(t=None) == INV and norm(t=entry(grad=None)) == INV and norm(t=entry(grad=ODD)) == INV


def test_bindings_name_what_is_wrong():
    with pytest.raises(ValueError, match="score"):
        _lib.make_balance_dims(4, 64, 4, score="max")
    with pytest.raises(ValueError, match="dtype"):
        _lib.make_xent_dims(4, 64, 100, dtype="f16")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _lib.moe_xent_fwd(_lib.make_xent_dims(4, 64, 100), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _lib.moe_balance_bwd(_lib.make_balance_dims(4, 64, 4), x, x, None, None, None, x)
    with pytest.raises(ValueError, match="grads.0. must be a CUDA tensor"):
        _lib.make_grad_tensors([x])
    with pytest.raises(ValueError, match="params.0. must be a CUDA tensor"):
        _lib.make_adamw_tensors([x], [x], [x], [x])
    with pytest.raises(ValueError, match="grads must have 1 entries"):
        _lib.make_adamw_tensors([x], [x, x], [x], [x])
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([x], [x], 0.1, state_bits=4)
