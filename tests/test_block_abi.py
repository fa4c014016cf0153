"""Refusals of the norm, gate and linear entry points that need no GPU: every argument check comes before
anything is enqueued, and the binding hands over no host tensors."""
import ctypes

import pytest
import torch

from expert_grouped_gemm_gb300 import _lib, build

INV, UNS, WSP = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
FAKE, ODD = 0x10000, 0x10002  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def norm(**kw):
    d = dict(T=4, H=64, dtype=0, kind=0, eps=1e-5)
    d.update(kw)
    return _lib.NormDims(**d)


def gate(**kw):
    d = dict(T=4, E=64, k=4, n_group=1, topk_group=1, group_take=1, score=0, renorm=1, dtype=1, grad_dtype=1, scale=1.0)
    d.update(kw)
    return _lib.GateDims(**d)


def linear(**kw):
    d = dict(M=4, K=64, N=64, dtype=0, act=0, out_f32=0)
    d.update(kw)
    return _lib.LinearDims(**d)


def fwd_norm(lib, d, **kw):
    a = dict(x=FAKE, res=None, w=FAKE, b=None, y=FAKE, sum=None, mean=None, rstd=None)
    a.update(kw)
    return lib.moe_norm_fwd(ctypes.byref(d), None, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INV), (dict(H=0), INV), (dict(H=65537), UNS), (dict(T=2 ** 31), UNS), (dict(dtype=7), INV),
    (dict(kind=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV)])
def test_norm_dims(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert lib.moe_norm_workspace_size(ctypes.byref(norm(**kw)), ctypes.byref(n)) == code
    assert fwd_norm(lib, norm(**kw)) == code and _lib.moe_last_error()


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=ODD), dict(y=ODD), dict(b=ODD), dict(sum=0x20000),
    dict(res=FAKE, sum=FAKE), dict(mean=0x10001), dict(rstd=0x10001)])
def test_norm_fwd_arguments(lib, kw):
    assert fwd_norm(lib, norm(), **kw) == INV


def test_norm_mean_belongs_to_layer_norm(lib):
    assert fwd_norm(lib, norm(kind=1), mean=FAKE) == INV
    ws = lambda d: (FAKE, 1 << 30)
    call = lambda d, mean, w=FAKE, n=1 << 30: lib.moe_norm_bwd(ctypes.byref(d), w, n, None, FAKE, None, FAKE, FAKE, mean,
                                                               FAKE, FAKE, FAKE, None)
    assert call(norm(kind=1), FAKE) == INV
    assert call(norm(kind=0), None) == INV
    assert call(norm(), FAKE, None) == WSP
    assert call(norm(), FAKE, 0x10010) == WSP
    assert call(norm(), FAKE, FAKE, 16) == WSP


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=65), INV), (dict(E=1025), UNS),
    (dict(T=1 << 26), UNS), (dict(E=128, k=33), UNS), (dict(n_group=0), INV), (dict(n_group=5), INV),
    (dict(E=66, n_group=33), UNS), (dict(n_group=8, topk_group=9), INV), (dict(topk_group=0), INV),
    (dict(n_group=16, topk_group=1, k=5), INV), (dict(group_take=0), INV), (dict(group_take=3), INV),
    (dict(score=2), INV), (dict(scale=float("inf")), INV), (dict(dtype=2), INV), (dict(grad_dtype=-1), INV)])
def test_gate_dims(lib, kw, code):
    d = gate(**kw)
    assert lib.moe_gate_fwd(ctypes.byref(d), None, FAKE, None, FAKE, FAKE, None) == code and _lib.moe_last_error()
    assert lib.moe_gate_bwd(ctypes.byref(d), None, FAKE, FAKE, FAKE, FAKE) == code


@pytest.mark.parametrize("at", [0, 2, 3])
def test_gate_null_arguments(lib, at):
    a = [FAKE, None, FAKE, FAKE, None]
    a[at] = None
    assert lib.moe_gate_fwd(ctypes.byref(gate()), None, *a) == INV
    b = [FAKE] * 4
    b[at] = None
    assert lib.moe_gate_bwd(ctypes.byref(gate()), None, *b) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(M=2 ** 31), UNS), (dict(K=1 << 24), UNS),
    (dict(N=1 << 24), UNS), (dict(act=5), INV), (dict(act=-1), INV), (dict(out_f32=2), INV), (dict(dtype=3), INV)])
def test_linear_dims(lib, kw, code):
    n = ctypes.c_size_t(0)
    d = linear(**kw)
    assert lib.moe_linear_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.moe_linear_fwd(ctypes.byref(d), FAKE, 1 << 40, None, FAKE, FAKE, None, None, FAKE, None) == code


def test_linear_arguments(lib):
    n = ctypes.c_size_t(0)
    d = linear()
    assert lib.moe_linear_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value >= 4096

    def fwd(d, ws=FAKE, size=1 << 30, x=FAKE, w=FAKE, b=None, r=None, y=0x20000, pre=None):
        return lib.moe_linear_fwd(ctypes.byref(d), ws, size, None, x, w, b, r, y, pre)

    def bwd(d, ws=FAKE, size=1 << 30, dy=FAKE, x=FAKE, w=FAKE, pre=None, add=None, dx=FAKE, dw=FAKE, db=None):
        return lib.moe_linear_bwd(ctypes.byref(d), ws, size, None, dy, x, w, pre, add, dx, dw, db)

    assert fwd(d, ws=None) == WSP and fwd(d, size=4095) == WSP and fwd(d, ws=0x10080) == WSP
    for k in ("x", "w", "y"):
        assert fwd(d, **{k: None}) == INV and fwd(d, **{k: ODD}) == INV
    for k in ("b", "r", "pre"):
        assert fwd(d, **{k: ODD}) == INV
    assert fwd(d, pre=0x20000) == INV
    assert fwd(linear(out_f32=1), r=0x20000) == INV
    assert bwd(linear(act=2)) == INV            # the activation's input is missing
    assert bwd(linear(), pre=FAKE) == INV       # and here there is no activation
    assert bwd(linear(), dy=None) == INV
    assert bwd(linear(), add=FAKE, dx=None) == INV and bwd(linear(), add=ODD) == INV
    assert bwd(linear(), x=None) == INV and bwd(linear(), w=None) == INV


def test_binding_checks_shapes_types_and_devices(lib):
    d = _lib.make_norm_dims(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _lib.moe_norm_fwd(d, x, None, x[0], None, x)
    with pytest.raises(ValueError, match="kind"):
        _lib.make_norm_dims(4, 64, kind="batch")
    with pytest.raises(ValueError, match="score"):
        _lib.make_gate_dims(4, 64, 4, score="max")
    with pytest.raises(ValueError, match="act"):
        _lib.make_linear_dims(4, 64, 64, act="tanh")
    with pytest.raises(ValueError, match="dtype"):
        _lib.make_linear_dims(4, 64, 64, dtype="f16")


@pytest.mark.gpu
def test_binding_checks_of_device_tensors(lib):
    d = _lib.make_norm_dims(4, 64)
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf, device="cuda"), torch.zeros(64, dtype=bf, device="cuda")
    y = torch.zeros_like(x)
    with pytest.raises(TypeError, match="weight"):
        _lib.moe_norm_fwd(d, x, None, w.float(), None, y)
    with pytest.raises(ValueError, match="shape"):
        _lib.moe_norm_fwd(d, x[:3], None, w, None, y)
    with pytest.raises(ValueError, match="contiguous"):
        _lib.moe_norm_fwd(d, torch.zeros(64, 4, dtype=bf, device="cuda").t(), None, w, None, y)
    with pytest.raises(ValueError, match="required"):
        _lib.moe_norm_fwd(d, x, None, None, None, y)
    with pytest.raises(_lib.MoeError, match="aligned"):
        _lib.moe_norm_fwd(_lib.make_norm_dims(1, 64), torch.zeros(65, dtype=bf, device="cuda")[1:].view(1, 64), None, w, None,
                          torch.zeros(1, 64, dtype=bf, device="cuda"))
