"""Digits that a rounding of a shared factor, of a sum near one or of a large sum would cost the training operators."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from tests import train_checks as C
from tests.block_checks import E32, U, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- AdamW
@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (1e-5, 0.01), (1e-4, 0.1)])
@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_adamw_small_decay(lr, wd, bits, master):
    """A decay of 2e-8 to 1e-5 of a weight beside an update of some lr: each weight is off by its one rounding alone, and
    what they move by on average is not off at all."""
    n = 1 << 20
    c = C.adamw_case([n], "bf16" if master else "f32", "f32", master, bits, seed=21, lr=lr, wd=wd)
    w = 0.5 + 1.5 * torch.rand(n, generator=torch.Generator().manual_seed(23)).cuda()
    if master:
        c["master"][0].copy_(w)
        c["p"][0].copy_(w)
    else:
        c["p"][0].copy_(w)
    before = C.adamw_before(c)
    C.run_adamw(c)
    p, g, m, v = before[0]
    lr32, wd32 = float(np.float32(lr)), float(np.float32(wd))
    want = C.O.adamw(p, g, m, v, lr32, 0.9, 0.99, float(np.float32(1e-8)), 7, wd32, 1.0)[0]
    # the update's own roundings, as in check_adamw, and those of the decay: all relative to a part of the change
    mm = (0.9 * np.abs(m) + 0.1 * np.abs(g)) / (1 - 0.9 ** 7)
    den = np.sqrt((0.99 * v + 0.01 * g * g) / (1 - 0.99 ** 7)) + 1e-8
    part = 72 * E32 * lr * mm / den + 8 * E32 * lr * wd * np.abs(p)
    ulp = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64)
    ulp = np.maximum(ulp, np.spacing(np.abs(p).astype(np.float32)))  # at a power of two
    err = f64(c["p"][0] if not master else c["master"][0]) - want
    assert (np.abs(err) <= 0.5 * ulp + part).all()
    # 2^20 roundings of at most half a step h either way: their mean passes 0.0053 h with a chance of
    # 2 e^{-2^20 0.0053^2 / 2} = 8e-7 (Hoeffding's bound). The smallest decay is a sixth of a step and more.
    assert abs(err.mean()) <= 0.5 * ulp.max() * 0.0053 + part.mean()


# ---------------------------------------------------------------- cross entropy
@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e7, 1e9])
def test_xent_large_logits_of_one_sign(M, size):
    """Logits of -1e3 to -1e9, and targets that are the largest of their row: losses are finite and not below zero, and
    within what the logits are off."""
    H, V = 2048, 900
    r = C.rand(M)
    x, w = r(M, H).abs(), -(1 + 0.2 * r(V, H)).abs()
    s = (size / (0.8 * H)) ** 0.5
    x, w = (x * s).bfloat16(), (w * s).bfloat16()
    for sign in (1, -1):
        l = sign * (x.double() @ w.double().t())
        c = dict(M=M, H=H, V=V, dtype="bf16", tied=True, z=0.0, x=x, w=sign * w, target=l.argmax(1).int(), dloss=r(M))
        out = C.run_xent_fwd(c)
        assert torch.isfinite(out[0]).all() and float(out[0].min()) >= 0.0
        C.check_xent_fwd(c, out)
        if size <= 1e7:  # where a float still has the logits' units
            for t in C.run_xent_bwd(c, out[1], c["dloss"]):
                assert torch.isfinite(t).all()
