"""The norm, gate and linear operators where fp32 runs out: scores that are denormal numbers, rows whose mean is large
against their spread, the far tails of the activations. Bounds follow from the arithmetic, with no slack that covers the
value itself."""
import numpy as np
import pytest
import torch

from expert_grouped_gemm_gb300 import _lib
from oracle import block_oracle as B
from tests import block_checks as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


# ---------------------------------------------------------------- gate
@pytest.mark.parametrize("k", [1, 2, 8])
def test_gate_gradient_of_denormal_sigmoid_scores(k):
    """Logits of -85 to -88.7: sigmoid scores down to 2^-128, whose reciprocal is past fp32's range. The renormalised
    weights and their gradients are ordinary numbers all the same."""
    T, E = 200, 16
    g = torch.Generator().manual_seed(k)
    logits = (-88.7 + 3.7 * torch.rand(T, E, generator=g)).cuda()
    logits[0, :], logits[1, :] = -88.7, -87.0
    dw = (4 * torch.randn(T, k, generator=g)).cuda()
    idx, w, _ = C.run_gate(logits, None, k, "sigmoid", True, 2.5)
    dl = C.run_gate_bwd(logits, idx, dw, "sigmoid", True, 2.5)
    l, i = C.f64(logits), idx.cpu().numpy().astype(np.int64)
    # a score of 2^-128 or more is a multiple of 2^-149 (2^-22 of it, half of that its rounding) with a few ulp of exp
    # and of a division: 2^-21. w carries it twice and one division; dl = w (dw - sum w dw) (1 - s) carries w's three
    # times, and the sums' roundings.
    e = 2.0 ** -19
    W = B.gate_weights(l, i, "sigmoid", True, 2.5)
    C.close(w, W, e * W, "topk_w")
    want = B.gate_bwd(l, i, C.f64(dw), "sigmoid", True, 2.5)
    mag = 2.5 * np.abs(C.f64(dw)).max(1, keepdims=True)
    dense = np.zeros((T, E))
    np.put_along_axis(dense, i, W / 2.5, 1)
    C.close(dl, want, 4 * e * dense * mag, "dlogits")
