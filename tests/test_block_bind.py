"""What the module of csrc/bind.cpp is needed for, and when it counts as built (no GPU)."""
import os
import subprocess
import sys

import pytest

from expert_grouped_gemm_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_the_library_loads_without_the_module():
    """The experts' calls go through ctypes alone; the norm, gate and linear calls say what is missing."""
    code = """
import sys
sys.modules["expert_grouped_gemm_gb300._bind"] = None  # an import of it fails
import torch
from expert_grouped_gemm_gb300 import _lib
assert _lib.moe_workspace_size(_lib.make_dims(128, 256, 128, 16, 4)) > 0
x = torch.zeros(4, 64, dtype=torch.bfloat16)
try:
    _lib.moe_norm_fwd(_lib.make_norm_dims(4, 64), x, None, x[0], None, x)
except RuntimeError as e:
    assert "_bind.so" in str(e)
else:
    raise AssertionError("a call without the module went through")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_module_of_another_pytorch_is_not_current(monkeypatch):
    """It reads PyTorch's structures: after a change of PyTorch it counts as stale, and is not called if it loads."""
    import torch

    from expert_grouped_gemm_gb300 import _lib

    assert build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0+other")
    assert not build.up_to_date()
    monkeypatch.setattr(_lib, "_bind", None)
    with pytest.raises(RuntimeError, match="0.0.other"):
        _lib._fast()


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels run on the current device, with its stream: a tensor that lies on another one is named, in every call."""
    import torch

    from expert_grouped_gemm_gb300 import _lib

    class Other(torch.Tensor):  # a host tensor that says it is on the second GPU
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 1

    monkeypatch.setattr(_lib, "_device", lambda: 0, raising=False)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    bf = torch.bfloat16
    t = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype).as_subclass(Other)
    x, w = t(4, 64), t(64, 64)
    ws = t(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x is on cuda:1, the current device is cuda:0"):
        _lib.moe_norm_fwd(_lib.make_norm_dims(4, 64), x, None, w[0], None, x)
    with pytest.raises(ValueError, match="ws is on cuda:1"):
        _lib.moe_linear_fwd(_lib.make_linear_dims(4, 64, 64), ws, x, w, None, None, x)
    with pytest.raises(ValueError, match="ws is on cuda:1"):
        _lib.moe_fwd_routed(_lib.make_dims(4, 64, 64, 16, 2), ws, x, t(4, 2, dtype=torch.int32),
                            t(4, 2, dtype=torch.float32), w, w, w, None, None, None, x)
