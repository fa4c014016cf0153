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
