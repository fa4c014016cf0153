"""AdamW: decoupled weight decay over all tensors of a model, one launch a step.

Holds the states (fp32, or e4m3 in blocks of 256 values with a scale each), the fp32 copies of bf16
weights and the tensors' list, and drives moe_grad_norm and moe_adamw_step. Weights and gradients stay
the caller's buffers, the same ones every step: MoEBlock.p and MoEBlock.grads, say.
"""
from __future__ import annotations

import torch

from . import _lib

BLOCK = 256  # values that share a scale of the 8-bit states


class AdamW:
    def __init__(self, params, grads, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay=0.01, lr_scale=1.0, state_bits: int = 32, master: bool = True, max_norm: float = 0.0,
                 grad_scale: float = 1.0, capturable: bool = False):
        """params, grads: lists of tensors, pairwise. master: bf16 weights get an fp32 copy, which the steps change.
        max_norm > 0 (inf too): gradients are clipped to that norm, and a step whose norm is inf or NaN leaves weights and
        states as they are, but is counted. capturable: lr and the step count live on the device (self.lr, self.t), so
        that a captured step moves on."""
        params, grads = list(params), list(grads)
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        if not params:
            raise ValueError("params is empty")
        dev = params[0].device
        dt = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        zeros = lambda n, dtype: torch.zeros(n, dtype=dtype, device=dev)
        state = lambda: [zeros(p.numel(), torch.uint8 if state_bits == 8 else dt).view(dt) for p in params]
        scales = lambda: [zeros(-(-p.numel() // BLOCK), torch.float32) for p in params] if state_bits == 8 else None
        self.params, self.grads = params, grads
        self.m, self.v, self.m_scale, self.v_scale = state(), state(), scales(), scales()
        self.master = [p.float() if master and p.dtype == torch.bfloat16 else None for p in params]
        self.tensors = _lib.make_adamw_tensors(params, grads, self.m, self.v, self.master, self.m_scale, self.v_scale,
                                               weight_decay, lr_scale)
        self.dims = _lib.make_adamw_dims(lr, beta1, beta2, eps, 1, state_bits, max_norm, grad_scale)
        self.norm = zeros(1, torch.float32)
        self.ws = _lib.alloc_grad_norm_workspace(self.tensors, dev) if max_norm > 0 else None
        self.steps = 0
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=dev) if capturable else None
        self.t = zeros(1, torch.int32) if capturable else None

    def step(self, lr: float | None = None) -> None:
        """One step on the gradients as they are, on the current stream. lr: from this step on (not with capturable,
        where the caller writes self.lr)."""
        if lr is not None:
            if self.lr is not None:
                raise ValueError("with capturable the step reads self.lr: write it there")
            self.dims.lr = lr
        if self.ws is not None:
            _lib.moe_grad_norm(self.tensors, self.ws, self.norm, self.dims.grad_scale)
        if self.t is not None:
            self.t.add_(1)
        self.steps += 1
        self.dims.step = self.steps
        _lib.moe_adamw_step(self.dims, self.tensors, None if self.ws is None else self.norm, self.lr, self.t)
