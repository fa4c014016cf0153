"""MoEBlock: the pre-norm feed-forward half of a transformer layer around the expert block.

    h      = residual + attn w_o + b_o              (moe_linear_fwd)
    n      = norm(h) * norm_w + norm_b              (moe_norm_fwd)
    logits = n w_router                             (moe_linear_fwd, fp32 logits)
    idx, w = gate(logits, balance_bias)             (moe_gate_fwd)
    y      = experts(n; idx, w) + shared(n)         (moe_fwd_routed)

(y, h) go on to the next block, whose norm adds them. Holds the device weights, the workspaces and
the buffers and drives the C ABI; every step runs in the library's kernels. The buffers belong to
the block: a second forward overwrites the first one's outputs.
"""
from __future__ import annotations

import torch

from . import _lib
from .inputs import Workload

WEIGHTS = ["w_o", "b_o", "norm_w", "norm_b", "w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"]


class MoEBlock:
    def __init__(self, w: Workload, params: dict, device="cuda", norm: str = "rms", eps: float = 1e-5,
                 score: str = "softmax", renorm: bool = True, scale: float = 1.0, n_group: int = 1,
                 topk_group: int = 1, group_take: int = 1, recompute: bool = False):
        """params: tensors named as in WEIGHTS (b_o, norm_b and, without a shared expert, ws_* may be missing)
        and the optional fp32 balance_bias[E]. recompute: as in MoELayer."""
        self.w = w
        dev = torch.device(device)
        io = torch.bfloat16 if w.dtype == "bf16" else torch.float32
        T, H, F, E, k, Fs = w.T, w.H, w.F, w.E, w.k, w.F_shared
        self.p = {n: None if params.get(n) is None else params[n].to(dev).contiguous()
                  for n in WEIGHTS + ["balance_bias"]}
        A = self.p["w_o"].shape[0]
        self.proj = _lib.make_linear_dims(T, A, H, w.dtype)
        self.norm = _lib.make_norm_dims(T, H, w.dtype, norm, eps)
        self.router = _lib.make_linear_dims(T, H, E, w.dtype, out_f32=True)
        # dlogits in the io type: the router's products read it as a tensor-core operand
        self.gate = _lib.make_gate_dims(T, E, k, score, renorm, scale, n_group, topk_group, group_take, "f32", w.dtype)
        self.moe = _lib.make_dims(T, H, F, E, k, Fs, w.dtype, w.frozen, recompute)
        self.ws_proj = _lib.alloc_linear_workspace(self.proj, dev)
        self.ws_norm = _lib.alloc_norm_workspace(self.norm, dev)
        self.ws_router = _lib.alloc_linear_workspace(self.router, dev)
        self.ws_moe = _lib.alloc_workspace(self.moe, dev)
        new = lambda *s, dtype=io: torch.empty(*s, dtype=dtype, device=dev)
        f32 = torch.float32
        self.h, self.n, self.y = new(T, H), new(T, H), new(T, H)
        self.mean = new(T, dtype=f32) if norm == "layer" else None
        self.rstd = new(T, dtype=f32)
        self.logits, self.topk_w, self.dtopk_w = new(T, E, dtype=f32), new(T, k, dtype=f32), new(T, k, dtype=f32)
        self.topk_idx, self.expert_count = new(T, k, dtype=torch.int32), new(E, dtype=torch.int32)
        self.dn, self.dh, self.dattn, self.dlogits = new(T, H), new(T, H), new(T, A), new(T, E)
        g = dict(w_o=new(A, H), norm_w=new(H), w_router=new(H, E))
        if self.p["b_o"] is not None:
            g["b_o"] = new(H)
        if self.p["norm_b"] is not None:
            g["norm_b"] = new(H)
        if not w.frozen:
            g.update(w_gate=new(E, H, F), w_up=new(E, H, F), w_down=new(E, F, H))
            if Fs:
                g.update(ws_gate=new(H, Fs), ws_up=new(H, Fs), ws_down=new(Fs, H))
        self.grads = g

    def forward(self, attn: torch.Tensor, residual: torch.Tensor, stream=None):
        """attn[T,A] (the attention's heads side by side) and residual[T,H] -> (y, h)."""
        p = self.p
        _lib.moe_linear_fwd(self.proj, self.ws_proj, attn, p["w_o"], p["b_o"], residual, self.h, stream=stream)
        _lib.moe_norm_fwd(self.norm, self.h, None, p["norm_w"], p["norm_b"], self.n, None, self.mean, self.rstd,
                          stream=stream)
        _lib.moe_linear_fwd(self.router, self.ws_router, self.n, p["w_router"], None, None, self.logits, stream=stream)
        _lib.moe_gate_fwd(self.gate, self.logits, p["balance_bias"], self.topk_idx, self.topk_w, self.expert_count,
                          stream=stream)
        _lib.moe_fwd_routed(self.moe, self.ws_moe, self.n, self.topk_idx, self.topk_w, p["w_gate"], p["w_up"],
                            p["w_down"], p["ws_gate"], p["ws_up"], p["ws_down"], self.y, stream=stream)
        return self.y, self.h

    def select(self, dy: torch.Tensor, quota: torch.Tensor | None, stream=None) -> None:
        """The token-expert pairs of the last forward that backward(use_retained=True) on this dy keeps."""
        _lib.moe_select_retained(self.moe, self.ws_moe, dy, quota, stream=stream)

    def backward(self, attn: torch.Tensor, dy: torch.Tensor, dh: torch.Tensor, stream=None, use_retained: bool = False):
        """Gradients of <dy, y> + <dh, h> for the attn of the last forward: (dattn, dresidual, weight gradients).

        use_retained (after select): the experts' part over the kept pairs only; the routing weights' gradient is
        that of every pair."""
        p, g = self.p, self.grads
        _lib.moe_bwd_routed(self.moe, self.ws_moe, dy, self.n, use_retained, self.dn, self.dtopk_w, g.get("w_gate"),
                            g.get("w_up"), g.get("w_down"), g.get("ws_gate"), g.get("ws_up"), g.get("ws_down"),
                            stream=stream)
        _lib.moe_gate_bwd(self.gate, self.logits, self.topk_idx, self.dtopk_w, self.dlogits, stream=stream)
        # the router's part of dn is added to the experts' in the product's epilogue
        _lib.moe_linear_bwd(self.router, self.ws_router, self.dlogits, self.n, p["w_router"], None, self.dn,
                            g["w_router"], None, dx_add=self.dn, stream=stream)
        _lib.moe_norm_bwd(self.norm, self.ws_norm, self.dn, dh, self.h, p["norm_w"], self.mean, self.rstd, self.dh,
                          g["norm_w"], g.get("norm_b"), stream=stream)
        _lib.moe_linear_bwd(self.proj, self.ws_proj, self.dh, attn, p["w_o"], None, self.dattn, g["w_o"], g.get("b_o"),
                            stream=stream)
        return self.dattn, self.dh, g

    def status(self, stream=None) -> int:
        """The first device status that is not MOE_OK (synchronises the stream and clears them)."""
        codes = [_lib.moe_read_status(ws, stream) for ws in (self.ws_proj, self.ws_router, self.ws_moe)]
        return next((c for c in codes if c != _lib.MOE_OK), _lib.MOE_OK)
