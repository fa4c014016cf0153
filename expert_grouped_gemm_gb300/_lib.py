"""ctypes binding of libmoe_gb300.so: the C ABI of include/moe.h, same names.

Argument marshalling only: each function checks that tensors are contiguous,
on the current device and of the expected dtype, passes their pointers and the current
CUDA stream, and raises MoeError on a non-OK status. Every step of the layer
runs in the library's kernels. The operators around the experts, whose
calls can be as short as a launch, do the same in one step of _bind
(csrc/bind.cpp). There is no fallback: if the library is missing or fails to
load, every call raises, and if _bind is, those operators' calls do.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_STATE = -5
MOE_ERR_TIMEOUT = -6
MOE_ERR_DEVICE_ARG = -7
MOE_BF16 = 0
MOE_F32 = 1
MOE_FROZEN = 1
MOE_RECOMPUTE = 2
MOE_NORM_KINDS = {"layer": 0, "rms": 1}
MOE_SCORES = {"softmax": 0, "sigmoid": 1}
MOE_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

EXPORTED = ["moe_workspace_size", "moe_fwd", "moe_select_retained", "moe_bwd", "moe_read_status",
            "moe_last_error", "moe_workspace_entry", "moe_kernel_launches", "moe_timing_enable",
            "moe_timing_read", "moe_route_noalloc", "moe_plan_quota", "moe_selftest_wait", "moe_fwd_decode",
            "moe_selftest_decode_wait", "moe_norm_workspace_size", "moe_norm_fwd", "moe_norm_bwd", "moe_gate_fwd",
            "moe_gate_bwd", "moe_linear_workspace_size", "moe_linear_fwd", "moe_linear_bwd",
            "moe_fwd_routed", "moe_bwd_routed", "moe_balance_workspace_size", "moe_balance_fwd", "moe_balance_bwd",
            "moe_xent_workspace_size", "moe_xent_fwd", "moe_xent_bwd", "moe_grad_norm_workspace_size", "moe_grad_norm",
            "moe_adamw_step"]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moe status {code}: {msg}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("F", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("F_shared", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class NormDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class GateDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64), ("n_group", ctypes.c_int64),
                ("topk_group", ctypes.c_int64), ("group_take", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class LinearDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("out_f32", ctypes.c_int32)]


class BalanceDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64), ("S", ctypes.c_int64),
                ("score", ctypes.c_int32), ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("z_coef", ctypes.c_float)]


class XentDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("H", ctypes.c_int64), ("V", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("tied", ctypes.c_int32), ("z_coef", ctypes.c_float)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class AdamWDims(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("step", ctypes.c_int64), ("lr", ctypes.c_float),
                ("eps", ctypes.c_float), ("grad_scale", ctypes.c_float), ("max_norm", ctypes.c_float),
                ("state_bits", ctypes.c_int32)]


_lib = None
_bind = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library once (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} not found: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    vp, i32p, f32p, i64 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64
    D = ctypes.POINTER(Dims)
    lib.moe_workspace_size.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_fwd.argtypes = [D, vp, ctypes.c_size_t, vp] + [vp] * 10 + [i32p, f32p, i32p, i32p, f32p]
    lib.moe_fwd_decode.argtypes = [D, vp, ctypes.c_size_t, vp] + [vp] * 10 + [i32p, f32p, f32p]
    lib.moe_selftest_decode_wait.argtypes = [D, vp, ctypes.c_size_t, vp] + [vp] * 10 + [ctypes.c_int, ctypes.c_int64]
    lib.moe_select_retained.argtypes = [D, vp, ctypes.c_size_t, vp, vp, i32p, i32p, i32p, f32p]
    lib.moe_bwd.argtypes = [D, vp, ctypes.c_size_t, vp, vp, vp, ctypes.c_int] + [vp] * 8
    lib.moe_read_status.argtypes = [vp, vp]
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_workspace_entry.argtypes = [D, ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                        ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_route_noalloc.argtypes = [D, vp, vp, vp, vp, i32p, f32p, i32p, i32p, i32p]
    lib.moe_route_noalloc.restype = ctypes.c_int
    lib.moe_plan_quota.argtypes = [D, vp, ctypes.c_size_t, vp, ctypes.c_int64, ctypes.c_int64, i32p, i32p]
    lib.moe_plan_quota.restype = ctypes.c_int
    lib.moe_selftest_wait.argtypes = [vp, ctypes.c_int, ctypes.c_int64, i32p]
    lib.moe_selftest_wait.restype = ctypes.c_int
    lib.moe_kernel_launches.argtypes = []
    lib.moe_kernel_launches.restype = ctypes.c_int64
    lib.moe_timing_enable.argtypes = [ctypes.c_int]
    lib.moe_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
    ND, GD, LD = ctypes.POINTER(NormDims), ctypes.POINTER(GateDims), ctypes.POINTER(LinearDims)
    sz = ctypes.c_size_t
    lib.moe_norm_workspace_size.argtypes = [ND, ctypes.POINTER(sz)]
    lib.moe_norm_fwd.argtypes = [ND] + [vp] * 9
    lib.moe_norm_bwd.argtypes = [ND, vp, sz] + [vp] * 10
    lib.moe_gate_fwd.argtypes = [GD] + [vp] * 6
    lib.moe_gate_bwd.argtypes = [GD] + [vp] * 5
    lib.moe_linear_workspace_size.argtypes = [LD, ctypes.POINTER(sz)]
    lib.moe_linear_fwd.argtypes = [LD, vp, sz] + [vp] * 7
    lib.moe_linear_bwd.argtypes = [LD, vp, sz] + [vp] * 9
    lib.moe_fwd_routed.argtypes = [D, vp, sz] + [vp] * 13
    lib.moe_bwd_routed.argtypes = [D, vp, sz] + [vp] * 3 + [ctypes.c_int] + [vp] * 8
    BD, XD, AD, AT = (ctypes.POINTER(t) for t in (BalanceDims, XentDims, AdamWDims, AdamWTensor))
    lib.moe_balance_workspace_size.argtypes = [BD, ctypes.POINTER(sz)]
    lib.moe_balance_fwd.argtypes = [BD, vp, sz] + [vp] * 7
    lib.moe_balance_bwd.argtypes = [BD] + [vp] * 7
    lib.moe_xent_workspace_size.argtypes = [XD, ctypes.c_int, ctypes.POINTER(sz)]
    lib.moe_xent_fwd.argtypes = [XD, vp, sz] + [vp] * 7
    lib.moe_xent_bwd.argtypes = [XD, vp, sz] + [vp] * 9
    lib.moe_grad_norm_workspace_size.argtypes = [AT, i64, ctypes.POINTER(sz)]
    lib.moe_grad_norm.argtypes = [AT, i64, vp, sz, vp, ctypes.c_float, vp]
    lib.moe_adamw_step.argtypes = [AD, AT, i64, vp, vp, vp, vp]
    for name in ["moe_balance_workspace_size", "moe_balance_fwd", "moe_balance_bwd", "moe_xent_workspace_size",
                 "moe_xent_fwd", "moe_xent_bwd", "moe_grad_norm_workspace_size", "moe_grad_norm", "moe_adamw_step"]:
        getattr(lib, name).restype = ctypes.c_int
    for name in ["moe_norm_workspace_size", "moe_norm_fwd", "moe_norm_bwd", "moe_gate_fwd", "moe_gate_bwd",
                 "moe_linear_workspace_size", "moe_linear_fwd", "moe_linear_bwd", "moe_fwd_routed", "moe_bwd_routed"]:
        getattr(lib, name).restype = ctypes.c_int
    for name in ["moe_workspace_size", "moe_fwd", "moe_fwd_decode", "moe_selftest_decode_wait", "moe_select_retained",
                 "moe_bwd", "moe_read_status",
                 "moe_workspace_entry", "moe_timing_enable", "moe_timing_read"]:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _fast():
    """The module that checks the tensors and calls the library in one step, for the operators around the experts."""
    global _bind
    if _bind is None:
        lib = load()
        try:
            from . import _bind as bind
        except ImportError as e:
            raise RuntimeError("_bind.so not found or built for another PyTorch: build it first (python -c "
                               "'import __graft_entry__ as g; g.build()')") from e
        from .build import bind_target
        built_for = getattr(bind, "built_for", "another PyTorch")
        if built_for != bind_target():
            raise RuntimeError(f"_bind.so was built for {built_for}, this is {bind_target()}: build it again "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        bind.init(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
            "moe_norm_fwd", "moe_norm_bwd", "moe_gate_fwd", "moe_gate_bwd", "moe_linear_fwd", "moe_linear_bwd",
            "moe_balance_fwd", "moe_balance_bwd", "moe_xent_fwd", "moe_xent_bwd", "moe_grad_norm", "moe_adamw_step")))
        _bind = bind
    return _bind


def _check(rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, load().moe_last_error().decode(errors="replace"))


def make_dims(T, H, F, E, k, F_shared=0, dtype="bf16", frozen=False, recompute=False) -> Dims:
    return Dims(T, H, F, E, k, F_shared, MOE_BF16 if dtype in ("bf16", MOE_BF16) else MOE_F32,
                (MOE_FROZEN if frozen else 0) | (MOE_RECOMPUTE if recompute else 0))


def _io_dtype(d: Dims):
    return torch.bfloat16 if d.dtype == MOE_BF16 else torch.float32


def _ptr(t, name, dtype=None, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle as a number, without a Stream object made for every call (3 us on a Grace
# core against 0.2); PyTorch versions without the functions take the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


_device = _raw_device or torch.cuda.current_device  # asked only once a CUDA tensor is at hand


def _here(t, name):
    """The library launches on the current device: a tensor of another one is refused."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{_device()}")


def _ws(ws):
    """The workspace's pointer. It stands for its call's device: the experts' calls pass up to twenty tensors, and a look
    at each one's device was 4 us of host time beside 30."""
    p = _ptr(ws, "ws", torch.uint8)
    if ws.get_device() != _device():
        _here(ws, "ws")
    return p


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def moe_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_workspace_size(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def alloc_workspace(dims: Dims, device="cuda") -> torch.Tensor:
    """A uint8 device tensor of moe_workspace_size bytes (torch allocations are 256-byte aligned)."""
    return torch.empty(moe_workspace_size(dims), dtype=torch.uint8, device=device)


def moe_fwd(dims: Dims, ws: torch.Tensor, x, w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down,
            y, topk_idx=None, topk_w=None, expert_offsets=None, row_of_pair=None, logits=None, stream=None):
    io = _io_dtype(dims)
    rc = load().moe_fwd(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream),
        _ptr(x, "x", io), _ptr(w_router, "w_router", io), _ptr(router_bias, "router_bias", torch.float32, False),
        _ptr(w_gate, "w_gate", io), _ptr(w_up, "w_up", io), _ptr(w_down, "w_down", io),
        _ptr(ws_gate, "ws_gate", io, False), _ptr(ws_up, "ws_up", io, False), _ptr(ws_down, "ws_down", io, False),
        _ptr(y, "y", io),
        _ptr(topk_idx, "topk_idx", torch.int32, False), _ptr(topk_w, "topk_w", torch.float32, False),
        _ptr(expert_offsets, "expert_offsets", torch.int32, False),
        _ptr(row_of_pair, "row_of_pair", torch.int32, False), _ptr(logits, "logits", torch.float32, False))
    _check(rc)


def moe_fwd_decode(dims: Dims, ws: torch.Tensor, x, w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                   ws_down, y, topk_idx=None, topk_w=None, logits=None, stream=None):
    """Fused inference forward for 1 <= T <= 16 tokens (bf16); keeps nothing for a backward."""
    io = _io_dtype(dims)
    rc = load().moe_fwd_decode(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream),
        _ptr(x, "x", io), _ptr(w_router, "w_router", io), _ptr(router_bias, "router_bias", torch.float32, False),
        _ptr(w_gate, "w_gate", io), _ptr(w_up, "w_up", io), _ptr(w_down, "w_down", io),
        _ptr(ws_gate, "ws_gate", io, False), _ptr(ws_up, "ws_up", io, False), _ptr(ws_down, "ws_down", io, False),
        _ptr(y, "y", io), _ptr(topk_idx, "topk_idx", torch.int32, False), _ptr(topk_w, "topk_w", torch.float32, False),
        _ptr(logits, "logits", torch.float32, False))
    _check(rc)


def moe_selftest_decode_wait(dims: Dims, ws: torch.Tensor, x, w_router, router_bias, w_gate, w_up, w_down, ws_gate,
                             ws_up, ws_down, y, barrier: int, limit_us: int, stream=None):
    """moe_fwd_decode with grid barrier `barrier` (1..4) unreachable and every wait bounded
    by limit_us: the workspace status word becomes MOE_ERR_TIMEOUT."""
    io = _io_dtype(dims)
    rc = load().moe_selftest_decode_wait(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream),
        _ptr(x, "x", io), _ptr(w_router, "w_router", io), _ptr(router_bias, "router_bias", torch.float32, False),
        _ptr(w_gate, "w_gate", io), _ptr(w_up, "w_up", io), _ptr(w_down, "w_down", io),
        _ptr(ws_gate, "ws_gate", io, False), _ptr(ws_up, "ws_up", io, False), _ptr(ws_down, "ws_down", io, False),
        _ptr(y, "y", io), int(barrier), int(limit_us))
    _check(rc)


def moe_select_retained(dims: Dims, ws: torch.Tensor, dy, quota=None, retained_offsets=None, retained_rows=None,
                        scores=None, stream=None):
    io = _io_dtype(dims)
    rc = load().moe_select_retained(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream), _ptr(dy, "dy", io),
        _ptr(quota, "quota", torch.int32, False), _ptr(retained_offsets, "retained_offsets", torch.int32, False),
        _ptr(retained_rows, "retained_rows", torch.int32, False), _ptr(scores, "scores", torch.float32, False))
    _check(rc)


def moe_bwd(dims: Dims, ws: torch.Tensor, dy, x, use_retained, dx, dw_router=None, dw_gate=None, dw_up=None,
            dw_down=None, dws_gate=None, dws_up=None, dws_down=None, stream=None):
    io = _io_dtype(dims)
    rc = load().moe_bwd(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream), _ptr(dy, "dy", io),
        _ptr(x, "x", io), 1 if use_retained else 0, _ptr(dx, "dx", io),
        _ptr(dw_router, "dw_router", io, False), _ptr(dw_gate, "dw_gate", io, False), _ptr(dw_up, "dw_up", io, False),
        _ptr(dw_down, "dw_down", io, False), _ptr(dws_gate, "dws_gate", io, False),
        _ptr(dws_up, "dws_up", io, False), _ptr(dws_down, "dws_down", io, False))
    _check(rc)


def moe_fwd_routed(dims: Dims, ws: torch.Tensor, x, topk_idx, topk_w, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                   expert_offsets=None, row_of_pair=None, stream=None):
    """moe_fwd with the caller's experts and weights of every token in place of the router."""
    io = _io_dtype(dims)
    rc = load().moe_fwd_routed(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream), _ptr(x, "x", io),
        _ptr(topk_idx, "topk_idx", torch.int32), _ptr(topk_w, "topk_w", torch.float32),
        _ptr(w_gate, "w_gate", io), _ptr(w_up, "w_up", io), _ptr(w_down, "w_down", io),
        _ptr(ws_gate, "ws_gate", io, False), _ptr(ws_up, "ws_up", io, False), _ptr(ws_down, "ws_down", io, False),
        _ptr(y, "y", io), _ptr(expert_offsets, "expert_offsets", torch.int32, False),
        _ptr(row_of_pair, "row_of_pair", torch.int32, False))
    _check(rc)


def moe_bwd_routed(dims: Dims, ws: torch.Tensor, dy, x, use_retained, dx, dtopk_w, dw_gate=None, dw_up=None, dw_down=None,
                   dws_gate=None, dws_up=None, dws_down=None, stream=None):
    """moe_bwd after moe_fwd_routed: dtopk_w receives the gradient of the routing weights."""
    io = _io_dtype(dims)
    rc = load().moe_bwd_routed(
        ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream), _ptr(dy, "dy", io),
        _ptr(x, "x", io), 1 if use_retained else 0, _ptr(dx, "dx", io), _ptr(dtopk_w, "dtopk_w", torch.float32),
        _ptr(dw_gate, "dw_gate", io, False), _ptr(dw_up, "dw_up", io, False), _ptr(dw_down, "dw_down", io, False),
        _ptr(dws_gate, "dws_gate", io, False), _ptr(dws_up, "dws_up", io, False),
        _ptr(dws_down, "dws_down", io, False))
    _check(rc)


def moe_route_noalloc(dims: Dims, x, w_router, router_bias, topk_idx, topk_w, expert_offsets, row_of_pair,
                      device_status=None, stream=None):
    """Routing stage of moe_fwd with no allocation and no workspace (fixed device scratch inside the library)."""
    io = _io_dtype(dims)
    rc = load().moe_route_noalloc(
        ctypes.byref(dims), _stream(stream), _ptr(x, "x", io), _ptr(w_router, "w_router", io),
        _ptr(router_bias, "router_bias", torch.float32, False), _ptr(topk_idx, "topk_idx", torch.int32),
        _ptr(topk_w, "topk_w", torch.float32), _ptr(expert_offsets, "expert_offsets", torch.int32),
        _ptr(row_of_pair, "row_of_pair", torch.int32), _ptr(device_status, "device_status", torch.int32, False))
    _check(rc)


def moe_plan_quota(dims: Dims, ws: torch.Tensor, rho_num: int, rho_den: int, quota, budget=None, stream=None):
    """Device-side retention quotas from the last forward's per-expert counts."""
    rc = load().moe_plan_quota(ctypes.byref(dims), _ws(ws), ws.numel(), _stream(stream),
                               int(rho_num), int(rho_den), _ptr(budget, "budget", torch.int32, False),
                               _ptr(quota, "quota", torch.int32))
    _check(rc)


def moe_selftest_wait(arrive: bool, limit_us: int, device_status, stream=None):
    """One bounded barrier wait on the GPU; device_status receives MOE_OK or MOE_ERR_TIMEOUT."""
    rc = load().moe_selftest_wait(_stream(stream), 1 if arrive else 0, int(limit_us),
                                  _ptr(device_status, "device_status", torch.int32))
    _check(rc)


# ---------------------------------------------------------------- around the experts
def _dt(dtype) -> int:
    if dtype not in ("bf16", "f32"):
        raise ValueError(f"dtype must be 'bf16' or 'f32', got {dtype!r}")
    return MOE_BF16 if dtype == "bf16" else MOE_F32


def _named(table: dict, value, what: str) -> int:
    if value not in table:
        raise ValueError(f"{what} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _tensor(t, name, dtype, shape, required=True):
    """The pointer of a contiguous CUDA tensor of this dtype and shape (None stays None when not required)."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    try:
        if t.is_cuda and t.get_device() == _device() and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    _here(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def make_norm_dims(T, H, dtype="bf16", kind="layer", eps=1e-5) -> NormDims:
    return NormDims(T, H, _dt(dtype), _named(MOE_NORM_KINDS, kind, "kind"), eps)


def alloc_norm_workspace(dims: NormDims, device="cuda") -> torch.Tensor:
    n = ctypes.c_size_t(0)
    _check(load().moe_norm_workspace_size(ctypes.byref(dims), ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def moe_norm_fwd(dims: NormDims, x, residual, weight, bias, y, sum=None, mean=None, rstd=None, stream=None):
    """y = norm(x + residual) * weight + bias; sum receives x + residual, mean and rstd the statistics."""
    rc = _fast().norm_fwd(dims, stream if stream is None else _stream(stream), x, residual, weight, bias, y, sum, mean,
                          rstd)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    io, f32 = _io_dtype(dims), torch.float32
    T, H = dims.T, dims.H
    th, h, t = (T, H), (H,), (T,)
    args = (
        _tensor(x, "x", io, th), _tensor(residual, "residual", io, th, False),
        _tensor(weight, "weight", io, h), _tensor(bias, "bias", io, h, False), _tensor(y, "y", io, th),
        _tensor(sum, "sum", io, th, False), _tensor(mean, "mean", f32, t, False), _tensor(rstd, "rstd", f32, t, False))
    _check(load().moe_norm_fwd(dims, _stream(stream), *args))


def moe_norm_bwd(dims: NormDims, ws, dy, dsum, x, weight, mean, rstd, dx, dweight, dbias=None, stream=None):
    """Gradients of moe_norm_fwd; x is the tensor that was normalised, dsum what reaches it past the norm."""
    rc = _fast().norm_bwd(dims, stream if stream is None else _stream(stream), ws, dy, dsum, x, weight, mean, rstd, dx,
                          dweight, dbias)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    io, f32 = _io_dtype(dims), torch.float32
    T, H = dims.T, dims.H
    th, h, t = (T, H), (H,), (T,)
    _check(load().moe_norm_bwd(
        dims, _ws(ws), ws.numel(), _stream(stream), _tensor(dy, "dy", io, th),
        _tensor(dsum, "dsum", io, th, False), _tensor(x, "x", io, th), _tensor(weight, "weight", io, h),
        _tensor(mean, "mean", f32, t, False), _tensor(rstd, "rstd", f32, t), _tensor(dx, "dx", io, th),
        _tensor(dweight, "dweight", io, h), _tensor(dbias, "dbias", io, h, False)))


def make_gate_dims(T, E, k, score="softmax", renorm=True, scale=1.0, n_group=1, topk_group=1, group_take=1,
                   dtype="f32", grad_dtype="f32") -> GateDims:
    return GateDims(T, E, k, n_group, topk_group, group_take, _named(MOE_SCORES, score, "score"), 1 if renorm else 0,
                    _dt(dtype), _dt(grad_dtype), scale)


def moe_gate_fwd(dims: GateDims, logits, bias, topk_idx, topk_w, expert_count=None, stream=None):
    """Experts and weights of every token from its router logits; bias takes part in the selection only."""
    rc = _fast().gate_fwd(dims, stream if stream is None else _stream(stream), logits, bias, topk_idx, topk_w,
                          expert_count)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    tk = (dims.T, dims.k)
    args = (
        _tensor(logits, "logits", _io_dtype(dims), (dims.T, dims.E)),
        _tensor(bias, "bias", torch.float32, (dims.E,), False), _tensor(topk_idx, "topk_idx", torch.int32, tk),
        _tensor(topk_w, "topk_w", torch.float32, tk),
        _tensor(expert_count, "expert_count", torch.int32, (dims.E,), False))
    _check(load().moe_gate_fwd(dims, _stream(stream), *args))


def moe_gate_bwd(dims: GateDims, logits, topk_idx, dtopk_w, dlogits, stream=None):
    """Gradient of the weights of moe_gate_fwd to the logits, the selection held fixed."""
    rc = _fast().gate_bwd(dims, stream if stream is None else _stream(stream), logits, topk_idx, dtopk_w, dlogits)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    tk, te = (dims.T, dims.k), (dims.T, dims.E)
    grad = torch.bfloat16 if dims.grad_dtype == MOE_BF16 else torch.float32
    args = (
        _tensor(logits, "logits", _io_dtype(dims), te),
        _tensor(topk_idx, "topk_idx", torch.int32, tk), _tensor(dtopk_w, "dtopk_w", torch.float32, tk),
        _tensor(dlogits, "dlogits", grad, te))
    _check(load().moe_gate_bwd(dims, _stream(stream), *args))


def make_linear_dims(M, K, N, dtype="bf16", act="none", out_f32=False) -> LinearDims:
    return LinearDims(M, K, N, _dt(dtype), _named(MOE_ACTS, act, "act"), 1 if out_f32 else 0)


def alloc_linear_workspace(dims: LinearDims, device="cuda") -> torch.Tensor:
    """A workspace of moe_linear_workspace_size bytes, its first 4096 bytes zero as the library wants them.

    They are zero on return (it waits for the current stream), so that the first call may run on any stream. In a
    graph that is being captured the zeroing is a part of the graph instead, ordered as the capture orders it."""
    n = ctypes.c_size_t(0)
    _check(load().moe_linear_workspace_size(ctypes.byref(dims), ctypes.byref(n)))
    return _workspace(n.value, 4096, device)


def _workspace(size: int, header: int, device) -> torch.Tensor:
    """A workspace whose first `header` bytes are zero on return, as alloc_linear_workspace says."""
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    ws[:header].zero_()
    if ws.is_cuda and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(ws.device).synchronize()
    return ws


def moe_linear_fwd(dims: LinearDims, ws, x, w, bias, residual, y, pre=None, stream=None):
    """y = act(x w + bias) + residual; pre receives x w + bias."""
    rc = _fast().linear_fwd(dims, stream if stream is None else _stream(stream), ws, x, w, bias, residual, y, pre)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    io = _io_dtype(dims)
    M, K, N = dims.M, dims.K, dims.N
    mn = (M, N)
    _check(load().moe_linear_fwd(
        dims, _ws(ws), ws.numel(), _stream(stream), _tensor(x, "x", io, (M, K)),
        _tensor(w, "w", io, (K, N)), _tensor(bias, "bias", io, (N,), False),
        _tensor(residual, "residual", io, mn, False), _tensor(y, "y", torch.float32 if dims.out_f32 else io, mn),
        _tensor(pre, "pre", io, mn, False)))


def moe_linear_bwd(dims: LinearDims, ws, dy, x, w, pre, dx=None, dw=None, dbias=None, dx_add=None, stream=None):
    """Gradients of moe_linear_fwd; pre is needed when the activation is not 'none'. dx_add is added to dx."""
    rc = _fast().linear_bwd(dims, stream if stream is None else _stream(stream), ws, dy, x, w, pre, dx_add, dx, dw,
                            dbias)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    io = _io_dtype(dims)
    M, K, N = dims.M, dims.K, dims.N
    mn, mk, kn = (M, N), (M, K), (K, N)
    _check(load().moe_linear_bwd(
        dims, _ws(ws), ws.numel(), _stream(stream), _tensor(dy, "dy", io, mn),
        _tensor(x, "x", io, mk), _tensor(w, "w", io, kn), _tensor(pre, "pre", io, mn, False),
        _tensor(dx_add, "dx_add", io, mk, False), _tensor(dx, "dx", io, mk, False), _tensor(dw, "dw", io, kn, False),
        _tensor(dbias, "dbias", io, (N,), False)))


def make_balance_dims(T, E, k, S=0, score="softmax", alpha=0.01, z_coef=0.0, dtype="f32", grad_dtype="f32") -> BalanceDims:
    """S: sequences of the call (their offsets are given on the device); 0: all tokens are one."""
    return BalanceDims(T, E, k, S, _named(MOE_SCORES, score, "score"), _dt(dtype), _dt(grad_dtype), alpha, z_coef)


def alloc_balance_workspace(dims: BalanceDims, device="cuda") -> torch.Tensor:
    """A workspace of moe_balance_fwd, its header zero on return (as alloc_linear_workspace's)."""
    n = ctypes.c_size_t(0)
    _check(load().moe_balance_workspace_size(ctypes.byref(dims), ctypes.byref(n)))
    return _workspace(n.value, 256, device)


def _seq(dims: BalanceDims, t):
    if t is not None and not dims.S:
        raise ValueError("seq_start given for dims without sequences (S is 0)")
    return _tensor(t, "seq_start", torch.int32, (dims.S + 1,), dims.S > 0)


def moe_balance_fwd(dims: BalanceDims, ws, logits, topk_idx, seq_start, loss, count, prob=None, stream=None):
    """loss[2]: balance loss and z loss of router logits; count and prob [max(S, 1), E]: choices and mean probabilities."""
    rc = _fast().balance_fwd(dims, stream if stream is None else _stream(stream), ws, logits, topk_idx, seq_start, loss,
                             count, prob)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    se, f32 = (max(dims.S, 1), dims.E), torch.float32
    _check(load().moe_balance_fwd(
        dims, _ws(ws), ws.numel(), _stream(stream), _tensor(logits, "logits", _io_dtype(dims), (dims.T, dims.E)),
        _tensor(topk_idx, "topk_idx", torch.int32, (dims.T, dims.k)), _seq(dims, seq_start),
        _tensor(loss, "loss", f32, (2,)), _tensor(count, "count", torch.int32, se), _tensor(prob, "prob", f32, se, False)))


def moe_balance_bwd(dims: BalanceDims, logits, count, seq_start, dloss, dlogits_add, dlogits, stream=None):
    """Gradient of the sum of moe_balance_fwd's losses to the logits, times dloss[1] (None: 1), plus dlogits_add."""
    rc = _fast().balance_bwd(dims, stream if stream is None else _stream(stream), logits, count, seq_start, dloss,
                             dlogits_add, dlogits)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    te, grad = (dims.T, dims.E), torch.bfloat16 if dims.grad_dtype == MOE_BF16 else torch.float32
    args = (
        _tensor(logits, "logits", _io_dtype(dims), te),
        _tensor(count, "count", torch.int32, (max(dims.S, 1), dims.E)), _seq(dims, seq_start),
        _tensor(dloss, "dloss", torch.float32, (1,), False), _tensor(dlogits_add, "dlogits_add", grad, te, False),
        _tensor(dlogits, "dlogits", grad, te))
    _check(load().moe_balance_bwd(dims, _stream(stream), *args))


def make_xent_dims(M, H, V, dtype="bf16", tied=False, z_coef=0.0) -> XentDims:
    """tied: w is an embedding table [V, H] in place of [H, V]."""
    return XentDims(M, H, V, _dt(dtype), 1 if tied else 0, z_coef)


def alloc_xent_workspace(dims: XentDims, device="cuda", backward=True) -> torch.Tensor:
    """A workspace of moe_xent_fwd, and of moe_xent_bwd unless backward is False; its header is zero on return."""
    n = ctypes.c_size_t(0)
    _check(load().moe_xent_workspace_size(ctypes.byref(dims), 1 if backward else 0, ctypes.byref(n)))
    return _workspace(n.value, 256, device)


def _xent_inputs(dims: XentDims, x, w, target):
    io = _io_dtype(dims)
    return (_tensor(x, "x", io, (dims.M, dims.H)),
            _tensor(w, "w", io, (dims.V, dims.H) if dims.tied else (dims.H, dims.V)),
            _tensor(target, "target", torch.int32, (dims.M,)))


def moe_xent_fwd(dims: XentDims, ws, x, w, target, loss, lse, total=None, stream=None):
    """Cross entropy of the logits x w: loss[M], lse[M], and total[2] = (sum of the losses, rows counted)."""
    rc = _fast().xent_fwd(dims, stream if stream is None else _stream(stream), ws, x, w, target, loss, lse, total)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    f32, m = torch.float32, (dims.M,)
    _check(load().moe_xent_fwd(
        dims, _ws(ws), ws.numel(), _stream(stream), *_xent_inputs(dims, x, w, target), _tensor(loss, "loss", f32, m),
        _tensor(lse, "lse", f32, m), _tensor(total, "total", f32, (2,), False)))


def moe_xent_bwd(dims: XentDims, ws, x, w, target, lse, dloss, total, dx=None, dw=None, stream=None):
    """Gradients to x and w for the rows' dloss[M], or of the mean loss (dloss None, the forward's total given)."""
    rc = _fast().xent_bwd(dims, stream if stream is None else _stream(stream), ws, x, w, target, lse, dloss, total, dx, dw)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    f32, m, io = torch.float32, (dims.M,), _io_dtype(dims)
    _check(load().moe_xent_bwd(
        dims, _ws(ws), ws.numel(), _stream(stream), *_xent_inputs(dims, x, w, target), _tensor(lse, "lse", f32, m),
        _tensor(dloss, "dloss", f32, m, False), _tensor(total, "total", f32, (2,), False),
        _tensor(dx, "dx", io, (dims.M, dims.H), False),
        _tensor(dw, "dw", io, (dims.V, dims.H) if dims.tied else (dims.H, dims.V), False)))


# ---------------------------------------------------------------- optimiser
class TensorList:
    """The tensors of an optimiser call as the library reads them; keeps them alive. Made once, used every step."""

    def __init__(self, entries, keep, bits, device):
        self.count, self.bits, self.device, self._keep = len(entries), bits, device, keep
        self.array = (AdamWTensor * max(1, len(entries)))(*entries)
        self.address = ctypes.addressof(self.array)


def _flat(t, name, i, dtypes, n=None):
    """The pointer of a contiguous CUDA tensor of one of these types (any shape, n values)."""
    what = f"{name}[{i}]"
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    _here(t, what)
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{what} must have {n} values, got {t.numel()}")
    return t.data_ptr() or None


_WEIGHT_TYPES = (torch.bfloat16, torch.float32)


def _code(t):
    return MOE_BF16 if t.dtype == torch.bfloat16 else MOE_F32


def make_grad_tensors(grads) -> TensorList:
    """Gradients alone, as moe_grad_norm takes them (a list of make_adamw_tensors serves as well)."""
    grads = list(grads)
    entries = [AdamWTensor(grad=_flat(g, "grads", i, _WEIGHT_TYPES), n=g.numel(), grad_dtype=_code(g))
               for i, g in enumerate(grads)]
    return TensorList(entries, grads, None, grads[0].get_device() if grads else None)


def make_adamw_tensors(params, grads, m, v, master=None, m_scale=None, v_scale=None, weight_decay=0.0,
                       lr_scale=1.0) -> TensorList:
    """The tensors of moe_adamw_step, one list each. m and v: fp32, or torch.float8_e4m3fn with the fp32 scales of their
    blocks of 256 values (v holds square roots then). master: fp32 copies of bf16 weights (None, or a list that may
    hold None). weight_decay and lr_scale: one number, or one for each tensor."""
    params, grads, m, v = list(params), list(grads), list(m), list(v)
    n = len(params)
    each = lambda x, fill: [fill] * n if x is None else list(x) if isinstance(x, (list, tuple)) else [x] * n
    master, m_scale, v_scale = each(master, None), each(m_scale, None), each(v_scale, None)
    decay, lrs = each(weight_decay, 0.0), each(lr_scale, 1.0)
    for name, x in (("grads", grads), ("m", m), ("v", v), ("master", master), ("m_scale", m_scale), ("v_scale", v_scale),
                    ("weight_decay", decay), ("lr_scale", lrs)):
        if len(x) != n:
            raise ValueError(f"{name} must have {n} entries, got {len(x)}")
    bits = 8 if n and isinstance(m[0], torch.Tensor) and m[0].dtype == torch.float8_e4m3fn else 32
    state = (torch.float8_e4m3fn,) if bits == 8 else (torch.float32,)
    entries, written = [], []
    for i in range(n):
        p = _flat(params[i], "params", i, _WEIGHT_TYPES)
        size = params[i].numel()
        scales = [None, None]
        if bits == 8:
            scales = [_flat(t, name, i, (torch.float32,), (size + 255) // 256)
                      for name, t in (("m_scale", m_scale[i]), ("v_scale", v_scale[i]))]
        elif m_scale[i] is not None or v_scale[i] is not None:
            raise ValueError(f"m_scale and v_scale belong to states in 8 bits, m[{i}] is {m[i].dtype}")
        mp = None if master[i] is None else _flat(master[i], "master", i, (torch.float32,), size)
        entries.append(AdamWTensor(p, _flat(grads[i], "grads", i, _WEIGHT_TYPES, size), mp,
                                   _flat(m[i], "m", i, state, size), _flat(v[i], "v", i, state, size), *scales, size,
                                   _code(params[i]), _code(grads[i]), lrs[i], decay[i]))
        written += [t for t in (params[i], m[i], v[i], master[i], m_scale[i], v_scale[i]) if t is not None and t.numel()]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), w)
                   for w, ts in ((1, written), (0, grads)) for t in ts if t.numel())
    last, last_written = 0, 0  # where what came before ends
    for a, b, w in spans:
        if a < (last if w else last_written):
            raise ValueError("weights, states or gradients overlap: every tensor may be listed once")
        last, last_written = max(last, b), max(last_written, b if w else 0)
    return TensorList(entries, (params, grads, m, v, master, m_scale, v_scale), bits,
                      params[0].get_device() if n else None)


def make_adamw_dims(lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_bits=32, max_norm=0.0, grad_scale=1.0) -> AdamWDims:
    return AdamWDims(beta1, beta2, step, lr, eps, grad_scale, max_norm, state_bits)


def _list_here(tensors: TensorList):
    if tensors.device is not None and tensors.device != _device():
        raise ValueError(f"the tensors are on cuda:{tensors.device}, the current device is cuda:{_device()}")


def alloc_grad_norm_workspace(tensors: TensorList, device="cuda") -> torch.Tensor:
    """A workspace of moe_grad_norm for these tensors, its header zero on return."""
    n = ctypes.c_size_t(0)
    _check(load().moe_grad_norm_workspace_size(tensors.array, tensors.count, ctypes.byref(n)))
    return _workspace(n.value, 256, device)


def moe_grad_norm(tensors: TensorList, ws, norm, grad_scale=1.0, stream=None):
    """norm[1] = grad_scale times the 2-norm of all gradients of the list."""
    rc = _fast().grad_norm(grad_scale, stream if stream is None else _stream(stream), ws, tensors.address, tensors.count,
                           tensors.device, norm)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    _list_here(tensors)
    norm = _tensor(norm, "norm", torch.float32, (1,))
    _check(load().moe_grad_norm(tensors.array, tensors.count, _ws(ws), ws.numel(), _stream(stream), grad_scale, norm))


def moe_adamw_step(dims: AdamWDims, tensors: TensorList, norm=None, lr=None, step=None, stream=None):
    """One AdamW step over the list, in place. norm[1]: the gradients' norm (clipping; a step on inf or NaN is left out);
    lr[1] (fp32), step[1] (int32): on the device, in place of dims'."""
    if tensors.bits != dims.state_bits and tensors.count:
        raise ValueError(f"the list's states have {tensors.bits} bits, dims say {dims.state_bits}")
    rc = _fast().adamw_step(dims, stream if stream is None else _stream(stream), tensors.address, tensors.count,
                            tensors.device, norm, lr, step)
    if rc is not None:
        return _check(rc)
    # something is not what the operator takes: the checks one by one, which name it
    _list_here(tensors)
    one = (1,)
    args = (_tensor(norm, "norm", torch.float32, one, False), _tensor(lr, "lr", torch.float32, one, False),
            _tensor(step, "step", torch.int32, one, False))
    _check(load().moe_adamw_step(dims, tensors.array, tensors.count, _stream(stream), *args))


def moe_read_status(ws: torch.Tensor, stream=None) -> int:
    """Device status word (MOE_OK, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_ARG); syncs the stream and clears it."""
    return load().moe_read_status(_ws(ws), _stream(stream))


def moe_workspace_entries(dims: Dims) -> dict:
    """{name: (byte offset, byte size)} of the workspace layout for these dims (diagnostic)."""
    out, i = {}, 0
    lib = load()
    while True:
        name, off, size = ctypes.c_char_p(), ctypes.c_size_t(), ctypes.c_size_t()
        rc = lib.moe_workspace_entry(ctypes.byref(dims), i, ctypes.byref(name), ctypes.byref(off), ctypes.byref(size))
        if rc == MOE_ERR_INVALID_ARG and i > 0:
            return out
        _check(rc)
        out[name.value.decode()] = (off.value, size.value)
        i += 1


def ws_view(ws: torch.Tensor, dims: Dims, name: str, dtype, shape) -> torch.Tensor:
    """A typed view of one workspace buffer (diagnostic; copies nothing)."""
    off, size = moe_workspace_entries(dims)[name]
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.tensor([], dtype=dtype).element_size()
    assert nbytes <= size, (name, nbytes, size)
    return ws[off:off + nbytes].view(dtype).view(*shape)


def moe_kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().moe_kernel_launches())


def moe_timing_enable(on: bool) -> None:
    _check(load().moe_timing_enable(1 if on else 0))


def moe_timing_read():
    """(ms[2], launches[2]) for families (grouped GEMMs, bandwidth kernels); resets the counters."""
    ms = (ctypes.c_double * 2)()
    n = (ctypes.c_int64 * 2)()
    _check(load().moe_timing_read(ms, n))
    return [ms[0], ms[1]], [n[0], n[1]]


def moe_last_error() -> str:
    return load().moe_last_error().decode(errors="replace")
