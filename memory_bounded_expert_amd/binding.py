"""Thin Python binding of libmoebound.so (ctypes).

Argument marshalling only: the functions carry the C ABI's names, check that
torch tensors have the shapes, dtypes and devices the C ABI expects, allocate
missing outputs and the workspace with torch, and pass raw device pointers
and the current HIP stream.  Every step of the layer runs in the library's
HIP kernels; there is no fallback.  Loading fails loudly when the library is
not built.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import re
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoebound.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
HEADERS = (os.path.join(INCLUDE, "moebound.h"), os.path.join(INCLUDE, "cce.h"))
# the operators around the layer
OPERATOR_HEADERS = tuple(os.path.join(INCLUDE, n) for n in
                         ("route.h", "lnorm.h", "embed.h", "distill.h"))
# the 8-bit path of an expert layer
EXPERT_HEADERS = tuple(os.path.join(INCLUDE, n) for n in ("rms.h", "q8.h", "gmm.h"))

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, 1, 2, 3, 4
STAGES = {"router": 0, "topk": 1, "plan": 2, "gather": 3, "gemm_up": 4, "gemm_down": 5,
          "combine": 6}
BSTAGES = {"zero": 0, "transpose": 1, "plan": 2, "recompute": 3, "dh": 4, "wgrad_down": 5,
           "wgrad_gate_up": 6, "dx": 7, "combine_bwd": 8, "dwr": 9}
MOE_F32, MOE_BF16 = 0, 1
GMM_BF16, GMM_Q8 = 0, 1
GMM8_CUT = 7.0 / 8192  # of the products' magnitudes: gmm8_forward's sums of more than four rows
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
CCE_STAGES = {"logits": 0, "fold": 1, "grad": 2, "dx": 3, "dw": 4}

_c = ctypes
_vp = _c.c_void_p


class MoePlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64),
        ("H", _c.c_int32), ("F", _c.c_int32), ("E", _c.c_int32), ("k", _c.c_int32),
        ("c", _c.c_int32), ("K_max", _c.c_int32), ("K", _c.c_int32), ("flags", _c.c_int32),
        ("c_eff", _c.c_int64), ("max_pairs_per_chunk", _c.c_int64),
        ("dispatch_bound_bytes", _c.c_int64), ("fwd_workspace_bytes", _c.c_int64),
        ("bwd_workspace_bytes", _c.c_int64), ("debug_workspace_bytes", _c.c_int64),
    ]


class MoeStats(_c.Structure):
    _fields_ = [
        ("K", _c.c_int32), ("launches", _c.c_int32), ("c_eff", _c.c_int64),
        ("max_pairs_per_chunk", _c.c_int64), ("dispatch_bytes", _c.c_int64),
        ("dispatch_bound_bytes", _c.c_int64), ("intermediate_bytes", _c.c_int64),
        ("workspace_bytes", _c.c_int64),
    ]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class CcePlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("V", _c.c_int64),
        ("H", _c.c_int32), ("v_chunk", _c.c_int32), ("S", _c.c_int32), ("reserved0", _c.c_int32),
        ("strip_bound_bytes", _c.c_int64), ("unchunked_logit_bytes", _c.c_int64),
        ("fwd_workspace_bytes", _c.c_int64), ("bwd_workspace_bytes", _c.c_int64),
    ]


class RoutePlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("score", _c.c_int32), ("N", _c.c_int64), ("E", _c.c_int32),
        ("k", _c.c_int32), ("n_group", _c.c_int32), ("topk_group", _c.c_int32),
        ("group_top", _c.c_int32), ("renorm", _c.c_int32), ("scale", _c.c_float),
        ("reserved0", _c.c_int32),
    ]


class LnormPlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("H", _c.c_int32),
        ("eps", _c.c_float), ("bwd_workspace_bytes", _c.c_int64),
    ]


class EmbedPlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("V", _c.c_int64),
        ("H", _c.c_int32), ("scale", _c.c_float), ("bwd_workspace_bytes", _c.c_int64),
    ]


class KdPlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("V", _c.c_int64),
        ("H", _c.c_int32), ("v_chunk", _c.c_int32), ("K", _c.c_int32),
        ("temperature", _c.c_float), ("dw_dtype", _c.c_int32), ("S", _c.c_int32),
        ("strip", _c.c_int32), ("reserved0", _c.c_int32), ("strip_bound_bytes", _c.c_int64), ("fwd_workspace_bytes", _c.c_int64),
        ("bwd_workspace_bytes", _c.c_int64),
    ]


class RmsPlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("H", _c.c_int32),
        ("eps", _c.c_float), ("row_pitch", _c.c_int32), ("scale_pitch", _c.c_int32),
        ("bwd_workspace_bytes", _c.c_int64),
    ]


class Q8Plan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("dtype", _c.c_int32), ("N", _c.c_int64), ("H", _c.c_int32),
        ("row_pitch", _c.c_int32), ("scale_pitch", _c.c_int32), ("reserved0", _c.c_int32),
    ]


class GmmPlan(_c.Structure):
    _fields_ = [
        ("magic", _c.c_uint32), ("operands", _c.c_int32), ("R", _c.c_int64), ("K", _c.c_int32),
        ("N", _c.c_int32), ("E", _c.c_int32), ("row_pitch", _c.c_int32),
        ("fwd_workspace_bytes", _c.c_int64), ("bwd_workspace_bytes", _c.c_int64),
    ]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded after torch, so that it binds to the HIP
    runtime torch already uses)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    L.moe_status_string.restype = _c.c_char_p
    L.moe_status_string.argtypes = [_c.c_int]
    L.moe_plan_chunks.restype = _c.c_int
    L.moe_plan_chunks.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32,
                                  _c.c_int32, _c.c_int32, _c.c_int32, _c.POINTER(MoePlan)]
    L.moe_plan_set_flags.restype = _c.c_int
    L.moe_plan_set_flags.argtypes = [_c.POINTER(MoePlan), _c.c_int32]
    L.moe_bounded_forward.restype = _c.c_int
    L.moe_bounded_forward.argtypes = [_c.POINTER(MoePlan)] + [_vp] * 10 + [_vp, _c.c_size_t, _vp,
                                                                         _c.POINTER(MoeStats)]
    L.moe_bounded_forward_static.restype = _c.c_int
    L.moe_bounded_forward_static.argtypes = [_c.POINTER(MoePlan)] + [_vp] * 10 + [
        _vp, _c.POINTER(MoeStats)]
    L.moe_bounded_backward.restype = _c.c_int
    L.moe_bounded_backward.argtypes = [_c.POINTER(MoePlan)] + [_vp] * 15 + [_vp, _c.c_size_t, _vp,
                                                                          _c.POINTER(MoeStats)]
    L.moe_debug_topk.restype = _c.c_int
    L.moe_debug_topk.argtypes = [_vp, _c.c_int64, _c.c_int32, _c.c_int32, _vp, _vp, _vp]
    L.moe_debug_plan.restype = _c.c_int
    L.moe_debug_plan.argtypes = [_c.POINTER(MoePlan), _vp, _vp, _vp, _vp, _vp, _c.c_size_t, _vp]
    L.moe_debug_stage.restype = _c.c_int
    L.moe_debug_stage.argtypes = [_c.POINTER(MoePlan), _c.c_int32, _c.c_int32] + [_vp] * 9 + [
        _vp, _c.c_size_t, _vp]
    L.moe_debug_stage_bwd.restype = _c.c_int
    L.moe_debug_stage_bwd.argtypes = [_c.POINTER(MoePlan), _c.c_int32, _c.c_int32] + [_vp] * 15 + [
        _vp, _c.c_size_t, _vp]
    L.cce_plan.restype = _c.c_int
    L.cce_plan.argtypes = [_c.c_int64, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                           _c.POINTER(CcePlan)]
    L.cce_forward.restype = _c.c_int
    L.cce_forward.argtypes = [_c.POINTER(CcePlan)] + [_vp] * 5 + [_vp, _c.c_size_t, _vp]
    L.cce_backward.restype = _c.c_int
    L.cce_backward.argtypes = [_c.POINTER(CcePlan)] + [_vp] * 7 + [_vp, _c.c_size_t, _vp]
    L.cce_debug_stage.restype = _c.c_int
    L.cce_debug_stage.argtypes = [_c.POINTER(CcePlan), _c.c_int32, _c.c_int32] + [_vp] * 8 + [
        _vp, _c.c_size_t, _vp]
    L.route_plan.restype = _c.c_int
    L.route_plan.argtypes = [_c.c_int64] + [_c.c_int32] * 7 + [_c.c_float, _c.POINTER(RoutePlan)]
    L.route_forward.restype = _c.c_int
    L.route_forward.argtypes = [_c.POINTER(RoutePlan)] + [_vp] * 5
    L.route_backward.restype = _c.c_int
    L.route_backward.argtypes = [_c.POINTER(RoutePlan)] + [_vp] * 5
    L.moe_routed_forward.restype = _c.c_int
    L.moe_routed_forward.argtypes = [_c.POINTER(MoePlan)] + [_vp] * 8 + [_c.c_size_t, _vp,
                                                                       _c.POINTER(MoeStats)]
    L.moe_routed_backward.restype = _c.c_int
    L.moe_routed_backward.argtypes = [_c.POINTER(MoePlan)] + [_vp] * 13 + [_c.c_size_t, _vp,
                                                                         _c.POINTER(MoeStats)]
    L.lnorm_plan.restype = _c.c_int
    L.lnorm_plan.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.c_float, _c.POINTER(LnormPlan)]
    L.lnorm_forward.restype = _c.c_int
    L.lnorm_forward.argtypes = [_c.POINTER(LnormPlan)] + [_vp] * 7
    L.lnorm_backward.restype = _c.c_int
    L.lnorm_backward.argtypes = [_c.POINTER(LnormPlan)] + [_vp] * 9 + [_c.c_size_t, _vp]
    L.embed_plan.restype = _c.c_int
    L.embed_plan.argtypes = [_c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_float,
                             _c.POINTER(EmbedPlan)]
    L.embed_forward.restype = _c.c_int
    L.embed_forward.argtypes = [_c.POINTER(EmbedPlan)] + [_vp] * 4
    L.embed_backward.restype = _c.c_int
    L.embed_backward.argtypes = [_c.POINTER(EmbedPlan)] + [_vp] * 3 + [_c.c_int32, _vp, _c.c_size_t,
                                                                     _vp]
    L.kd_plan.restype = _c.c_int
    L.kd_plan.argtypes = [_c.c_int64, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_float,
                          _c.c_int32, _c.c_int32, _c.POINTER(KdPlan)]
    L.kd_forward.restype = _c.c_int
    L.kd_forward.argtypes = [_c.POINTER(KdPlan)] + [_vp] * 8 + [_c.c_size_t, _vp]
    L.kd_backward.restype = _c.c_int
    L.kd_backward.argtypes = [_c.POINTER(KdPlan)] + [_vp] * 10 + [_c.c_size_t, _vp]
    L.rms_plan.restype = _c.c_int
    L.rms_plan.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.c_float, _c.POINTER(RmsPlan)]
    L.rms_forward.restype = _c.c_int
    L.rms_forward.argtypes = [_c.POINTER(RmsPlan)] + [_vp] * 7
    L.rms_forward_q8.restype = _c.c_int
    L.rms_forward_q8.argtypes = [_c.POINTER(RmsPlan)] + [_vp] * 8
    L.rms_backward.restype = _c.c_int
    L.rms_backward.argtypes = [_c.POINTER(RmsPlan)] + [_vp] * 8 + [_c.c_size_t, _vp]
    L.q8_plan.restype = _c.c_int
    L.q8_plan.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.POINTER(Q8Plan)]
    L.q8_pack.restype = _c.c_int
    L.q8_pack.argtypes = [_c.POINTER(Q8Plan)] + [_vp] * 4
    L.q8_unpack.restype = _c.c_int
    L.q8_unpack.argtypes = [_c.POINTER(Q8Plan)] + [_vp] * 4
    L.q8_pack_weights.restype = _c.c_int
    L.q8_pack_weights.argtypes = [_c.c_int32] * 4 + [_vp] * 6
    L.q8_swiglu_forward.restype = _c.c_int
    L.q8_swiglu_forward.argtypes = [_c.POINTER(Q8Plan)] + [_vp] * 9
    L.q8_swiglu_backward.restype = _c.c_int
    L.q8_swiglu_backward.argtypes = [_c.POINTER(Q8Plan)] + [_vp] * 8
    L.gmm_plan.restype = _c.c_int
    L.gmm_plan.argtypes = [_c.c_int64] + [_c.c_int32] * 4 + [_c.POINTER(GmmPlan)]
    for f in (L.gmm_forward, L.gmm_backward_dx):
        f.restype = _c.c_int
        f.argtypes = [_c.POINTER(GmmPlan)] + [_vp] * 5 + [_c.c_size_t, _vp]
    L.gmm_backward_dw.restype = _c.c_int
    L.gmm_backward_dw.argtypes = [_c.POINTER(GmmPlan)] + [_vp] * 4 + [_c.c_int32, _vp, _c.c_size_t, _vp]
    L.gmm8_forward.restype = _c.c_int
    L.gmm8_forward.argtypes = [_c.POINTER(GmmPlan)] + [_vp] * 7 + [_c.c_size_t, _vp]
    L.gmm8_backward_dw.restype = _c.c_int
    L.gmm8_backward_dw.argtypes = [_c.POINTER(GmmPlan)] + [_vp] * 5 + [_c.c_int32, _vp, _c.c_size_t, _vp]
    _LIB = L
    return L


def declared_functions() -> list:
    """Function names declared in include/moebound.h and include/cce.h."""
    return _declared(HEADERS, "moe|cce")


def declared_operators() -> list:
    """Function names declared in the headers of the operators around the layer."""
    return _declared(OPERATOR_HEADERS, "moe|route|lnorm|embed|kd")


def declared_expert_operators() -> list:
    """Function names declared in the headers of the 8-bit path of an expert layer."""
    return _declared(EXPERT_HEADERS, "rms|q8|gmm8?")


def _declared(headers, prefixes) -> list:
    names = set()
    for h in headers:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:%s)_[a-z0-9_]+)\s*\(" % prefixes, text))
    return sorted(names)


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def torch_dtype(dtype: int) -> torch.dtype:
    return torch.bfloat16 if dtype == MOE_BF16 else torch.float32


def moe_dtype(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return MOE_BF16
    if t == torch.float32:
        return MOE_F32
    raise ValueError(f"unsupported dtype {t}")


def _expect(t, name, shape, dtype, device):
    if (t is not None and t.shape == shape and t.dtype is dtype and t.device == device
            and t.is_contiguous()):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: device {t.device} != {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The raw handle of a device's current stream; torch's public call builds a
# Stream object for it, ten times the time (1.9 us of a call of 10).  And the
# current device without the public call's look at whether torch has started.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# A new tensor on the current device without the public call's reading of its arguments
# (0.8 us for 1.3, and a call has up to six).  Only where torch.empty does no more than that:
# it fills new memory under deterministic algorithms, and dispatch modes see it.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
_deterministic = getattr(torch._C, "_get_deterministic_algorithms", torch.are_deterministic_algorithms_enabled)
_dispatch_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
if _dispatch_modes is None:
    _empty_strided = None


def _stream(device, stream):
    if stream is None:
        if _raw_stream is not None and device.type == "cuda" and device.index is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context in which a call on ``device`` and ``stream`` (None: the device's
    current stream) allocates and launches: outputs and workspaces then belong
    to the stream that writes them, whatever device or stream is current."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        return torch.cuda.stream(stream)
    return _HERE if device.index == _current_device() else torch.cuda.device(device)


def _workspace(ws, plan, kind, device):
    """(workspace, its bytes): the one given, on the device and in one piece, or a new one."""
    if ws is None:
        ws = workspace(plan, kind, device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return ws, ws.numel() * ws.element_size()


def _out(t, name, shape, dtype, device):
    """The output tensor given, checked, or a new one (on the current device, see _on)."""
    if t is None:
        if _empty_strided is not None and not _deterministic() and not _dispatch_modes():
            n = len(shape)
            if n == 2:
                return _empty_strided(shape, (shape[1] or 1, 1), dtype)
            if n == 1:
                return _empty_strided(shape, (1,), dtype)
            if n == 3:
                row = shape[2] or 1
                return _empty_strided(shape, ((shape[1] or 1) * row, row, 1), dtype)
        return torch.empty(*shape, dtype=dtype, device=device)  # sizes one by one: 1.2 us, a tuple 1.6
    _expect(t, name, shape, dtype, device)
    return t


def moe_plan_chunks(N: int, H: int, F: int, E: int, k: int, c: int, K_max: int,
                    dtype: int) -> MoePlan:
    plan = MoePlan()
    _check(lib().moe_plan_chunks(N, H, F, E, k, c, K_max, dtype, ctypes.byref(plan)),
           "moe_plan_chunks")
    return plan


MOE_PLAN_EXACT_DW = 1


def moe_plan_set_flags(plan: MoePlan, flags: int) -> MoePlan:
    """Set the plan's options in place (MOE_PLAN_EXACT_DW: order-invariant
    expert weight gradients); returns the plan."""
    _check(lib().moe_plan_set_flags(ctypes.byref(plan), flags), "moe_plan_set_flags")
    return plan


def workspace(plan, kind: str, device) -> torch.Tensor:
    """Workspace of a MoePlan ("fwd", "bwd", "debug"), CcePlan, KdPlan or GmmPlan ("fwd",
    "bwd"), LnormPlan, EmbedPlan or RmsPlan ("bwd"); "both" is large enough for "fwd" and
    "bwd"."""
    if kind == "both":
        n = max(plan.fwd_workspace_bytes, plan.bwd_workspace_bytes)
    else:
        n = getattr(plan, {"fwd": "fwd_workspace_bytes", "bwd": "bwd_workspace_bytes",
                           "debug": "debug_workspace_bytes"}[kind])
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def moe_bounded_forward(plan: MoePlan, X, W_r, router_bias, W_gate, W_up, W_down,
                        Y=None, topk_idx=None, gates=None, logits=None, want_logits=True,
                        ws=None, stream=None):
    """Returns (Y, topk_idx, gates, logits or None, stats dict)."""
    dev = X.device
    dt = torch_dtype(plan.dtype)
    N, H, F, E, k = plan.N, plan.H, plan.F, plan.E, plan.k
    _expect(X, "X", (N, H), dt, dev)
    _expect(W_r, "W_r", (H, E), dt, dev)
    if router_bias is not None:
        _expect(router_bias, "router_bias", (E,), torch.float32, dev)
    _expect(W_gate, "W_gate", (E, H, F), dt, dev)
    _expect(W_up, "W_up", (E, H, F), dt, dev)
    _expect(W_down, "W_down", (E, F, H), dt, dev)
    Y = torch.empty((N, H), dtype=dt, device=dev) if Y is None else Y
    topk_idx = torch.empty((N, k), dtype=torch.int32, device=dev) if topk_idx is None else topk_idx
    gates = torch.empty((N, k), dtype=torch.float32, device=dev) if gates is None else gates
    if logits is None and want_logits:
        logits = torch.empty((N, E), dtype=torch.float32, device=dev)
    _expect(Y, "Y", (N, H), dt, dev)
    _expect(topk_idx, "topk_idx", (N, k), torch.int32, dev)
    _expect(gates, "gates", (N, k), torch.float32, dev)
    if logits is not None:
        _expect(logits, "logits", (N, E), torch.float32, dev)
    ws = workspace(plan, "fwd", dev) if ws is None else ws
    st = MoeStats()
    _check(lib().moe_bounded_forward(
        ctypes.byref(plan), _ptr(X), _ptr(W_r), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
        _ptr(W_down), _ptr(Y), _ptr(topk_idx), _ptr(gates), _ptr(logits), _ptr(ws),
        ws.numel(), _stream(dev, stream), ctypes.byref(st)), "moe_bounded_forward")
    return Y, topk_idx, gates, logits, st.as_dict()


def moe_bounded_forward_static(plan: MoePlan, X, W_r, router_bias, W_gate, W_up, W_down,
                               Y=None, topk_idx=None, gates=None, logits=None,
                               want_logits=True, stream=None):
    """moe_bounded_forward on the library's static scratch array (no
    workspace).  Returns (Y, topk_idx, gates, logits or None, stats dict)."""
    dev = X.device
    dt = torch_dtype(plan.dtype)
    N, H, F, E, k = plan.N, plan.H, plan.F, plan.E, plan.k
    _expect(X, "X", (N, H), dt, dev)
    _expect(W_r, "W_r", (H, E), dt, dev)
    if router_bias is not None:
        _expect(router_bias, "router_bias", (E,), torch.float32, dev)
    _expect(W_gate, "W_gate", (E, H, F), dt, dev)
    _expect(W_up, "W_up", (E, H, F), dt, dev)
    _expect(W_down, "W_down", (E, F, H), dt, dev)
    Y = torch.empty((N, H), dtype=dt, device=dev) if Y is None else Y
    topk_idx = torch.empty((N, k), dtype=torch.int32, device=dev) if topk_idx is None else topk_idx
    gates = torch.empty((N, k), dtype=torch.float32, device=dev) if gates is None else gates
    if logits is None and want_logits:
        logits = torch.empty((N, E), dtype=torch.float32, device=dev)
    _expect(Y, "Y", (N, H), dt, dev)
    _expect(topk_idx, "topk_idx", (N, k), torch.int32, dev)
    _expect(gates, "gates", (N, k), torch.float32, dev)
    if logits is not None:
        _expect(logits, "logits", (N, E), torch.float32, dev)
    st = MoeStats()
    _check(lib().moe_bounded_forward_static(
        ctypes.byref(plan), _ptr(X), _ptr(W_r), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
        _ptr(W_down), _ptr(Y), _ptr(topk_idx), _ptr(gates), _ptr(logits),
        _stream(dev, stream), ctypes.byref(st)), "moe_bounded_forward_static")
    return Y, topk_idx, gates, logits, st.as_dict()


def moe_bounded_backward(plan: MoePlan, X, W_r, W_gate, W_up, W_down, dY, topk_idx, gates,
                         dX=None, dW_gate=None, dW_up=None, dW_down=None, dlogits=None,
                         dgates=None, want_dgates=True, dW_r=None, want_dW_r=True, ws=None,
                         stream=None):
    """Returns dict with dX, dW_gate, dW_up, dW_down, dlogits, dgates, dW_r, stats."""
    dev = X.device
    dt = torch_dtype(plan.dtype)
    N, H, F, E, k = plan.N, plan.H, plan.F, plan.E, plan.k
    f32 = torch.float32
    for t, n, s, d in ((X, "X", (N, H), dt), (W_r, "W_r", (H, E), dt),
                       (W_gate, "W_gate", (E, H, F), dt), (W_up, "W_up", (E, H, F), dt),
                       (W_down, "W_down", (E, F, H), dt), (dY, "dY", (N, H), dt),
                       (topk_idx, "topk_idx", (N, k), torch.int32), (gates, "gates", (N, k), f32)):
        _expect(t, n, s, d, dev)
    new = lambda shape, d=f32: torch.empty(shape, dtype=d, device=dev)
    dX = new((N, H), dt) if dX is None else dX
    dW_gate = new((E, H, F)) if dW_gate is None else dW_gate
    dW_up = new((E, H, F)) if dW_up is None else dW_up
    dW_down = new((E, F, H)) if dW_down is None else dW_down
    dlogits = new((N, E)) if dlogits is None else dlogits
    if dgates is None and want_dgates:
        dgates = new((N, k))
    if dW_r is None and want_dW_r:
        dW_r = new((H, E))
    _expect(dX, "dX", (N, H), dt, dev)
    _expect(dW_gate, "dW_gate", (E, H, F), f32, dev)
    _expect(dW_up, "dW_up", (E, H, F), f32, dev)
    _expect(dW_down, "dW_down", (E, F, H), f32, dev)
    _expect(dlogits, "dlogits", (N, E), f32, dev)
    if dgates is not None:
        _expect(dgates, "dgates", (N, k), f32, dev)
    if dW_r is not None:
        _expect(dW_r, "dW_r", (H, E), f32, dev)
    ws = workspace(plan, "bwd", dev) if ws is None else ws
    st = MoeStats()
    _check(lib().moe_bounded_backward(
        ctypes.byref(plan), _ptr(X), _ptr(W_r), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(dY), _ptr(topk_idx), _ptr(gates), _ptr(dX), _ptr(dW_gate), _ptr(dW_up),
        _ptr(dW_down), _ptr(dlogits), _ptr(dgates), _ptr(dW_r), _ptr(ws), ws.numel(),
        _stream(dev, stream), ctypes.byref(st)), "moe_bounded_backward")
    return dict(dX=dX, dW_gate=dW_gate, dW_up=dW_up, dW_down=dW_down, dlogits=dlogits,
                dgates=dgates, dW_r=dW_r, stats=st.as_dict())


def moe_debug_topk(logits: torch.Tensor, k: int, stream=None):
    dev = logits.device
    N, E = logits.shape
    _expect(logits, "logits", (N, E), torch.float32, dev)
    idx = torch.empty((N, k), dtype=torch.int32, device=dev)
    gates = torch.empty((N, k), dtype=torch.float32, device=dev)
    _check(lib().moe_debug_topk(_ptr(logits), N, E, k, _ptr(idx), _ptr(gates),
                                _stream(dev, stream)), "moe_debug_topk")
    return idx, gates


def moe_debug_plan(plan: MoePlan, topk_idx: torch.Tensor, stream=None):
    """Returns (offsets [K, E+1], perm [N*k], pos [N*k]) as int32 device tensors."""
    dev = topk_idx.device
    _expect(topk_idx, "topk_idx", (plan.N, plan.k), torch.int32, dev)
    offsets = torch.empty((plan.K, plan.E + 1), dtype=torch.int32, device=dev)
    perm = torch.empty(plan.N * plan.k, dtype=torch.int32, device=dev)
    pos = torch.empty(plan.N * plan.k, dtype=torch.int32, device=dev)
    ws = workspace(plan, "debug", dev)
    _check(lib().moe_debug_plan(ctypes.byref(plan), _ptr(topk_idx), _ptr(offsets), _ptr(perm),
                                _ptr(pos), _ptr(ws), ws.numel(), _stream(dev, stream)),
           "moe_debug_plan")
    return offsets, perm, pos


def moe_debug_stage(plan: MoePlan, stage: str, chunk: int, X, W_r, router_bias, W_gate, W_up,
                    W_down, Y, topk_idx, gates, ws, stream=None):
    """Re-launch one forward stage for one chunk (state from the last forward
    call on ``ws``, which must have been made with logits=None)."""
    _check(lib().moe_debug_stage(ctypes.byref(plan), STAGES[stage], chunk, _ptr(X), _ptr(W_r),
                                 _ptr(router_bias), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                 _ptr(Y), _ptr(topk_idx), _ptr(gates), _ptr(ws), ws.numel(),
                                 _stream(X.device, stream)), "moe_debug_stage")


def moe_debug_stage_bwd(plan: MoePlan, stage: str, chunk: int, X, W_r, W_gate, W_up, W_down, dY,
                        topk_idx, gates, grads: dict, ws, stream=None):
    """Re-launch one backward stage (for one chunk) on the state of the last
    backward call on ``ws``; ``grads`` holds that call's output tensors (the
    dict moe_bounded_backward returns, or the tensors passed to it)."""
    _check(lib().moe_debug_stage_bwd(
        ctypes.byref(plan), BSTAGES[stage], chunk, _ptr(X), _ptr(W_r), _ptr(W_gate), _ptr(W_up),
        _ptr(W_down), _ptr(dY), _ptr(topk_idx), _ptr(gates), _ptr(grads["dX"]),
        _ptr(grads["dW_gate"]), _ptr(grads["dW_up"]), _ptr(grads["dW_down"]),
        _ptr(grads["dlogits"]), _ptr(grads.get("dgates")), _ptr(grads.get("dW_r")), _ptr(ws),
        ws.numel(), _stream(X.device, stream)), "moe_debug_stage_bwd")


# ---- vocabulary projection with cross-entropy over vocabulary strips


def cce_plan(N: int, H: int, V: int, v_chunk: int, dtype: int = MOE_BF16) -> CcePlan:
    plan = CcePlan()
    _check(lib().cce_plan(N, H, V, v_chunk, dtype, ctypes.byref(plan)), "cce_plan")
    return plan


def cce_forward(plan: CcePlan, X, W, targets, loss=None, lse=None, ws=None, stream=None):
    """Returns (loss [N], lse [N]) fp32."""
    dev = X.device
    N, H, V = plan.N, plan.H, plan.V
    _expect(X, "X", (N, H), torch.bfloat16, dev)
    _expect(W, "W", (V, H), torch.bfloat16, dev)
    _expect(targets, "targets", (N,), torch.int32, dev)
    loss = torch.empty(N, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    _expect(loss, "loss", (N,), torch.float32, dev)
    _expect(lse, "lse", (N,), torch.float32, dev)
    ws = workspace(plan, "fwd", dev) if ws is None else ws
    _check(lib().cce_forward(ctypes.byref(plan), _ptr(X), _ptr(W), _ptr(targets), _ptr(loss),
                             _ptr(lse), _ptr(ws), ws.numel(), _stream(dev, stream)),
           "cce_forward")
    return loss, lse


def cce_backward(plan: CcePlan, X, W, targets, lse, dloss, dX=None, dW=None, ws=None,
                 stream=None):
    """Returns (dX [N, H] bf16, dW [V, H] fp32)."""
    dev = X.device
    N, H, V = plan.N, plan.H, plan.V
    f32 = torch.float32
    for t, n, shp, d in ((X, "X", (N, H), torch.bfloat16), (W, "W", (V, H), torch.bfloat16),
                         (targets, "targets", (N,), torch.int32), (lse, "lse", (N,), f32),
                         (dloss, "dloss", (N,), f32)):
        _expect(t, n, shp, d, dev)
    dX = torch.empty((N, H), dtype=torch.bfloat16, device=dev) if dX is None else dX
    dW = torch.empty((V, H), dtype=f32, device=dev) if dW is None else dW
    _expect(dX, "dX", (N, H), torch.bfloat16, dev)
    _expect(dW, "dW", (V, H), f32, dev)
    ws = workspace(plan, "bwd", dev) if ws is None else ws
    _check(lib().cce_backward(ctypes.byref(plan), _ptr(X), _ptr(W), _ptr(targets), _ptr(lse),
                              _ptr(dloss), _ptr(dX), _ptr(dW), _ptr(ws), ws.numel(),
                              _stream(dev, stream)), "cce_backward")
    return dX, dW


def cce_debug_stage(plan: CcePlan, stage: str, strip: int, X, W, targets, loss, lse, dloss, dX,
                    dW, ws, stream=None):
    """Re-launch one kernel of one strip (state from the last cce_forward or
    cce_backward call on ``ws``)."""
    _check(lib().cce_debug_stage(ctypes.byref(plan), CCE_STAGES[stage], strip, _ptr(X), _ptr(W),
                                 _ptr(targets), _ptr(loss), _ptr(lse), _ptr(dloss), _ptr(dX),
                                 _ptr(dW), _ptr(ws), ws.numel(), _stream(X.device, stream)),
           "cce_debug_stage")


# ---- routing by scores, and the layer under a given routing


def route_plan(N: int, E: int, k: int, score: str = "softmax", n_group: int = 1,
               topk_group: int = 1, group_top: int = 2, renorm: bool = True,
               scale: float = 1.0) -> RoutePlan:
    """Routing of N tokens to k of E experts; score "softmax" or "sigmoid"."""
    if score not in ROUTE_SCORES:
        raise ValueError(f"score {score!r} is not one of {sorted(ROUTE_SCORES)}")
    plan = RoutePlan()
    _check(lib().route_plan(N, E, k, ROUTE_SCORES[score], n_group, topk_group, group_top,
                            int(renorm), scale, ctypes.byref(plan)), "route_plan")
    return plan


def route_forward(plan: RoutePlan, logits, bias=None, topk_idx=None, gates=None, stream=None):
    """Returns (topk_idx [N, k] int32, gates [N, k] fp32)."""
    dev = logits.device
    N, E, k = plan.N, plan.E, plan.k
    _expect(logits, "logits", (N, E), torch.float32, dev)
    if bias is not None:
        _expect(bias, "bias", (E,), torch.float32, dev)
    with _on(dev, stream):
        topk_idx = _out(topk_idx, "topk_idx", (N, k), torch.int32, dev)
        gates = _out(gates, "gates", (N, k), torch.float32, dev)
        _check(lib().route_forward(ctypes.byref(plan), _ptr(logits), _ptr(bias), _ptr(topk_idx),
                                   _ptr(gates), _stream(dev, None)), "route_forward")
    return topk_idx, gates


def route_backward(plan: RoutePlan, logits, topk_idx, dgates, dlogits=None, stream=None):
    """Returns dlogits [N, E] fp32."""
    dev = logits.device
    N, E, k = plan.N, plan.E, plan.k
    _expect(logits, "logits", (N, E), torch.float32, dev)
    _expect(topk_idx, "topk_idx", (N, k), torch.int32, dev)
    _expect(dgates, "dgates", (N, k), torch.float32, dev)
    with _on(dev, stream):
        dlogits = _out(dlogits, "dlogits", (N, E), torch.float32, dev)
        _check(lib().route_backward(ctypes.byref(plan), _ptr(logits), _ptr(topk_idx), _ptr(dgates),
                                    _ptr(dlogits), _stream(dev, None)), "route_backward")
    return dlogits


def moe_routed_forward(plan: MoePlan, X, W_gate, W_up, W_down, topk_idx, gates, Y=None, ws=None,
                       stream=None):
    """The layer's experts under a given routing.  Returns (Y, stats dict)."""
    dev = X.device
    dt = torch_dtype(plan.dtype)
    N, H, F, E, k = plan.N, plan.H, plan.F, plan.E, plan.k
    for t, n, s, d in ((X, "X", (N, H), dt), (W_gate, "W_gate", (E, H, F), dt),
                       (W_up, "W_up", (E, H, F), dt), (W_down, "W_down", (E, F, H), dt),
                       (topk_idx, "topk_idx", (N, k), torch.int32),
                       (gates, "gates", (N, k), torch.float32)):
        _expect(t, n, s, d, dev)
    with _on(dev, stream):
        Y = _out(Y, "Y", (N, H), dt, dev)
        ws, ws_bytes = _workspace(ws, plan, "fwd", dev)
        st = MoeStats()
        _check(lib().moe_routed_forward(
            ctypes.byref(plan), _ptr(X), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(topk_idx),
            _ptr(gates), _ptr(Y), _ptr(ws), ws_bytes, _stream(dev, None), ctypes.byref(st)),
            "moe_routed_forward")
    return Y, st.as_dict()


def moe_routed_backward(plan: MoePlan, X, W_gate, W_up, W_down, dY, topk_idx, gates, dX=None,
                        dW_gate=None, dW_up=None, dW_down=None, dgates=None, ws=None, stream=None):
    """Returns dict with dX (the experts' share), dW_gate, dW_up, dW_down, dgates, stats."""
    dev = X.device
    dt = torch_dtype(plan.dtype)
    N, H, F, E, k = plan.N, plan.H, plan.F, plan.E, plan.k
    f32 = torch.float32
    for t, n, s, d in ((X, "X", (N, H), dt), (W_gate, "W_gate", (E, H, F), dt),
                       (W_up, "W_up", (E, H, F), dt), (W_down, "W_down", (E, F, H), dt),
                       (dY, "dY", (N, H), dt), (topk_idx, "topk_idx", (N, k), torch.int32),
                       (gates, "gates", (N, k), f32)):
        _expect(t, n, s, d, dev)
    with _on(dev, stream):
        dX = _out(dX, "dX", (N, H), dt, dev)
        dW_gate = _out(dW_gate, "dW_gate", (E, H, F), f32, dev)
        dW_up = _out(dW_up, "dW_up", (E, H, F), f32, dev)
        dW_down = _out(dW_down, "dW_down", (E, F, H), f32, dev)
        dgates = _out(dgates, "dgates", (N, k), f32, dev)
        ws, ws_bytes = _workspace(ws, plan, "bwd", dev)
        st = MoeStats()
        _check(lib().moe_routed_backward(
            ctypes.byref(plan), _ptr(X), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(dY),
            _ptr(topk_idx), _ptr(gates), _ptr(dX), _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down),
            _ptr(dgates), _ptr(ws), ws_bytes, _stream(dev, None), ctypes.byref(st)),
            "moe_routed_backward")
    return dict(dX=dX, dW_gate=dW_gate, dW_up=dW_up, dW_down=dW_down, dgates=dgates,
                stats=st.as_dict())


# ---- layer norm


def lnorm_plan(N: int, H: int, dtype: int = MOE_BF16, eps: float = 1e-5) -> LnormPlan:
    plan = LnormPlan()
    _check(lib().lnorm_plan(N, H, dtype, eps, ctypes.byref(plan)), "lnorm_plan")
    return plan


def lnorm_forward(plan: LnormPlan, X, gamma, beta=None, Y=None, mean=None, rstd=None, stream=None):
    """Returns (Y [N, H], mean [N], rstd [N])."""
    dev = X.device
    dt, f32 = torch_dtype(plan.dtype), torch.float32
    N, H = plan.N, plan.H
    _expect(X, "X", (N, H), dt, dev)
    _expect(gamma, "gamma", (H,), f32, dev)
    if beta is not None:
        _expect(beta, "beta", (H,), f32, dev)
    with _on(dev, stream):
        Y = _out(Y, "Y", (N, H), dt, dev)
        mean = _out(mean, "mean", (N,), f32, dev)
        rstd = _out(rstd, "rstd", (N,), f32, dev)
        _check(lib().lnorm_forward(ctypes.byref(plan), _ptr(X), _ptr(gamma), _ptr(beta), _ptr(Y),
                                   _ptr(mean), _ptr(rstd), _stream(dev, None)), "lnorm_forward")
    return Y, mean, rstd


def lnorm_backward(plan: LnormPlan, X, gamma, dY, mean, rstd, dX=None, dgamma=None, dbeta=None,
                   want_dbeta=True, ws=None, stream=None):
    """Returns (dX [N, H], dgamma [H], dbeta [H] or None)."""
    dev = X.device
    dt, f32 = torch_dtype(plan.dtype), torch.float32
    N, H = plan.N, plan.H
    for t, n, s, d in ((X, "X", (N, H), dt), (gamma, "gamma", (H,), f32), (dY, "dY", (N, H), dt),
                       (mean, "mean", (N,), f32), (rstd, "rstd", (N,), f32)):
        _expect(t, n, s, d, dev)
    with _on(dev, stream):
        dX = _out(dX, "dX", (N, H), dt, dev)
        dgamma = _out(dgamma, "dgamma", (H,), f32, dev)
        if dbeta is not None or want_dbeta:
            dbeta = _out(dbeta, "dbeta", (H,), f32, dev)
        ws, ws_bytes = _workspace(ws, plan, "bwd", dev)
        _check(lib().lnorm_backward(ctypes.byref(plan), _ptr(X), _ptr(gamma), _ptr(dY), _ptr(mean),
                                    _ptr(rstd), _ptr(dX), _ptr(dgamma), _ptr(dbeta), _ptr(ws),
                                    ws_bytes, _stream(dev, None)), "lnorm_backward")
    return dX, dgamma, dbeta


# ---- token embedding


def embed_plan(N: int, V: int, H: int, dtype: int = MOE_BF16, scale: float = 1.0) -> EmbedPlan:
    plan = EmbedPlan()
    _check(lib().embed_plan(N, V, H, dtype, scale, ctypes.byref(plan)), "embed_plan")
    return plan


def embed_forward(plan: EmbedPlan, W, ids, Y=None, stream=None):
    """Returns Y [N, H] = scale W[ids] (0 for an id outside [0, V))."""
    dev = W.device
    dt = torch_dtype(plan.dtype)
    N, V, H = plan.N, plan.V, plan.H
    _expect(W, "W", (V, H), dt, dev)
    _expect(ids, "ids", (N,), torch.int32, dev)
    with _on(dev, stream):
        Y = _out(Y, "Y", (N, H), dt, dev)
        _check(lib().embed_forward(ctypes.byref(plan), _ptr(W), _ptr(ids), _ptr(Y),
                                   _stream(dev, None)), "embed_forward")
    return Y


def embed_backward(plan: EmbedPlan, ids, dY, dW=None, accumulate=False, ws=None, stream=None):
    """Returns dW [V, H] fp32; with accumulate the gradient is added to the dW given."""
    dev = dY.device
    N, V, H = plan.N, plan.V, plan.H
    _expect(ids, "ids", (N,), torch.int32, dev)
    _expect(dY, "dY", (N, H), torch_dtype(plan.dtype), dev)
    if accumulate and dW is None:
        raise ValueError("accumulate needs the dW to add to")
    with _on(dev, stream):
        dW = _out(dW, "dW", (V, H), torch.float32, dev)
        ws, ws_bytes = _workspace(ws, plan, "bwd", dev)
        _check(lib().embed_backward(ctypes.byref(plan), _ptr(ids), _ptr(dY), _ptr(dW),
                                    int(bool(accumulate)), _ptr(ws), ws_bytes,
                                    _stream(dev, None)), "embed_backward")
    return dW


# ---- distillation from a teacher's top logits over vocabulary strips


def kd_plan(N: int, H: int, V: int, v_chunk: int, K: int, temperature: float = 1.0,
            dtype: int = MOE_BF16, dw_dtype: int = MOE_F32) -> KdPlan:
    plan = KdPlan()
    _check(lib().kd_plan(N, H, V, v_chunk, K, temperature, dtype, dw_dtype, ctypes.byref(plan)),
           "kd_plan")
    return plan


def kd_forward(plan: KdPlan, X, W, t_idx, t_logit, loss=None, lse=None, y_top=None, ws=None,
               stream=None):
    """Returns (loss [N], lse [N], y_top [N, K]) fp32."""
    dev = X.device
    N, H, V, K = plan.N, plan.H, plan.V, plan.K
    f32 = torch.float32
    for t, n, s, d in ((X, "X", (N, H), torch.bfloat16), (W, "W", (V, H), torch.bfloat16),
                       (t_idx, "t_idx", (N, K), torch.int32), (t_logit, "t_logit", (N, K), f32)):
        _expect(t, n, s, d, dev)
    with _on(dev, stream):
        loss = _out(loss, "loss", (N,), f32, dev)
        lse = _out(lse, "lse", (N,), f32, dev)
        y_top = _out(y_top, "y_top", (N, K), f32, dev)
        ws, ws_bytes = _workspace(ws, plan, "fwd", dev)
        _check(lib().kd_forward(ctypes.byref(plan), _ptr(X), _ptr(W), _ptr(t_idx), _ptr(t_logit),
                                _ptr(loss), _ptr(lse), _ptr(y_top), _ptr(ws), ws_bytes,
                                _stream(dev, None)), "kd_forward")
    return loss, lse, y_top


def kd_backward(plan: KdPlan, X, W, t_idx, t_logit, lse, y_top, dloss, dX=None, dW=None, ws=None,
                stream=None):
    """Returns (dX [N, H] bf16, dW [V, H] in the plan's dw_dtype)."""
    dev = X.device
    N, H, V, K = plan.N, plan.H, plan.V, plan.K
    f32, bf16, wt = torch.float32, torch.bfloat16, torch_dtype(plan.dw_dtype)
    for t, n, s, d in ((X, "X", (N, H), bf16), (W, "W", (V, H), bf16),
                       (t_idx, "t_idx", (N, K), torch.int32), (t_logit, "t_logit", (N, K), f32),
                       (lse, "lse", (N,), f32), (y_top, "y_top", (N, K), f32),
                       (dloss, "dloss", (N,), f32)):
        _expect(t, n, s, d, dev)
    with _on(dev, stream):
        dX = _out(dX, "dX", (N, H), bf16, dev)
        dW = _out(dW, "dW", (V, H), wt, dev)
        ws, ws_bytes = _workspace(ws, plan, "bwd", dev)
        _check(lib().kd_backward(ctypes.byref(plan), _ptr(X), _ptr(W), _ptr(t_idx), _ptr(t_logit),
                                 _ptr(lse), _ptr(y_top), _ptr(dloss), _ptr(dX), _ptr(dW), _ptr(ws),
                                 ws_bytes, _stream(dev, None)), "kd_backward")
    return dX, dW


# ---- root-mean-square norm with the residual's addition

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def rms_plan(N: int, H: int, dtype: int = MOE_BF16, eps: float = 1e-6) -> RmsPlan:
    plan = RmsPlan()
    _check(lib().rms_plan(N, H, dtype, eps, ctypes.byref(plan)), "rms_plan")
    return plan


def _rms_inputs(plan, X, gamma, residual, S):
    dev, dt = X.device, torch_dtype(plan.dtype)
    N, H = plan.N, plan.H
    _expect(X, "X", (N, H), dt, dev)
    _expect(gamma, "gamma", (H,), torch.float32, dev)
    if residual is not None:
        _expect(residual, "residual", (N, H), dt, dev)
    elif S is not None:
        raise ValueError("S is X itself without a residual")
    return dev, dt, N, H


def rms_forward(plan: RmsPlan, X, gamma, residual=None, S=None, Y=None, rstd=None, stream=None):
    """Returns (Y [N, H], S = X + residual [N, H], rstd [N]); S is X itself without a residual."""
    dev, dt, N, H = _rms_inputs(plan, X, gamma, residual, S)
    with _on(dev, stream):
        if residual is not None:
            S = _out(S, "S", (N, H), dt, dev)
        Y = _out(Y, "Y", (N, H), dt, dev)
        rstd = _out(rstd, "rstd", (N,), torch.float32, dev)
        _check(lib().rms_forward(ctypes.byref(plan), _ptr(X), _ptr(residual), _ptr(gamma), _ptr(S),
                                 _ptr(Y), _ptr(rstd), _stream(dev, None)), "rms_forward")
    return Y, X if S is None else S, rstd


def rms_forward_q8(plan: RmsPlan, X, gamma, residual=None, S=None, Yq=None, Ys=None, rstd=None,
                   stream=None):
    """Returns (Yq, Ys, S, rstd): Y as rows of 8 bits (see q8_pack), the rest as rms_forward."""
    dev, dt, N, H = _rms_inputs(plan, X, gamma, residual, S)
    with _on(dev, stream):
        if residual is not None:
            S = _out(S, "S", (N, H), dt, dev)
        Yq = _out(Yq, "Yq", (N, plan.row_pitch), E4M3, dev)
        Ys = _out(Ys, "Ys", (N, plan.scale_pitch), E8M0, dev)
        rstd = _out(rstd, "rstd", (N,), torch.float32, dev)
        _check(lib().rms_forward_q8(ctypes.byref(plan), _ptr(X), _ptr(residual), _ptr(gamma),
                                    _ptr(S), _ptr(Yq), _ptr(Ys), _ptr(rstd), _stream(dev, None)),
               "rms_forward_q8")
    return Yq, Ys, X if S is None else S, rstd


def rms_backward(plan: RmsPlan, S, gamma, dY, rstd, dS=None, dX=None, dgamma=None, ws=None,
                 stream=None):
    """Returns (dX [N, H], the gradient of X and of the residual alike, dgamma [H])."""
    dev = S.device
    dt, f32 = torch_dtype(plan.dtype), torch.float32
    N, H = plan.N, plan.H
    for t, n, s, d in ((S, "S", (N, H), dt), (gamma, "gamma", (H,), f32), (dY, "dY", (N, H), dt),
                       (rstd, "rstd", (N,), f32)):
        _expect(t, n, s, d, dev)
    if dS is not None:
        _expect(dS, "dS", (N, H), dt, dev)
    with _on(dev, stream):
        dX = _out(dX, "dX", (N, H), dt, dev)
        dgamma = _out(dgamma, "dgamma", (H,), f32, dev)
        ws, ws_bytes = _workspace(ws, plan, "bwd", dev)
        _check(lib().rms_backward(ctypes.byref(plan), _ptr(S), _ptr(gamma), _ptr(dY), _ptr(rstd),
                                  _ptr(dS), _ptr(dX), _ptr(dgamma), _ptr(ws), ws_bytes,
                                  _stream(dev, None)), "rms_backward")
    return dX, dgamma


# ---- rows in 8 bits, SwiGLU with checkpoints in 8 bits


def q8_plan(N: int, H: int, dtype: int = MOE_BF16) -> Q8Plan:
    plan = Q8Plan()
    _check(lib().q8_plan(N, H, dtype, ctypes.byref(plan)), "q8_plan")
    return plan


def _expect_q8(plan, q, s, name, dev):
    _expect(q, name + "q", (plan.N, plan.row_pitch), E4M3, dev)
    _expect(s, name + "s", (plan.N, plan.scale_pitch), E8M0, dev)


def _out_q8(plan, q, s, name, dev):
    return (_out(q, name + "q", (plan.N, plan.row_pitch), E4M3, dev),
            _out(s, name + "s", (plan.N, plan.scale_pitch), E8M0, dev))


def q8_pack(plan: Q8Plan, X, q=None, s=None, stream=None):
    """Returns (q [N, row_pitch] float8_e4m3fn, s [N, scale_pitch] float8_e8m0fnu)."""
    dev = X.device
    _expect(X, "X", (plan.N, plan.H), torch_dtype(plan.dtype), dev)
    with _on(dev, stream):
        q, s = _out_q8(plan, q, s, "", dev)
        _check(lib().q8_pack(ctypes.byref(plan), _ptr(X), _ptr(q), _ptr(s), _stream(dev, None)),
               "q8_pack")
    return q, s


def q8_unpack(plan: Q8Plan, q, s, X=None, stream=None):
    """Returns the values X [N, H]."""
    dev = q.device
    _expect_q8(plan, q, s, "", dev)
    with _on(dev, stream):
        X = _out(X, "X", (plan.N, plan.H), torch_dtype(plan.dtype), dev)
        _check(lib().q8_unpack(ctypes.byref(plan), _ptr(q), _ptr(s), _ptr(X), _stream(dev, None)),
               "q8_unpack")
    return X


def q8_pack_weights(W, along="both", stream=None):
    """E matrices W [E, K, N] in 8 bits with a scale per 128 x 128: along "K" (qt [E, N, K to 128],
    st), for products that sum over K; along "N" (q [E, K, N to 128], s), for those that sum over N;
    or "both" (qt, st, q, s)."""
    if along not in ("K", "N", "both"):
        raise ValueError(f"along: {along!r}")
    if W.dim() != 3:
        raise ValueError(f"W: {W.dim()} dimensions, 3 are wanted")
    dev, dtype = W.device, moe_dtype(W.dtype)
    E, K, N = W.shape
    _expect(W, "W", (E, K, N), W.dtype, dev)
    kb, nb = -(-K // 128), -(-N // 128)
    with _on(dev, stream):
        qt = st = q = s = None
        if along != "N":
            qt = torch.empty((E, N, kb * 128), dtype=E4M3, device=dev)
            st = torch.empty((E, nb, -(-kb // 4) * 4), dtype=E8M0, device=dev)
        if along != "K":
            q = torch.empty((E, K, nb * 128), dtype=E4M3, device=dev)
            s = torch.empty((E, kb, -(-nb // 4) * 4), dtype=E8M0, device=dev)
        _check(lib().q8_pack_weights(E, K, N, dtype, _ptr(W), _ptr(q), _ptr(s), _ptr(qt), _ptr(st),
                                     _stream(dev, None)), "q8_pack_weights")
    return {"K": (qt, st), "N": (q, s), "both": (qt, st, q, s)}[along]


def q8_swiglu_forward(plan: Q8Plan, A, U, keep=True, H=None, kept=None, stream=None):
    """Returns (Hq, Hs, kept): silu(A) U in 8 bits, and the checkpoint (Aq, As, Uq, Us) of A and U
    that q8_swiglu_backward reads (None with keep=False).  H: a pair (Hq, Hs) to write."""
    dev, dt = A.device, torch_dtype(plan.dtype)
    _expect(A, "A", (plan.N, plan.H), dt, dev)
    _expect(U, "U", (plan.N, plan.H), dt, dev)
    with _on(dev, stream):
        Hq, Hs = _out_q8(plan, *(H or (None, None)), "H", dev)
        if keep or kept is not None:
            kept = kept or (None,) * 4
            kept = _out_q8(plan, *kept[:2], "A", dev) + _out_q8(plan, *kept[2:], "U", dev)
        _check(lib().q8_swiglu_forward(ctypes.byref(plan), _ptr(A), _ptr(U), _ptr(Hq), _ptr(Hs),
                                       *(map(_ptr, kept or (None,) * 4)), _stream(dev, None)),
               "q8_swiglu_forward")
    return Hq, Hs, kept


def q8_swiglu_backward(plan: Q8Plan, kept, dH, dA=None, dU=None, stream=None):
    """Returns (dA, dU) [N, H] at the checkpoint's values."""
    dev, dt = dH.device, torch_dtype(plan.dtype)
    Aq, As, Uq, Us = kept
    _expect_q8(plan, Aq, As, "A", dev)
    _expect_q8(plan, Uq, Us, "U", dev)
    _expect(dH, "dH", (plan.N, plan.H), dt, dev)
    with _on(dev, stream):
        dA = _out(dA, "dA", (plan.N, plan.H), dt, dev)
        dU = _out(dU, "dU", (plan.N, plan.H), dt, dev)
        _check(lib().q8_swiglu_backward(ctypes.byref(plan), _ptr(Aq), _ptr(As), _ptr(Uq), _ptr(Us),
                                        _ptr(dH), _ptr(dA), _ptr(dU), _stream(dev, None)),
               "q8_swiglu_backward")
    return dA, dU


# ---- products grouped by expert


def gmm_plan(R: int, K: int, N: int, E: int, operands: int = GMM_BF16) -> GmmPlan:
    plan = GmmPlan()
    _check(lib().gmm_plan(R, K, N, E, operands, ctypes.byref(plan)), "gmm_plan")
    return plan


def _gmm_offsets(plan, offsets, dev):
    if offsets is None:
        if plan.E != 1:
            raise ValueError("offsets are required where there is more than one expert")
    else:
        _expect(offsets, "offsets", (plan.E + 1,), torch.int32, dev)


def _gmm_call(name, plan, kind, tensors, offsets, out, more, ws, dev):
    needed = plan.fwd_workspace_bytes if kind == "fwd" else plan.bwd_workspace_bytes
    ws, ws_bytes = _workspace(ws, plan, kind, dev) if needed or ws is not None else (None, 0)
    _check(getattr(lib(), name)(ctypes.byref(plan), *map(_ptr, tensors), _ptr(offsets), _ptr(out),
                                *more, _ptr(ws), ws_bytes, _stream(dev, None)), name)
    return out


def gmm_forward(plan: GmmPlan, X, W, offsets=None, Y=None, ws=None, stream=None):
    """Returns Y [R, N]: rows offsets[e] to offsets[e + 1] of X [R, K] times W[e] [K, N] (rows of no
    expert are left as they are).  offsets None, with one expert: all rows."""
    dev, bf = X.device, torch.bfloat16
    R, K, N, E = plan.R, plan.K, plan.N, plan.E
    _expect(X, "X", (R, K), bf, dev)
    _expect(W, "W", (E, K, N), bf, dev)
    _gmm_offsets(plan, offsets, dev)
    with _on(dev, stream):
        Y = _out(Y, "Y", (R, N), bf, dev)
        return _gmm_call("gmm_forward", plan, "fwd", (X, W), offsets, Y, (), ws, dev)


def gmm_backward_dx(plan: GmmPlan, dY, W, offsets=None, dX=None, ws=None, stream=None):
    """Returns dX [R, K] = dY [R, N] W[e]^T."""
    dev, bf = dY.device, torch.bfloat16
    R, K, N, E = plan.R, plan.K, plan.N, plan.E
    _expect(dY, "dY", (R, N), bf, dev)
    _expect(W, "W", (E, K, N), bf, dev)
    _gmm_offsets(plan, offsets, dev)
    with _on(dev, stream):
        dX = _out(dX, "dX", (R, K), bf, dev)
        return _gmm_call("gmm_backward_dx", plan, "fwd", (dY, W), offsets, dX, (), ws, dev)


def gmm_backward_dw(plan: GmmPlan, X, dY, offsets=None, dW=None, accumulate=False, ws=None,
                    stream=None):
    """Returns dW [E, K, N] fp32 = X_e^T dY_e, added to the dW given with accumulate."""
    dev, bf = X.device, torch.bfloat16
    R, K, N, E = plan.R, plan.K, plan.N, plan.E
    _expect(X, "X", (R, K), bf, dev)
    _expect(dY, "dY", (R, N), bf, dev)
    _gmm_offsets(plan, offsets, dev)
    if accumulate and dW is None:
        raise ValueError("accumulate needs the dW to add to")
    with _on(dev, stream):
        dW = _out(dW, "dW", (E, K, N), torch.float32, dev)
        return _gmm_call("gmm_backward_dw", plan, "bwd", (X, dY), offsets, dW, (int(accumulate),), ws, dev)


def _expect_gmm8_rows(plan, Xq, Xs, dev):
    _expect(Xq, "Xq", (plan.R, plan.row_pitch), E4M3, dev)
    _expect(Xs, "Xs", (plan.R, -(-plan.K // 512) * 4), E8M0, dev)


def gmm8_forward(plan: GmmPlan, Xq, Xs, Wq, Ws, offsets=None, Y=None, ws=None, stream=None):
    """Returns Y [R, N] bfloat16 from rows in 8 bits (q8_pack) and weights in 8 bits along K
    (q8_pack_weights(W, "K")).  Sums of more than four rows are off by up to GMM8_CUT of their
    products' magnitudes."""
    dev = Xq.device
    R, K, N, E = plan.R, plan.K, plan.N, plan.E
    _expect_gmm8_rows(plan, Xq, Xs, dev)
    _expect(Wq, "Wq", (E, N, plan.row_pitch), E4M3, dev)
    _expect(Ws, "Ws", (E, -(-N // 128), -(-K // 512) * 4), E8M0, dev)
    _gmm_offsets(plan, offsets, dev)
    with _on(dev, stream):
        Y = _out(Y, "Y", (R, N), torch.bfloat16, dev)
        return _gmm_call("gmm8_forward", plan, "fwd", (Xq, Xs, Wq, Ws), offsets, Y, (), ws, dev)


def gmm8_backward_dw(plan: GmmPlan, Xq, Xs, dY, offsets=None, dW=None, accumulate=False, ws=None,
                     stream=None):
    """Returns dW [E, K, N] fp32 from X in 8 bits and dY bfloat16, added to the dW given with
    accumulate."""
    dev = Xq.device
    R, K, N, E = plan.R, plan.K, plan.N, plan.E
    _expect_gmm8_rows(plan, Xq, Xs, dev)
    _expect(dY, "dY", (R, N), torch.bfloat16, dev)
    _gmm_offsets(plan, offsets, dev)
    if accumulate and dW is None:
        raise ValueError("accumulate needs the dW to add to")
    with _on(dev, stream):
        dW = _out(dW, "dW", (E, K, N), torch.float32, dev)
        return _gmm_call("gmm8_backward_dw", plan, "bwd", (Xq, Xs, dY), offsets, dW, (int(accumulate),), ws, dev)
