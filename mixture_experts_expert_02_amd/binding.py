"""ctypes binding of libmoe_experts.so (include/moe_experts.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the hipStream_t. Every step of the computation runs in the HIP
library; if the library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
from typing import NamedTuple, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_experts.so")

MOE_OK, MOE_EINVAL, MOE_ENOTSUP, MOE_ENOSPC, MOE_EHIP, MOE_ETIMEDOUT = 0, -1, -2, -3, -4, -5
MOE_W_BF16, MOE_W_MXFP4 = 0, 1
MOE_ACT_SILU, MOE_ACT_SWIGLU_OAI, MOE_ACT_SITU = 0, 1, 2

_ACT = {"silu": MOE_ACT_SILU, "swiglu_oai": MOE_ACT_SWIGLU_OAI, "situ": MOE_ACT_SITU}
_WFMT = {"bf16": MOE_W_BF16, "mxfp4": MOE_W_MXFP4}
MOE_A_BF16, MOE_A_MXFP8 = 0, 1
_AFMT = {"bf16": MOE_A_BF16, "mxfp8": MOE_A_MXFP8}

EXPORTED = (
    "moe_experts_workspace_bytes", "moe_experts_workspace_layout", "moe_experts_forward",
    "moe_experts_forward_timed", "moe_align_workspace_bytes", "moe_align",
    "moe_experts_grouped_workspace_bytes", "moe_experts_forward_grouped", "moe_device_error",
    "moe_strerror", "moe_route", "moe_experts_forward_grouped_timed", "moe_experts_forward_noalloc",
    "moe_check_expert_params", "moe_mx_packed_bytes", "moe_mx_pack_weights", "moe_bf16_packed_bytes",
    "moe_bf16_pack_weights", "moe_mx_quantize", "moe_mx_dequantize", "moe_add_rmsnorm", "moe_mx_linear",
    "moe_route_topk",
)
MOE_ROUTE_RENORMALIZE, MOE_ROUTE_DEEPSEEK_V3 = 0, 1
_ROUTE = {"renormalize": MOE_ROUTE_RENORMALIZE, "deepseek_v3": MOE_ROUTE_DEEPSEEK_V3}
MOE_T_BF16, MOE_T_FP16, MOE_T_FP32 = 0, 1, 2
_TYPE = {torch.bfloat16: MOE_T_BF16, torch.float16: MOE_T_FP16, torch.float32: MOE_T_FP32}
MOE_MX_NONE, MOE_MX_FP4, MOE_MX_FP8 = 0, 1, 2
_MX = {"mxfp4": MOE_MX_FP4, "mxfp8": MOE_MX_FP8}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
_SCORE = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1
_GROUP = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}


class MoeProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("wfmt", ctypes.c_int32),
                ("act", ctypes.c_int32), ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("limit", ctypes.c_float), ("weight_on_input", ctypes.c_int32), ("a_fmt", ctypes.c_int32),
                ("alpha_e", ctypes.c_void_p), ("beta_e", ctypes.c_void_p), ("limit_e", ctypes.c_void_p),
                ("fc1_alpha", ctypes.c_void_p), ("fc2_alpha", ctypes.c_void_p), ("mx_packed", ctypes.c_void_p),
                ("bf16_packed", ctypes.c_void_p)]


class MoeRouteProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("method", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float)]


class MoeMxRows(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("K", ctypes.c_int32), ("type", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("ld", ctypes.c_int64), ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


class MoeNormProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("type", ctypes.c_int32), ("w_type", ctypes.c_int32),
                ("mx_fmt", ctypes.c_int32), ("eps", ctypes.c_float), ("ldx", ctypes.c_int64),
                ("ld_res", ctypes.c_int64), ("ld_res_out", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


class MoeMxLinearProblem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("a_fmt", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("alpha", ctypes.c_float), ("lda", ctypes.c_int64),
                ("ld_as", ctypes.c_int64), ("ldo", ctypes.c_int64), ("ld_add", ctypes.c_int64), ("exact", ctypes.c_int32)]


class MoeRouteTopkProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("type", ctypes.c_int32),
                ("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("ld", ctypes.c_int64)]


class MoeWsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("status", "counts", "cu_seqlens", "perm", "inv_perm", "w_sorted", "act", "y", "total",
                 "xq", "xq_rows", "aq", "single_launch", "mx_tiled", "aq_sc")]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        P = ctypes.POINTER(MoeProblem)
        L.moe_experts_workspace_bytes.argtypes = [P]
        L.moe_experts_workspace_bytes.restype = sz
        L.moe_experts_workspace_layout.argtypes = [P, ctypes.POINTER(MoeWsLayout)]
        L.moe_experts_workspace_layout.restype = ctypes.c_int
        fwd = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_experts_forward.argtypes = fwd
        L.moe_experts_forward.restype = ctypes.c_int
        L.moe_experts_forward_timed.argtypes = fwd + [ctypes.POINTER(vp), ctypes.c_int]
        L.moe_experts_forward_timed.restype = ctypes.c_int
        L.moe_experts_forward_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_experts_forward_noalloc.restype = ctypes.c_int
        L.moe_align_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_align_workspace_bytes.restype = sz
        L.moe_align.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_align.restype = ctypes.c_int
        L.moe_experts_grouped_workspace_bytes.argtypes = [P]
        L.moe_experts_grouped_workspace_bytes.restype = sz
        L.moe_experts_forward_grouped.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_experts_forward_grouped.restype = ctypes.c_int
        L.moe_experts_forward_grouped_timed.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                                        ctypes.POINTER(vp), ctypes.c_int]
        L.moe_experts_forward_grouped_timed.restype = ctypes.c_int
        L.moe_device_error.argtypes = [vp, ctypes.POINTER(i32)]
        L.moe_device_error.restype = ctypes.c_int
        L.moe_route.argtypes = [ctypes.POINTER(MoeRouteProblem), vp, vp, vp, vp, vp]
        L.moe_route.restype = ctypes.c_int
        fp = ctypes.POINTER(ctypes.c_float)
        L.moe_check_expert_params.argtypes = [P, fp, fp, fp, fp, fp]
        L.moe_check_expert_params.restype = ctypes.c_int
        L.moe_mx_packed_bytes.argtypes = [P]
        L.moe_mx_packed_bytes.restype = sz
        L.moe_mx_pack_weights.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_mx_pack_weights.restype = ctypes.c_int
        L.moe_bf16_packed_bytes.argtypes = [P]
        L.moe_bf16_packed_bytes.restype = sz
        L.moe_bf16_pack_weights.argtypes = [P, vp, vp, vp, vp, sz, vp]
        L.moe_bf16_pack_weights.restype = ctypes.c_int
        L.moe_mx_quantize.argtypes = [ctypes.POINTER(MoeMxRows), vp, vp, vp, vp]
        L.moe_mx_quantize.restype = ctypes.c_int
        L.moe_mx_dequantize.argtypes = [ctypes.POINTER(MoeMxRows), vp, vp, vp, vp]
        L.moe_mx_dequantize.restype = ctypes.c_int
        L.moe_add_rmsnorm.argtypes = [ctypes.POINTER(MoeNormProblem), vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_add_rmsnorm.restype = ctypes.c_int
        L.moe_mx_linear.argtypes = [ctypes.POINTER(MoeMxLinearProblem), vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_mx_linear.restype = ctypes.c_int
        L.moe_route_topk.argtypes = [ctypes.POINTER(MoeRouteTopkProblem), vp, vp, vp, vp, vp]
        L.moe_route_topk.restype = ctypes.c_int
        L.moe_strerror.argtypes = [ctypes.c_int]
        L.moe_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().moe_strerror(status).decode()


EXPERT_PARAMS = ("alpha_e", "beta_e", "limit_e", "fc1_alpha", "fc2_alpha")


def problem(T, H, I, E, k=1, wfmt="bf16", act="silu", alpha=1.0, beta=0.0, limit=math.inf,
            weight_on_input=False, act_fmt="bf16", expert_params=None) -> MoeProblem:
    """expert_params: optional dict from EXPERT_PARAMS names to device float32
    tensors of E values (their pointers go into the problem)."""
    p = MoeProblem(int(T), int(H), int(I), int(E), int(k), _WFMT[wfmt] if isinstance(wfmt, str) else int(wfmt),
                   _ACT[act] if isinstance(act, str) else int(act), float(alpha), float(beta), float(limit),
                   int(weight_on_input), _AFMT[act_fmt] if isinstance(act_fmt, str) else int(act_fmt))
    for name, t in (expert_params or {}).items():
        if name not in EXPERT_PARAMS:
            raise KeyError(name)
        setattr(p, name, None if t is None else t.data_ptr())
    return p


def moe_check_expert_params(p: MoeProblem, alpha_e=None, beta_e=None, limit_e=None, fc1_alpha=None,
                            fc2_alpha=None) -> int:
    """Host-side check; each argument None or a sequence / CPU tensor of p.E floats."""
    keep = []

    def arr(v):
        if v is None:
            return None
        a = (ctypes.c_float * p.E)(*[float(x) for x in (v.tolist() if hasattr(v, "tolist") else v)])
        keep.append(a)
        return ctypes.cast(a, ctypes.POINTER(ctypes.c_float))

    return lib().moe_check_expert_params(ctypes.byref(p), arr(alpha_e), arr(beta_e), arr(limit_e), arr(fc1_alpha),
                                         arr(fc2_alpha))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


# ---------------------------------------------------------------- C ABI, same names
def moe_experts_workspace_bytes(p: MoeProblem) -> int:
    return lib().moe_experts_workspace_bytes(ctypes.byref(p))


def moe_experts_workspace_layout(p: MoeProblem) -> MoeWsLayout:
    lay = MoeWsLayout()
    _check(lib().moe_experts_workspace_layout(ctypes.byref(p), ctypes.byref(lay)), "moe_experts_workspace_layout")
    return lay


def moe_mx_packed_bytes(p: MoeProblem) -> int:
    return lib().moe_mx_packed_bytes(ctypes.byref(p))


def moe_mx_pack_weights(p: MoeProblem, w_gate, w_up, w_down, s_gate, s_up, s_down, packed, stream=None) -> int:
    return lib().moe_mx_pack_weights(ctypes.byref(p), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate),
                                     _ptr(s_up), _ptr(s_down), _ptr(packed), packed.numel() * packed.element_size(),
                                     _stream(stream))


def mx_pack_weights(p: MoeProblem, w_gate, w_up, w_down, s_gate, s_up, s_down, stream=None) -> torch.Tensor:
    """Packed weights of problem p (a new uint8 device tensor); set p.mx_packed to its pointer."""
    n = moe_mx_packed_bytes(p)
    if n == 0:
        raise MoeError(MOE_EINVAL, "moe_mx_packed_bytes")
    packed = torch.empty(n, dtype=torch.uint8, device=w_gate.device)
    _check(moe_mx_pack_weights(p, w_gate, w_up, w_down, s_gate, s_up, s_down, packed, stream=stream),
           "moe_mx_pack_weights")
    return packed


def moe_bf16_packed_bytes(p: MoeProblem) -> int:
    return lib().moe_bf16_packed_bytes(ctypes.byref(p))


def moe_bf16_pack_weights(p: MoeProblem, w_gate, w_up, w_down, packed, stream=None) -> int:
    return lib().moe_bf16_pack_weights(ctypes.byref(p), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(packed),
                                       packed.numel() * packed.element_size(), _stream(stream))


def bf16_pack_weights(p: MoeProblem, w_gate, w_up, w_down, stream=None) -> torch.Tensor:
    """Operand-block weights of problem p (a new uint8 device tensor); set p.bf16_packed to its pointer."""
    n = moe_bf16_packed_bytes(p)
    if n == 0:
        raise MoeError(MOE_EINVAL, "moe_bf16_packed_bytes")
    packed = torch.empty(n, dtype=torch.uint8, device=w_gate.device)
    _check(moe_bf16_pack_weights(p, w_gate, w_up, w_down, packed, stream=stream), "moe_bf16_pack_weights")
    return packed


def moe_experts_forward(p: MoeProblem, x, topk_ids, topk_weights, w_gate, w_up, w_down, s_gate, s_up, s_down,
                        out, workspace, stream=None) -> int:
    return lib().moe_experts_forward(ctypes.byref(p), _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(w_gate),
                                     _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(out),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream))


def moe_experts_forward_timed(p: MoeProblem, x, topk_ids, topk_weights, w_gate, w_up, w_down, s_gate, s_up,
                              s_down, out, workspace, events: Sequence[int], stream=None) -> int:
    arr = (ctypes.c_void_p * len(events))(*events)
    return lib().moe_experts_forward_timed(ctypes.byref(p), _ptr(x), _ptr(topk_ids), _ptr(topk_weights),
                                           _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up),
                                           _ptr(s_down), _ptr(out), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream), arr,
                                           len(events))


def moe_experts_forward_noalloc(p: MoeProblem, x, topk_ids, topk_weights, w_gate, w_up, w_down, s_gate, s_up,
                                s_down, out, stream=None) -> int:
    return lib().moe_experts_forward_noalloc(ctypes.byref(p), _ptr(x), _ptr(topk_ids), _ptr(topk_weights),
                                             _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up),
                                             _ptr(s_down), _ptr(out), _stream(stream))


def moe_align_workspace_bytes(T: int, k: int, E: int) -> int:
    return lib().moe_align_workspace_bytes(T, k, E)


def moe_align(topk_ids, T, k, E, counts, cu_seqlens, perm, inv_perm, workspace, stream=None) -> int:
    return lib().moe_align(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(cu_seqlens), _ptr(perm), _ptr(inv_perm),
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))


def moe_experts_grouped_workspace_bytes(p: MoeProblem) -> int:
    return lib().moe_experts_grouped_workspace_bytes(ctypes.byref(p))


def moe_experts_forward_grouped(p: MoeProblem, x_nvs, cu_seqlens, route_w, w_gate, w_up, w_down, s_gate, s_up,
                                s_down, out_nvs, workspace, stream=None) -> int:
    return lib().moe_experts_forward_grouped(ctypes.byref(p), _ptr(x_nvs), _ptr(cu_seqlens), _ptr(route_w),
                                             _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up),
                                             _ptr(s_down), _ptr(out_nvs), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream))


def moe_experts_forward_grouped_timed(p: MoeProblem, x_nvs, cu_seqlens, route_w, w_gate, w_up, w_down, s_gate,
                                      s_up, s_down, out_nvs, workspace, events: Sequence[int], stream=None) -> int:
    arr = (ctypes.c_void_p * len(events))(*events)
    return lib().moe_experts_forward_grouped_timed(ctypes.byref(p), _ptr(x_nvs), _ptr(cu_seqlens), _ptr(route_w),
                                                   _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate),
                                                   _ptr(s_up), _ptr(s_down), _ptr(out_nvs), _ptr(workspace),
                                                   workspace.numel() * workspace.element_size(), _stream(stream),
                                                   arr, len(events))


def moe_device_error(workspace) -> int:
    n = ctypes.c_int32(0)
    _check(lib().moe_device_error(_ptr(workspace), ctypes.byref(n)), "moe_device_error")
    return n.value


def moe_strerror(status: int) -> str:
    return strerror(status)


def moe_route(p: MoeRouteProblem, logits, bias, topk_ids, topk_weights, stream=None) -> int:
    return lib().moe_route(ctypes.byref(p), _ptr(logits), _ptr(bias), _ptr(topk_ids), _ptr(topk_weights),
                           _stream(stream))


def moe_mx_quantize(p: MoeMxRows, x, codes, scales, stream=None) -> int:
    return lib().moe_mx_quantize(ctypes.byref(p), _ptr(x), _ptr(codes), _ptr(scales), _stream(stream))


def moe_mx_dequantize(p: MoeMxRows, codes, scales, out, stream=None) -> int:
    return lib().moe_mx_dequantize(ctypes.byref(p), _ptr(codes), _ptr(scales), _ptr(out), _stream(stream))


def moe_add_rmsnorm(p: MoeNormProblem, x, residual, weight, residual_out, y, codes, scales, stream=None) -> int:
    return lib().moe_add_rmsnorm(ctypes.byref(p), _ptr(x), _ptr(residual), _ptr(weight), _ptr(residual_out), _ptr(y),
                                 _ptr(codes), _ptr(scales), _stream(stream))


def moe_mx_linear(p: MoeMxLinearProblem, a, a_scales, w, w_scales, bias, add, out, stream=None) -> int:
    return lib().moe_mx_linear(ctypes.byref(p), _ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), _ptr(bias),
                               _ptr(add), _ptr(out), _stream(stream))


def moe_route_topk(p: MoeRouteTopkProblem, logits, bias, topk_ids, topk_weights, stream=None) -> int:
    return lib().moe_route_topk(ctypes.byref(p), _ptr(logits), _ptr(bias), _ptr(topk_ids), _ptr(topk_weights),
                                _stream(stream))


# ---------------------------------------------------------------- torch conveniences
def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A caller-owned workspace (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def experts_forward(x, topk_ids, topk_weights, w_gate, w_up, w_down, scales=None, act="silu", alpha=1.0, beta=0.0,
                    limit=math.inf, out=None, workspace=None, weight_on_input=False,
                    act_fmt="bf16", expert_params=None, mx_packed=None, bf16_packed=None) -> torch.Tensor:
    """Token-major experts step on torch tensors; allocates out/workspace if not given.
    mx_packed: the weights packed by mx_pack_weights (MXFP4 x MXFP8 only), or None.
    bf16_packed: the weights packed by bf16_pack_weights (bf16 only), or None."""
    T, H = x.shape
    k = topk_ids.shape[1]
    E = w_gate.shape[0]
    wfmt = "mxfp4" if w_gate.dtype == torch.uint8 else "bf16"
    I = w_gate.shape[1]
    p = problem(T, H, I, E, k, wfmt, act, alpha, beta, limit, weight_on_input, act_fmt, expert_params)
    if mx_packed is not None:
        p.mx_packed = mx_packed.data_ptr()
    if bf16_packed is not None:
        p.bf16_packed = bf16_packed.data_ptr()
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(moe_experts_workspace_bytes(p), x.device)
    sg, su, sd = scales if scales is not None else (None, None, None)
    _check(moe_experts_forward(p, x, topk_ids, topk_weights, w_gate, w_up, w_down, sg, su, sd, out, workspace),
           "moe_experts_forward")
    return out


def experts_forward_grouped(x_nvs, cu_seqlens, route_w, w_gate, w_up, w_down, scales=None, act="silu", alpha=1.0,
                            beta=0.0, limit=math.inf, out=None, workspace=None, weight_on_input=False,
                            act_fmt="bf16", expert_params=None, bf16_packed=None, mx_packed=None) -> torch.Tensor:
    """Pre-grouped experts step; bf16_packed / mx_packed: the weights packed by bf16_pack_weights /
    mx_pack_weights (for bf16 / MXFP4 weights), or None."""
    NvS, H = x_nvs.shape
    G = w_gate.shape[0]
    I = w_gate.shape[1]
    wfmt = "mxfp4" if w_gate.dtype == torch.uint8 else "bf16"
    p = problem(NvS, H, I, G, 1, wfmt, act, alpha, beta, limit, weight_on_input, act_fmt, expert_params)
    if bf16_packed is not None:
        p.bf16_packed = bf16_packed.data_ptr()
    if mx_packed is not None:
        p.mx_packed = mx_packed.data_ptr()
    if out is None:
        out = torch.empty(NvS, H, dtype=torch.bfloat16, device=x_nvs.device)
    if workspace is None:
        workspace = alloc_workspace(moe_experts_grouped_workspace_bytes(p), x_nvs.device)
    sg, su, sd = scales if scales is not None else (None, None, None)
    _check(moe_experts_forward_grouped(p, x_nvs, cu_seqlens, route_w, w_gate, w_up, w_down, sg, su, sd, out,
                                       workspace), "moe_experts_forward_grouped")
    return out


def route_problem(T, E, k, method="renormalize", n_group=0, topk_group=0,
                  routed_scaling_factor=1.0) -> MoeRouteProblem:
    return MoeRouteProblem(int(T), int(E), int(k), _ROUTE[method] if isinstance(method, str) else int(method),
                           int(n_group), int(topk_group), float(routed_scaling_factor))


def route(logits, k: int, method="renormalize", bias=None, n_group=0, topk_group=0, routed_scaling_factor=1.0,
          ids=None, weights=None):
    """moe_route on a float32 [T, E] tensor; returns (ids int32 [T, k], weights float32 [T, k])."""
    T, E = logits.shape
    dev = logits.device
    if ids is None:
        ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, k, dtype=torch.float32, device=dev)
    p = route_problem(T, E, k, method, n_group, topk_group, routed_scaling_factor)
    _check(moe_route(p, logits, bias, ids, weights), "moe_route")
    return ids, weights


def align(topk_ids, E: int, workspace=None):
    """moe_align on a torch int32 [T, k] tensor; returns (counts, cu_seqlens, perm, inv_perm)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    cu = torch.empty(E, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(moe_align_workspace_bytes(T, k, E), dev)
    _check(moe_align(topk_ids, T, k, E, counts, cu, perm, inv, workspace), "moe_align")
    return counts, cu, perm, inv, workspace


# ---------------------------------------------------------------- operators around the experts step
# These check every tensor against the problem before they hand its pointer
# over, and run on the current stream of the tensors' own device. The checks
# that pass are kept short: for a single token a call's host time is what counts.
class NormOut(NamedTuple):
    """add_rmsnorm's results; what was not asked for is None."""
    y: Optional[torch.Tensor]
    residual: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def _refuse(where: str, what: str, status: int = MOE_EINVAL):
    raise MoeError(status, f"{where}: {what}")


# Sizes are 32-bit in the problem structures, and ctypes keeps the low bits of a larger number.
_INT_MAX = 2 ** 31 - 1


def _size(n: int, where: str) -> int:
    if n > _INT_MAX:
        _refuse(where, f"a size of {n} is too large", MOE_ENOTSUP)
    return n


def _count(n, where: str, name: str) -> int:
    try:
        n = operator.index(n)
    except TypeError:
        _refuse(where, f"{name} must be an integer")
    if not -_INT_MAX <= n <= _INT_MAX:
        _refuse(where, f"{name} is out of range")
    return n


def _matrix(t, where: str, name: str):
    """(rows, columns, device index) of a GPU matrix."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(where, f"{name} must be a matrix")
    dev = t.get_device()
    if dev < 0:
        _refuse(where, f"{name} must be on a GPU")
    r, c = t.shape
    return _size(r, where), _size(c, where), dev


def _ld(t, shape, dtypes, dev: int, where: str, name: str) -> int:
    """Elements between the rows of t (0: contiguous), a matrix of the given
    shape and one of the types, with contiguous rows, on device dev."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.get_device() == dev:
        if t.is_contiguous():
            return 0
        r, c = shape
        if (c < 2 or t.stride(1) == 1) and (r < 2 or t.stride(0) >= c):
            return t.stride(0) if r > 1 else 0
        _refuse(where, f"{name} needs contiguous rows that do not overlap")
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        _refuse(where, f"{name} must have shape {tuple(shape)}, not {tuple(getattr(t, 'shape', ()))}")
    if t.get_device() != dev:
        _refuse(where, f"{name} must be on the GPU of the other tensors")
    _refuse(where, f"{name} has type {t.dtype}")


def _rows(t, where: str, name: str):
    """(rows, columns, device index, elements between rows) of a GPU matrix of values."""
    if isinstance(t, torch.Tensor) and t.dim() == 2 and t.dtype in _TYPE and t.is_contiguous():
        dev = t.get_device()
        r, c = t.shape
        if dev >= 0 and r <= _INT_MAX and c <= _INT_MAX:
            return r, c, dev, 0
    r, c, dev = _matrix(t, where, name)
    return r, c, dev, _ld(t, (r, c), _TYPE, dev, where, name)


def _vector(t, n: int, dtypes, dev: int, where: str, name: str) -> int:
    """Address of a contiguous vector of n values."""
    if not (isinstance(t, torch.Tensor) and t.shape == (n,) and t.is_contiguous()):
        _refuse(where, f"{name} must be a contiguous vector of {n} values")
    if t.get_device() != dev:
        _refuse(where, f"{name} must be on the GPU of the other tensors")
    if t.dtype not in dtypes:
        _refuse(where, f"{name} has type {t.dtype}")
    return t.data_ptr()


# The current stream's handle by device index, without building a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# The current device's index; whoever has a GPU tensor has initialised the runtime.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(fn, where: str, dev: int, *args) -> None:
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != MOE_OK:
        raise MoeError(rc, where)


_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _mx_fmt(fmt, where: str) -> int:
    f = _MX.get(fmt) if isinstance(fmt, str) else None
    if f is None:
        _refuse(where, f"unknown format {fmt!r}")
    return f


def _blocks(K: int, where: str) -> int:
    if K % 32:
        _refuse(where, "rows of a multiple of 32 values are needed", MOE_ENOTSUP)
    return _size(K, where) // 32


def _mx_out(like, codes, scales, rows: int, K: int, fmt: int, dev: int, where: str):
    """(codes, ld, scales, ld): the given code and scale tensors, checked, or new ones."""
    nb = _blocks(K, where)
    cols = K // 2 if fmt == MOE_MX_FP4 else K
    lc = ls = 0
    if codes is None:
        codes = like.new_empty(rows, cols, dtype=torch.uint8)
    else:
        lc = _ld(codes, (rows, cols), _U8, dev, where, "codes")
    if scales is None:
        scales = like.new_empty(rows, nb, dtype=torch.uint8)
    else:
        ls = _ld(scales, (rows, nb), _U8, dev, where, "scales")
    return codes, lc, scales, ls


def mx_quantize(x, fmt: str = "mxfp4", codes=None, scales=None):
    """x [rows, K] (bf16, float16 or float32; rows may be strided) as microscaled
    rows: (codes uint8 [rows, K/2] for "mxfp4" or [rows, K] for "mxfp8", scales
    uint8 [rows, K/32]). See moe_mx_quantize."""
    where = "mx_quantize"
    f = _mx_fmt(fmt, where)
    rows, K, dev, ld = _rows(x, where, "x")
    codes, lc, scales, ls = _mx_out(x, codes, scales, rows, K, f, dev, where)
    p = MoeMxRows(rows, K, _TYPE[x.dtype], f, ld, lc, ls)
    _run(lib().moe_mx_quantize, "moe_mx_quantize", dev, ctypes.byref(p), x.data_ptr(), codes.data_ptr(),
         scales.data_ptr())
    return codes, scales


def mx_dequantize(codes, scales, fmt: str = "mxfp4", dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """The values that microscaled rows stand for, [rows, K]. See moe_mx_dequantize."""
    where = "mx_dequantize"
    f = _mx_fmt(fmt, where)
    rows, cols, dev = _matrix(codes, where, "codes")
    K = 2 * cols if f == MOE_MX_FP4 else cols
    lc = _ld(codes, (rows, cols), _U8, dev, where, "codes")
    ls = _ld(scales, (rows, _blocks(K, where)), _U8, dev, where, "scales")
    ld = 0
    if out is None:
        if dtype not in _TYPE:
            _refuse(where, f"unsupported type {dtype}", MOE_ENOTSUP)
        out = codes.new_empty(rows, K, dtype=dtype)
    else:
        ld = _ld(out, (rows, K), _TYPE, dev, where, "out")
    p = MoeMxRows(rows, K, _TYPE[out.dtype], f, ld, lc, ls)
    _run(lib().moe_mx_dequantize, "moe_mx_dequantize", dev, ctypes.byref(p), codes.data_ptr(), scales.data_ptr(),
         out.data_ptr())
    return out


def add_rmsnorm(x, weight, residual=None, eps: float = 1e-6, want_y: bool = True, mx: Optional[str] = None,
                residual_out=None, y=None, codes=None, scales=None) -> NormOut:
    """h = x + residual (stored in residual_out), y = h * weight / rms(h); y in
    x's type (unless want_y is false) and, with mx "mxfp8" or "mxfp4", as
    microscaled rows. See moe_add_rmsnorm."""
    where = "add_rmsnorm"
    T, H, dev, ldx = _rows(x, where, "x")
    shape = (T, H)
    same = (x.dtype,)
    f = MOE_MX_NONE if mx is None else _mx_fmt(mx, where)
    if f == MOE_MX_NONE:
        if codes is not None or scales is not None:
            _refuse(where, "codes and scales need mx")
        if not want_y and y is None:
            _refuse(where, "no output asked for")
    ld_res = ld_out = ldy = lc = ls = 0
    res_ptr = out_ptr = y_ptr = c_ptr = s_ptr = None
    if residual is not None:
        ld_res = _ld(residual, shape, same, dev, where, "residual")
        res_ptr = residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty_like(x)
        else:
            ld_out = _ld(residual_out, shape, same, dev, where, "residual_out")
        out_ptr = residual_out.data_ptr()
    elif residual_out is not None:
        _refuse(where, "residual_out needs residual")
    if y is not None:
        ldy = _ld(y, shape, same, dev, where, "y")
        y_ptr = y.data_ptr()
    elif want_y:
        y = torch.empty_like(x)
        y_ptr = y.data_ptr()
    if f != MOE_MX_NONE:
        codes, lc, scales, ls = _mx_out(x, codes, scales, T, H, f, dev, where)
        c_ptr, s_ptr = codes.data_ptr(), scales.data_ptr()
    w_ptr = _vector(weight, H, _TYPE, dev, where, "weight")
    p = MoeNormProblem(T, H, _TYPE[x.dtype], _TYPE[weight.dtype], f, eps, ldx, ld_res, ld_out, ldy, lc, ls)
    _run(lib().moe_add_rmsnorm, "moe_add_rmsnorm", dev, ctypes.byref(p), x.data_ptr(), res_ptr, w_ptr, out_ptr, y_ptr,
         c_ptr, s_ptr)
    return NormOut(y, residual_out, codes, scales)


def mx_linear(a, a_scales, w, w_scales, a_fmt: str = "mxfp8", bias=None, add=None, alpha: float = 1.0,
              dtype=torch.bfloat16, out=None, exact: bool = False) -> torch.Tensor:
    """alpha * a w^T + bias + add for microscaled rows a (codes uint8 [M, K] for
    "mxfp8" or [M, K/2] for "mxfp4", scales [M, K/32]) and MXFP4 weights w (codes
    [N, K/2], scales [N, K/32], contiguous); add and out are [M, N] of one type
    (out may be add). exact: MXFP8 rows with 16-bit results also without the matrix
    instruction's cut of small products, in up to 2.2 times the time. See moe_mx_linear."""
    where = "mx_linear"
    f = _mx_fmt(a_fmt, where)
    lda = ld_as = 0
    # A call takes less time on the GPU than its checks take here, so the usual case (all
    # contiguous) is looked over in one expression; what fails it is checked one by one.
    try:
        (M, cols), (N, half), dev, u8 = a.shape, w.shape, a.get_device(), torch.uint8
        K, nb = 2 * half, half >> 4
        plain = (dev >= 0 and M | N | K <= _INT_MAX and cols == (half if f == MOE_MX_FP4 else K) and not half & 15
                 and a.dtype is u8 and w.dtype is u8 and a_scales.dtype is u8 and w_scales.dtype is u8
                 and a_scales.shape == (M, nb) and w_scales.shape == (N, nb)
                 and w.get_device() == dev and a_scales.get_device() == dev and w_scales.get_device() == dev
                 and a.is_contiguous() and w.is_contiguous() and a_scales.is_contiguous() and w_scales.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        plain = False
    if not plain:
        M, cols, dev = _matrix(a, where, "a")
        N, half, _ = _matrix(w, where, "w")
        K = 2 * half
        nb = _blocks(K, where)
        lda = _ld(a, (M, half if f == MOE_MX_FP4 else K), _U8, dev, where, "a")
        ld_as = _ld(a_scales, (M, nb), _U8, dev, where, "a_scales")
        if _ld(w, (N, half), _U8, dev, where, "w") or _ld(w_scales, (N, nb), _U8, dev, where, "w_scales"):
            _refuse(where, "w and w_scales must be contiguous")
    b_ptr = None if bias is None else _vector(bias, N, _F32, dev, where, "bias")
    ldo = ld_add = 0
    if out is not None:
        ldo = _ld(out, (M, N), _TYPE, dev, where, "out")
        dtype = out.dtype
    elif dtype not in _TYPE:
        _refuse(where, f"unsupported type {dtype}", MOE_ENOTSUP)
    add_ptr = None
    if add is not None:
        ld_add = _ld(add, (M, N), (dtype,), dev, where, "add")
        add_ptr = add.data_ptr()
    if out is None:
        out = a.new_empty(M, N, dtype=dtype)
    p = MoeMxLinearProblem(M, N, K, f, _TYPE[dtype], alpha, lda, ld_as, ldo, ld_add, 1 if exact else 0)
    _run(lib().moe_mx_linear, "moe_mx_linear", dev, ctypes.byref(p), a.data_ptr(), a_scales.data_ptr(), w.data_ptr(),
         w_scales.data_ptr(), b_ptr, add_ptr, out.data_ptr())
    return out


def route_topk(logits, k: int, score: str = "softmax", bias=None, n_group: int = 0, topk_group: int = 0,
               group_score: str = "top2", renormalize: bool = True, routed_scaling_factor: float = 1.0, ids=None,
               weights=None):
    """Top-k experts of logits [T, E] (bf16, float16 or float32; rows may be
    strided): (ids int32 [T, k], weights float32 [T, k]). See moe_route_topk."""
    where = "route_topk"
    T, E, dev, ld = _rows(logits, where, "logits")
    if score not in _SCORE:
        _refuse(where, f"unknown score {score!r}")
    if group_score not in _GROUP:
        _refuse(where, f"unknown group score {group_score!r}")
    if not isinstance(k, int) or not 0 < k <= _INT_MAX:
        _refuse(where, "k must be a positive integer")
    if n_group or topk_group:
        n_group, topk_group = _count(n_group, where, "n_group"), _count(topk_group, where, "topk_group")
    b_ptr = None if bias is None else _vector(bias, E, _F32, dev, where, "bias")
    if ids is None:
        ids = logits.new_empty(T, k, dtype=torch.int32)
    elif _ld(ids, (T, k), _I32, dev, where, "ids"):
        _refuse(where, "ids must be contiguous")
    if weights is None:
        weights = logits.new_empty(T, k, dtype=torch.float32)
    elif _ld(weights, (T, k), _F32, dev, where, "weights"):
        _refuse(where, "weights must be contiguous")
    p = MoeRouteTopkProblem(T, E, k, _TYPE[logits.dtype], _SCORE[score], n_group, topk_group, _GROUP[group_score],
                            1 if renormalize else 0, routed_scaling_factor, ld)
    _run(lib().moe_route_topk, "moe_route_topk", dev, ctypes.byref(p), logits.data_ptr(), b_ptr, ids.data_ptr(),
         weights.data_ptr())
    return ids, weights
