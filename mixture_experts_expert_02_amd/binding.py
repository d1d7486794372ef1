"""ctypes binding of libmoe_experts.so (include/moe_experts.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the hipStream_t. Every step of the computation runs in the HIP
library; if the library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import math
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
                ("ld_as", ctypes.c_int64), ("ldo", ctypes.c_int64), ("ld_add", ctypes.c_int64)]


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
# over, and run on the current stream of the tensors' own device.
class NormOut(NamedTuple):
    """add_rmsnorm's results; what was not asked for is None."""
    y: Optional[torch.Tensor]
    residual: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def _need(ok: bool, where: str, what: str, status: int = MOE_EINVAL):
    if not ok:
        raise MoeError(status, f"{where}: {what}")


def _rows2d(t, where: str, name: str, shape, dtypes, device) -> None:
    """t is a matrix of the given shape (None: any) with contiguous rows, on `device`."""
    _need(isinstance(t, torch.Tensor) and t.dim() == 2, where, f"{name} must be a matrix")
    _need(t.device == device and t.is_cuda, where, f"{name} must be on the GPU of the other tensors")
    _need(t.dtype in dtypes, where, f"{name} has type {t.dtype}")
    _need(tuple(t.shape) == tuple(shape), where, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    r, c = t.shape
    _need((c < 2 or t.stride(1) == 1) and (r < 2 or t.stride(0) >= c), where, f"{name} needs contiguous rows")


def _vector(t, where: str, name: str, n: int, dtypes, device) -> None:
    _need(isinstance(t, torch.Tensor) and tuple(t.shape) == (n,) and t.is_contiguous(), where,
          f"{name} must be a contiguous vector of {n} values")
    _need(t.device == device, where, f"{name} must be on the GPU of the other tensors")
    _need(t.dtype in dtypes, where, f"{name} has type {t.dtype}")


def _ld(t) -> int:
    """Elements between the rows of a matrix (0, contiguous, where it has one row or none)."""
    return t.stride(0) if t.shape[0] > 1 else 0


def _addr(t):
    return None if t is None else t.data_ptr()


def _run(fn, where: str, device, *args) -> None:
    if device.index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != MOE_OK:
        raise MoeError(rc, where)


_U8 = (torch.uint8,)
_F32 = (torch.float32,)


def _code_cols(fmt: int, K: int) -> int:
    return K // 2 if fmt == MOE_MX_FP4 else K


def _mx_fmt(fmt, where: str) -> int:
    _need(fmt in _MX, where, f"unknown format {fmt!r}")
    return _MX[fmt]


def _mx_out(codes, scales, where: str, rows: int, K: int, fmt: int, device):
    """The given code and scale tensors, checked, or new ones."""
    _need(K % 32 == 0, where, "rows of a multiple of 32 values are needed", MOE_ENOTSUP)
    if codes is None:
        codes = torch.empty(rows, _code_cols(fmt, K), dtype=torch.uint8, device=device)
    else:
        _rows2d(codes, where, "codes", (rows, _code_cols(fmt, K)), _U8, device)
    if scales is None:
        scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=device)
    else:
        _rows2d(scales, where, "scales", (rows, K // 32), _U8, device)
    return codes, scales


def mx_quantize(x, fmt: str = "mxfp4", codes=None, scales=None):
    """x [rows, K] (bf16, float16 or float32; rows may be strided) as microscaled
    rows: (codes uint8 [rows, K/2] for "mxfp4" or [rows, K] for "mxfp8", scales
    uint8 [rows, K/32]). See moe_mx_quantize."""
    where = "mx_quantize"
    f = _mx_fmt(fmt, where)
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, where, "x must be a matrix")
    rows, K = x.shape
    _rows2d(x, where, "x", (rows, K), _TYPE, x.device)
    codes, scales = _mx_out(codes, scales, where, rows, K, f, x.device)
    p = MoeMxRows(rows, K, _TYPE[x.dtype], f, _ld(x), _ld(codes), _ld(scales))
    _run(lib().moe_mx_quantize, "moe_mx_quantize", x.device, ctypes.byref(p), _addr(x), _addr(codes), _addr(scales))
    return codes, scales


def mx_dequantize(codes, scales, fmt: str = "mxfp4", dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """The values that microscaled rows stand for, [rows, K]. See moe_mx_dequantize."""
    where = "mx_dequantize"
    f = _mx_fmt(fmt, where)
    _need(isinstance(codes, torch.Tensor) and codes.dim() == 2, where, "codes must be a matrix")
    rows = codes.shape[0]
    K = codes.shape[1] * (2 if f == MOE_MX_FP4 else 1)
    dev = codes.device
    _need(scales is not None, where, "scales are needed")
    _mx_out(codes, scales, where, rows, K, f, dev)
    if out is None:
        _need(dtype in _TYPE, where, f"unsupported type {dtype}", MOE_ENOTSUP)
        out = torch.empty(rows, K, dtype=dtype, device=dev)
    else:
        _rows2d(out, where, "out", (rows, K), _TYPE, dev)
    p = MoeMxRows(rows, K, _TYPE[out.dtype], f, _ld(out), _ld(codes), _ld(scales))
    _run(lib().moe_mx_dequantize, "moe_mx_dequantize", dev, ctypes.byref(p), _addr(codes), _addr(scales), _addr(out))
    return out


def add_rmsnorm(x, weight, residual=None, eps: float = 1e-6, want_y: bool = True, mx: Optional[str] = None,
                residual_out=None, y=None, codes=None, scales=None) -> NormOut:
    """h = x + residual (stored in residual_out), y = h * weight / rms(h); y in
    x's type (unless want_y is false) and, with mx "mxfp8" or "mxfp4", as
    microscaled rows. See moe_add_rmsnorm."""
    where = "add_rmsnorm"
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, where, "x must be a matrix")
    T, H = x.shape
    dev = x.device
    _rows2d(x, where, "x", (T, H), _TYPE, dev)
    _vector(weight, where, "weight", H, _TYPE, dev)
    same = (x.dtype,)
    f = MOE_MX_NONE if mx is None else _mx_fmt(mx, where)
    _need(want_y or y is not None or f != MOE_MX_NONE, where, "no output asked for")
    _need(f != MOE_MX_NONE or (codes is None and scales is None), where, "codes and scales need mx")
    if residual is None:
        _need(residual_out is None, where, "residual_out needs residual")
    else:
        _rows2d(residual, where, "residual", (T, H), same, dev)
        if residual_out is None:
            residual_out = torch.empty(T, H, dtype=x.dtype, device=dev)
        else:
            _rows2d(residual_out, where, "residual_out", (T, H), same, dev)
    if y is not None:
        _rows2d(y, where, "y", (T, H), same, dev)
    elif want_y:
        y = torch.empty(T, H, dtype=x.dtype, device=dev)
    if f != MOE_MX_NONE:
        codes, scales = _mx_out(codes, scales, where, T, H, f, dev)
    ld = lambda t: 0 if t is None else _ld(t)  # noqa: E731
    p = MoeNormProblem(T, H, _TYPE[x.dtype], _TYPE[weight.dtype], f, eps, _ld(x), ld(residual), ld(residual_out),
                       ld(y), ld(codes), ld(scales))
    _run(lib().moe_add_rmsnorm, "moe_add_rmsnorm", dev, ctypes.byref(p), _addr(x), _addr(residual), _addr(weight),
         _addr(residual_out), _addr(y), _addr(codes), _addr(scales))
    return NormOut(y, residual_out, codes, scales)


def mx_linear(a, a_scales, w, w_scales, a_fmt: str = "mxfp8", bias=None, add=None, alpha: float = 1.0,
              dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """alpha * a w^T + bias + add for microscaled rows a (codes uint8 [M, K] for
    "mxfp8" or [M, K/2] for "mxfp4", scales [M, K/32]) and MXFP4 weights w (codes
    [N, K/2], scales [N, K/32], contiguous); add and out are [M, N] of one type
    (out may be add). See moe_mx_linear."""
    where = "mx_linear"
    f = _mx_fmt(a_fmt, where)
    _need(isinstance(w, torch.Tensor) and w.dim() == 2, where, "w must be a matrix")
    _need(isinstance(a, torch.Tensor) and a.dim() == 2, where, "a must be a matrix")
    dev = a.device
    N, K = w.shape[0], 2 * w.shape[1]
    M = a.shape[0]
    _need(K % 32 == 0, where, "rows of a multiple of 32 values are needed", MOE_ENOTSUP)
    _rows2d(a, where, "a", (M, _code_cols(f, K)), _U8, dev)
    _rows2d(a_scales, where, "a_scales", (M, K // 32), _U8, dev)
    _rows2d(w, where, "w", (N, K // 2), _U8, dev)
    _rows2d(w_scales, where, "w_scales", (N, K // 32), _U8, dev)
    _need(w.is_contiguous() and w_scales.is_contiguous(), where, "w and w_scales must be contiguous")
    if bias is not None:
        _vector(bias, where, "bias", N, _F32, dev)
    if out is not None:
        _rows2d(out, where, "out", (M, N), _TYPE, dev)
        dtype = out.dtype
    _need(dtype in _TYPE, where, f"unsupported type {dtype}", MOE_ENOTSUP)
    if add is not None:
        _rows2d(add, where, "add", (M, N), (dtype,), dev)
    if out is None:
        out = torch.empty(M, N, dtype=dtype, device=dev)
    p = MoeMxLinearProblem(M, N, K, f, _TYPE[dtype], alpha, _ld(a), _ld(a_scales), _ld(out),
                           0 if add is None else _ld(add))
    _run(lib().moe_mx_linear, "moe_mx_linear", dev, ctypes.byref(p), _addr(a), _addr(a_scales), _addr(w),
         _addr(w_scales), _addr(bias), _addr(add), _addr(out))
    return out


def route_topk(logits, k: int, score: str = "softmax", bias=None, n_group: int = 0, topk_group: int = 0,
               group_score: str = "top2", renormalize: bool = True, routed_scaling_factor: float = 1.0, ids=None,
               weights=None):
    """Top-k experts of logits [T, E] (bf16, float16 or float32; rows may be
    strided): (ids int32 [T, k], weights float32 [T, k]). See moe_route_topk."""
    where = "route_topk"
    _need(isinstance(logits, torch.Tensor) and logits.dim() == 2, where, "logits must be a matrix")
    T, E = logits.shape
    dev = logits.device
    _rows2d(logits, where, "logits", (T, E), _TYPE, dev)
    _need(score in _SCORE, where, f"unknown score {score!r}")
    _need(group_score in _GROUP, where, f"unknown group score {group_score!r}")
    if bias is not None:
        _vector(bias, where, "bias", E, _F32, dev)
    _need(isinstance(k, int) and k > 0, where, "k must be a positive integer")
    if ids is None:
        ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    else:
        _rows2d(ids, where, "ids", (T, k), (torch.int32,), dev)
        _need(ids.is_contiguous(), where, "ids must be contiguous")
    if weights is None:
        weights = torch.empty(T, k, dtype=torch.float32, device=dev)
    else:
        _rows2d(weights, where, "weights", (T, k), _F32, dev)
        _need(weights.is_contiguous(), where, "weights must be contiguous")
    p = MoeRouteTopkProblem(T, E, k, _TYPE[logits.dtype], _SCORE[score], n_group, topk_group, _GROUP[group_score],
                            int(bool(renormalize)), routed_scaling_factor, _ld(logits))
    _run(lib().moe_route_topk, "moe_route_topk", dev, ctypes.byref(p), _addr(logits), _addr(bias), _addr(ids),
         _addr(weights))
    return ids, weights
