"""Float64 CPU oracle of the operators around the experts step (test
infrastructure only): microscaled rows, row norm, dense MXFP4 product, general
routing.

Sources: the vLLM page "trtllm_mxfp4_moe" names the formats (MXFP4 weights,
MXFP8 activations) and the routing parameters (correction bias, expert groups,
groups kept, routed scaling factor); it prints no formulas, so parity is
unpinned for the formulas and the pins check these readings (OCP Microscaling
v1.0 for the blocks) against other formulations of them.
"""
from __future__ import annotations

import numpy as np

EMAX = {"mxfp4": 2, "mxfp8": 8}
TOP = {"mxfp4": 6.0, "mxfp8": 448.0}
MIN_EXP = {"mxfp4": 0, "mxfp8": -6}     # exponent of the smallest normal element
MANT = {"mxfp4": 1, "mxfp8": 3}         # mantissa bits


def element_spacing(v, fmt: str) -> np.ndarray:
    """Distance between neighbouring elements at |v| (below the largest element)."""
    _, ex = np.frexp(np.abs(np.asarray(v, np.float64)))
    return np.ldexp(1.0, (np.maximum(ex - 1, MIN_EXP[fmt]) - MANT[fmt]).astype(np.int32))


def element_round(v, fmt: str) -> np.ndarray:
    """Nearest element, ties to even, saturated."""
    v = np.clip(np.asarray(v, np.float64), -TOP[fmt], TOP[fmt])
    q = element_spacing(v, fmt)
    return np.round(v / q) * q


def mx_quantize(x, fmt: str):
    """(values, elements, scale codes) of x in blocks of 32 along the last
    axis. A block with a non-finite value: code 255, elements 0, values NaN."""
    x = np.asarray(x, np.float64)
    blk = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(blk).all(-1)
    blk = np.where(bad[..., None], 0.0, blk)
    top = np.abs(blk).max(-1)
    _, ex = np.frexp(top)
    code = np.where(top > 0, np.clip(ex - 1 - EMAX[fmt] + 127, 0, 254), 0)
    X = np.ldexp(1.0, (code - 127).astype(np.int32))[..., None]
    elem = element_round(blk / X, fmt)
    vals = np.where(bad[..., None], np.nan, elem * X)
    code = np.where(bad, 255, code).astype(np.uint8)
    return vals.reshape(x.shape), elem.reshape(x.shape), code


E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values() -> np.ndarray:
    """The 256 e4m3 values by code (NaN at 0x7f and 0xff)."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.ldexp(1.0, (e - 10).astype(np.int32)))
    v[127] = np.nan
    return np.concatenate([v, -v])


def mx_values(codes, scales, fmt: str) -> np.ndarray:
    """The float64 values of microscaled rows (codes and scales as bytes)."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8)
    if fmt == "mxfp4":
        e = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(codes.shape[0], -1)
    else:
        e = e4m3_values()[codes]
    X = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int32) - 127))
    return (e.reshape(e.shape[0], -1, 32) * X[..., None]).reshape(e.shape)


def rmsnorm(h, w, eps: float) -> np.ndarray:
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def mx_linear(a, w, bias=None, add=None, alpha: float = 1.0) -> np.ndarray:
    """alpha a w^T + bias + add on dequantized operands."""
    y = alpha * (np.asarray(a, np.float64) @ np.asarray(w, np.float64).T)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    if add is not None:
        y = y + np.asarray(add, np.float64)
    return y


def _first(score: np.ndarray, k: int) -> np.ndarray:
    """Indices of the k largest per row, descending, ties to the lower index."""
    return np.argsort(-score, axis=-1, kind="stable")[:, :k]


def route_topk(logits, k: int, score: str = "softmax", bias=None, n_group: int = 0, topk_group: int = 0,
               group_score: str = "top2", renormalize: bool = True, routed_scaling_factor: float = 1.0):
    """(ids int32, weights float64). Scores are float64 rounded once to
    float32; selection and group scores are float32 sums of them, so that
    every decision is on float32 values."""
    fmax = np.float64(np.finfo(np.float32).max)
    x = np.asarray(logits, np.float64)
    x = np.clip(np.where(np.isnan(x), -fmax, x), -fmax, fmax)
    with np.errstate(over="ignore"):
        if score == "softmax":
            e = np.exp(x - x.max(-1, keepdims=True))
            s = (e / e.sum(-1, keepdims=True)).astype(np.float32)
        else:
            s = (1.0 / (1.0 + np.exp(-x))).astype(np.float32)
    sel = s if bias is None else s + np.asarray(bias, np.float32)
    T, E = s.shape
    if n_group > 1:
        by = sel.reshape(T, n_group, E // n_group)
        best = -np.sort(-by, axis=-1)
        of = best[..., 0] + best[..., 1] if group_score == "top2" else best[..., 0]
        keep = np.zeros((T, n_group), bool)
        np.put_along_axis(keep, _first(of, topk_group), True, axis=1)
        # a dropped group's experts come after every kept one, -infinity among them
        order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -sel, ~np.repeat(keep, E // n_group, axis=1)), axis=-1)
        ids = order[:, :k]
    else:
        ids = _first(sel, k)
    w = np.take_along_axis(s, ids, axis=1).astype(np.float64)
    if renormalize:
        tot = w.sum(-1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
    return ids.astype(np.int32), w * routed_scaling_factor
