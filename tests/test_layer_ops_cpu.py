"""The operators around the experts step without a GPU: the oracle's readings
against other formulations of them, and every refusal of the C ABI and of the
Python entry points (checked before anything is enqueued)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
import oracle
from mixture_experts_expert_02_amd import binding as B
from oracle import layer_ops as L

HERE = os.path.dirname(os.path.abspath(__file__))


# ------------------------------------------------------------------ oracle
def test_oracle_e2m1_table_is_the_golden_one():
    rows = [l.split() for l in open(os.path.join(HERE, "golden", "e2m1_values.txt")) if l[0] != "#"]
    assert [float(v) for _, v in rows] == L.E2M1.tolist()


def test_oracle_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, L.e4m3_values(), equal_nan=True)


def test_oracle_mxfp8_is_the_experts_steps_rule():
    x = np.random.default_rng(1).standard_normal((7, 96)) * np.exp(np.random.default_rng(2).standard_normal((7, 1)) * 5)
    x[0, :32] = 0
    v, e, c = L.mx_quantize(x, "mxfp8")
    v2, e2, c2 = oracle.mxfp8_quantize(x)
    assert np.array_equal(v, v2) and np.array_equal(e, e2) and np.array_equal(c, c2)


def test_oracle_mxfp4_rounding_by_nearest_grid_point():
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    v = np.linspace(0, 7.9, 1600)
    v = np.concatenate([v, (grid[1:] + grid[:-1]) / 2])
    got = L.element_round(v, "mxfp4")
    for a, g in zip(v, got):
        d = np.abs(grid - min(a, 6.0))
        near = np.flatnonzero(d == d.min())
        want = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
        assert g == grid[want], a


def test_oracle_nan_block():
    x = np.ones((1, 64))
    x[0, 40] = np.inf
    v, e, c = L.mx_quantize(x, "mxfp4")
    assert c[0, 1] == 255 and np.isnan(v[0, 32:]).all() and (v[0, :32] == 1).all() and (e[0, 32:] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_oracle_values_of_codes(fmt):
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 256, (3, 32 if fmt == "mxfp4" else 64), dtype=np.uint8)
    sc = rng.integers(100, 140, (3, 2), dtype=np.uint8)
    v = L.mx_values(codes, sc, fmt)
    assert v.shape == (3, 64)
    one = codes[1, 20] >> 4 if fmt == "mxfp4" else codes[1, 41]
    want = L.E2M1[one] if fmt == "mxfp4" else L.e4m3_values()[one]
    assert np.array_equal(v[1, 41], want * 2.0 ** (int(sc[1, 1]) - 127), equal_nan=True)


def test_oracle_route_agrees_with_the_fixed_methods():
    rng = np.random.default_rng(4)
    l = rng.standard_normal((50, 64)).astype(np.float32)
    ids, w = L.route_topk(l, 6)
    rid, rw = oracle.route_renormalize(l, 6)
    assert np.array_equal(ids, rid)
    np.testing.assert_allclose(w, rw, rtol=1e-6)
    b = (0.1 * rng.standard_normal(64)).astype(np.float32)
    ids, w = L.route_topk(l, 6, "sigmoid", b, 8, 3, "top2", True, 2.5)
    rid, rw = oracle.route_deepseek_v3(l, 6, bias=b, n_group=8, topk_group=3, routed_scaling_factor=2.5)
    assert np.array_equal(ids, rid)
    np.testing.assert_allclose(w, rw, rtol=1e-6)


def test_oracle_route_max_groups_by_enumeration():
    rng = np.random.default_rng(5)
    l = rng.standard_normal((40, 12))
    ids, w = L.route_topk(l, 3, "softmax", None, 4, 2, "max", False, 1.0)
    p = np.exp(l) / np.exp(l).sum(-1, keepdims=True)
    for t in range(40):
        best = sorted(range(4), key=lambda g: -p[t, 3 * g: 3 * g + 3].max())[:2]
        cand = sorted((e for e in range(12) if e // 3 in best), key=lambda e: -p[t, e])[:3]
        assert ids[t].tolist() == cand
        np.testing.assert_allclose(w[t], p[t, cand], rtol=1e-6)


# ---------------------------------------------------------------- refusals
# Addresses that are never read: every call below is refused first.
OK = 4096


def rows(**kw):
    return B.MoeMxRows(**{**dict(rows=4, K=64, type=0, fmt=1), **kw})


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(rows=-1), (OK, OK, OK), B.MOE_EINVAL),
    (dict(K=0), (OK, OK, OK), B.MOE_EINVAL),
    (dict(type=3), (OK, OK, OK), B.MOE_EINVAL),
    (dict(type=-1), (OK, OK, OK), B.MOE_EINVAL),
    (dict(fmt=0), (OK, OK, OK), B.MOE_EINVAL),
    (dict(fmt=3), (OK, OK, OK), B.MOE_EINVAL),
    (dict(K=48), (OK, OK, OK), B.MOE_ENOTSUP),
    (dict(rows=1 << 30, K=1 << 10), (OK, OK, OK), B.MOE_ENOTSUP),
    (dict(ld=63), (OK, OK, OK), B.MOE_EINVAL),
    (dict(ld=-64), (OK, OK, OK), B.MOE_EINVAL),
    (dict(ld=68), (OK, OK, OK), B.MOE_ENOTSUP),         # rows 136 bytes apart
    (dict(ld_codes=16), (OK, OK, OK), B.MOE_EINVAL),
    (dict(ld_codes=40), (OK, OK, OK), B.MOE_ENOTSUP),
    (dict(ld_scales=1), (OK, OK, OK), B.MOE_EINVAL),
    ({}, (0, OK, OK), B.MOE_EINVAL),
    ({}, (OK, 0, OK), B.MOE_EINVAL),
    ({}, (OK, OK, 0), B.MOE_EINVAL),
    ({}, (OK + 2, OK, OK), B.MOE_EINVAL),
    ({}, (OK, OK + 4, OK), B.MOE_EINVAL),
    (dict(rows=0), (0, 0, 0), B.MOE_OK),
])
def test_mx_rows_refusals(kw, ptrs, code):
    p = rows(**kw)
    x, c, s = ptrs
    assert B.lib().moe_mx_quantize(ctypes.byref(p), x, c, s, 0) == code
    assert B.lib().moe_mx_dequantize(ctypes.byref(p), c, s, x, 0) == code


def test_null_problems():
    Lb = B.lib()
    assert Lb.moe_mx_quantize(None, OK, OK, OK, 0) == B.MOE_EINVAL
    assert Lb.moe_mx_dequantize(None, OK, OK, OK, 0) == B.MOE_EINVAL
    assert Lb.moe_add_rmsnorm(None, OK, OK, OK, OK, OK, 0, 0, 0) == B.MOE_EINVAL
    assert Lb.moe_mx_linear(None, OK, OK, OK, OK, 0, 0, OK, 0) == B.MOE_EINVAL
    assert Lb.moe_route_topk(None, OK, 0, OK, OK, 0) == B.MOE_EINVAL


NORM = dict(x=OK, residual=OK, weight=OK, residual_out=OK, y=OK, codes=0, scales=0)


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(T=-1), {}, B.MOE_EINVAL),
    (dict(H=0), {}, B.MOE_EINVAL),
    (dict(type=5), {}, B.MOE_EINVAL),
    (dict(w_type=5), {}, B.MOE_EINVAL),
    (dict(mx_fmt=3), {}, B.MOE_EINVAL),
    (dict(eps=-1.0), {}, B.MOE_EINVAL),
    (dict(eps=math.nan), {}, B.MOE_EINVAL),
    (dict(H=68), {}, B.MOE_ENOTSUP),
    (dict(H=16392), {}, B.MOE_ENOTSUP),
    (dict(T=1 << 24), {}, B.MOE_ENOTSUP),
    (dict(H=72, mx_fmt=1), dict(codes=OK, scales=OK), B.MOE_ENOTSUP),
    ({}, dict(x=0), B.MOE_EINVAL),
    ({}, dict(weight=0), B.MOE_EINVAL),
    ({}, dict(weight=OK + 4), B.MOE_EINVAL),
    ({}, dict(residual=0), B.MOE_EINVAL),               # residual_out without residual
    ({}, dict(residual_out=0), B.MOE_EINVAL),
    ({}, dict(y=0), B.MOE_EINVAL),                      # no output
    ({}, dict(y=OK + 8), B.MOE_EINVAL),
    (dict(mx_fmt=2), {}, B.MOE_EINVAL),                 # no codes
    (dict(mx_fmt=2), dict(codes=OK), B.MOE_EINVAL),     # no scales
    (dict(ldx=56), {}, B.MOE_EINVAL),
    (dict(ld_res=68), {}, B.MOE_ENOTSUP),
    (dict(ldy=60), {}, B.MOE_EINVAL),
    (dict(mx_fmt=1, ld_codes=24), dict(codes=OK, scales=OK), B.MOE_EINVAL),
    (dict(T=0), dict(x=0, weight=0, y=0), B.MOE_OK),
])
def test_norm_refusals(kw, ptrs, code):
    p = B.MoeNormProblem(**{**dict(T=4, H=64, eps=1e-6), **kw})
    a = {**NORM, **ptrs}
    assert B.lib().moe_add_rmsnorm(ctypes.byref(p), a["x"], a["residual"], a["weight"], a["residual_out"], a["y"],
                                   a["codes"], a["scales"], 0) == code


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(M=-1), {}, B.MOE_EINVAL),
    (dict(N=0), {}, B.MOE_EINVAL),
    (dict(K=0), {}, B.MOE_EINVAL),
    (dict(K=40), {}, B.MOE_ENOTSUP),
    (dict(K=(1 << 20) + 32), {}, B.MOE_ENOTSUP),
    (dict(M=1 << 24), {}, B.MOE_ENOTSUP),
    (dict(N=1 << 24), {}, B.MOE_ENOTSUP),
    (dict(a_fmt=0), {}, B.MOE_EINVAL),
    (dict(out_type=3), {}, B.MOE_EINVAL),
    (dict(alpha=math.inf), {}, B.MOE_EINVAL),
    (dict(lda=32), {}, B.MOE_EINVAL),
    (dict(lda=72), {}, B.MOE_ENOTSUP),
    (dict(lda=(1 << 22) + 16), {}, B.MOE_ENOTSUP),
    (dict(ld_as=1), {}, B.MOE_EINVAL),
    (dict(ldo=7), {}, B.MOE_EINVAL),
    (dict(ld_add=7), {}, B.MOE_EINVAL),
    ({}, dict(a=0), B.MOE_EINVAL),
    ({}, dict(a_scales=0), B.MOE_EINVAL),
    ({}, dict(w=0), B.MOE_EINVAL),
    ({}, dict(w_scales=0), B.MOE_EINVAL),
    ({}, dict(out=0), B.MOE_EINVAL),
    ({}, dict(a=OK + 8), B.MOE_EINVAL),
    ({}, dict(w=OK + 8), B.MOE_EINVAL),
    ({}, dict(out=OK + 1), B.MOE_EINVAL),
    ({}, dict(bias=OK + 2), B.MOE_EINVAL),
    ({}, dict(add=OK + 1), B.MOE_EINVAL),
    (dict(M=0), dict(a=0, out=0), B.MOE_OK),
])
def test_linear_refusals(kw, ptrs, code):
    p = B.MoeMxLinearProblem(**{**dict(M=4, N=8, K=64, a_fmt=2, out_type=0, alpha=1.0), **kw})
    a = {**dict(a=OK, a_scales=OK, w=OK, w_scales=OK, bias=0, add=0, out=OK), **ptrs}
    assert B.lib().moe_mx_linear(ctypes.byref(p), a["a"], a["a_scales"], a["w"], a["w_scales"], a["bias"], a["add"],
                                 a["out"], 0) == code


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(T=-1), {}, B.MOE_EINVAL),
    (dict(E=0), {}, B.MOE_EINVAL),
    (dict(k=0), {}, B.MOE_EINVAL),
    (dict(k=17), {}, B.MOE_EINVAL),
    (dict(E=1025), {}, B.MOE_ENOTSUP),
    (dict(T=1 << 24), {}, B.MOE_ENOTSUP),
    (dict(E=64, k=33), {}, B.MOE_ENOTSUP),
    (dict(type=3), {}, B.MOE_EINVAL),
    (dict(score=2), {}, B.MOE_EINVAL),
    (dict(group_score=2), {}, B.MOE_EINVAL),
    (dict(renormalize=2), {}, B.MOE_EINVAL),
    (dict(n_group=-1), {}, B.MOE_EINVAL),
    (dict(n_group=65), {}, B.MOE_ENOTSUP),
    (dict(n_group=3, topk_group=1), {}, B.MOE_EINVAL),
    (dict(n_group=4, topk_group=0), {}, B.MOE_EINVAL),
    (dict(n_group=4, topk_group=5), {}, B.MOE_EINVAL),
    (dict(n_group=8, topk_group=1, k=3), {}, B.MOE_EINVAL),
    (dict(n_group=16, topk_group=4, group_score=1), {}, B.MOE_EINVAL),
    (dict(routed_scaling_factor=math.inf), {}, B.MOE_EINVAL),
    (dict(ld=15), {}, B.MOE_EINVAL),
    ({}, dict(logits=0), B.MOE_EINVAL),
    ({}, dict(ids=0), B.MOE_EINVAL),
    ({}, dict(w=0), B.MOE_EINVAL),
    ({}, dict(logits=OK + 2), B.MOE_EINVAL),
    ({}, dict(bias=OK + 2), B.MOE_EINVAL),
    (dict(T=0), dict(logits=0, ids=0, w=0), B.MOE_OK),
])
def test_route_refusals(kw, ptrs, code):
    p = B.MoeRouteTopkProblem(**{**dict(T=4, E=16, k=2, type=2, routed_scaling_factor=1.0), **kw})
    a = {**dict(logits=OK, bias=0, ids=OK, w=OK), **ptrs}
    assert B.lib().moe_route_topk(ctypes.byref(p), a["logits"], a["bias"], a["ids"], a["w"], 0) == code


def test_python_entries_refuse_cpu_tensors():
    x, w = torch.zeros(2, 64), torch.zeros(64)
    c, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    for call in (lambda: moe.mx_quantize(x), lambda: moe.mx_dequantize(c, s), lambda: moe.add_rmsnorm(x, w),
                 lambda: moe.mx_linear(c, s, c, s, a_fmt="mxfp4"), lambda: moe.route_topk(x, 2)):
        with pytest.raises(moe.MoeError):
            call()
