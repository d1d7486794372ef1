"""moe_gated_linear and moe_gated_linear_backward on the GPU against the float64 oracle.

Tolerances, element by element. u = half a step of the type relative to the value, e = 2^-23.

A product of 16-bit values is exact in float32; a sum of K of them, in whatever
order, is K - 1 additions of partial sums that are at most S = sum |a||b|, each off by less than e of it (the
matrix instruction is not documented to round each to nearest), plus one for each of up to 64 joined
partial sums, so it is within acc(K, S) = (K + 66) e S.

Forward. |dg|, |du| <= acc(H, |x||W| + |bias|). f moves by at most Lg |dg| + Lu |du|, the largest slopes in the
rectangle of half sides |dg|, |du| around (g, u): the slopes at the point (inside the clamps, where one is near) and at most C (|dg| + |du|)
more, C a bound of the second derivatives. Those of silu are |f_gg| <= |u| / 2, |f_gu| <= 1.1, f_uu = 0; of SwiGLU-OAI
|f_gg| <= 1.702 (|u| + 1) / 2, |f_gu| <= 1.1; of SiTu, with tanh' <= 1, |tanh''| <= 0.77, alpha 1.5 and beta 2, all below 3: C = 2 (1 + |g| + |u|)
covers them (3 at g = u = 0 by the doubled slope, which is kept). Evaluating f in float32:
sigmoid by v_exp_f32 and v_rcp_f32 (1 ulp each) of an argument rounded to e |g| alpha, tanh within 2 ulp:
ev = e (8 + 2 alpha |g|) |f| for silu and SwiGLU-OAI; SiTu's sigmoid the same with alpha 1. Then the rounding, u |f|.

Backward, from the given gate and up: dg is evaluated within ev = e (16 + 2 alpha |g|) of the sum of its terms'
magnitudes, then rounded: r = u |dg| + tiny (u^2 |dg| + tiny where both parts are kept). A product of it over K terms with b: sum (ev + r) |b| + acc(K, |dg||b|), and
the last rounding. Biases' sums: ev summed plus (M + 66) e sum |dg|."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from dense16_cases import GATED, GATED_LARGE
from oracle import dense16 as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
E = 2.0 ** -23
ACTS = {"silu": dict(), "swiglu_oai": dict(alpha=1.702, beta=1.0, limit=7.0), "situ": dict(alpha=1.5, beta=2.0)}
T16 = [torch.bfloat16, torch.float16]


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return torch.finfo(dt).smallest_normal * half(dt)


def acc(K, S):
    return (K + 66) * E * S


def make(seed, M, H, I, dt, bias=False, gain=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = (rn(M, H) * torch.exp(0.3 * rn(M, 1))).to(dt)
    wg, wu = [(rn(I, H) * gain / H ** 0.5).to(dt) for _ in range(2)]
    b = [0.3 * rn(I) for _ in range(2)] if bias else [None, None]
    return x, wg, wu, *b


def slopes(name, g, u, kw):
    """A bound of |f_g|, |f_u| around the point."""
    fg, fu = O.act_grads(name, g, u, **kw)
    lim = kw.get("limit", float("inf"))
    # near a clamp the inner slope counts
    ig, iu = O.act_grads(name, g.clamp(max=lim), u.clamp(-lim, lim), **kw)
    return 2 * torch.maximum(fg.abs(), ig.abs()) + 0.1 * (1 + u.abs()), 2 * torch.maximum(fu.abs(), iu.abs()) + 0.1 * (1 + g.abs())


def check(got, ref, bound, what=""):
    assert torch.isfinite(got).all(), what
    r = ((got.double() - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert r <= 1, (what, r)


def check_forward(r, x, wg, wu, bg, bu, name, kw):
    dt, H = x.dtype, x.shape[1]
    out, g, u = O.gated(x, wg, wu, bg, bu, name, **kw)
    ax = x.double().abs()
    dg, du = [acc(H, ax @ w.double().abs().t() + (0 if b is None else b.double().abs())) for w, b in ((wg, bg), (wu, bu))]
    more = 2 * (1 + g.abs() + u.abs()) * (dg + du)
    lg, lu = [v + more for v in slopes(name, g, u, kw)]
    a = kw.get("alpha", 1.0) if name == "swiglu_oai" else 1.0
    b = lg * dg + lu * du + E * (8 + 2 * a * g.abs()) * out.abs()
    check(r.out, out, b * (1 + half(dt)) + half(dt) * out.abs() + tiny(dt), "out")
    if r.gate is not None:
        check(r.gate, g, dg * (1 + half(dt)) + half(dt) * g.abs() + tiny(dt), "gate")
        check(r.up, u, du * (1 + half(dt)) + half(dt) * u.abs() + tiny(dt), "up")


SHAPES = GATED


@pytest.mark.parametrize("M,H,I", SHAPES)
@pytest.mark.parametrize("dt", T16)
def test_forward_shapes(M, H, I, dt):
    name = list(ACTS)[(M + I) % 3]
    print(f"[gated] {M}x{H}x{I} {dt} {name}", flush=True)
    ops = make(M + H + I, M, H, I, dt, bias=M % 2 == 0)
    r = moe.gated_linear(*ops[:3], act=name, bias_gate=ops[3], bias_up=ops[4], save=I % 16 == 8, **ACTS[name])
    torch.cuda.synchronize()
    check_forward(r, *ops, name, ACTS[name])


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("M", [1, 40, 600])
def test_forward_activations(M, name):
    """Every activation with values far beyond its clamps (weights four times as large)."""
    print(f"[gated] act {name} M={M}", flush=True)
    ops = make(M, M, 320, 264, torch.bfloat16, bias=True, gain=6.0)
    r = moe.gated_linear(*ops[:3], act=name, bias_gate=ops[3], bias_up=ops[4], save=True, **ACTS[name])
    torch.cuda.synchronize()
    check_forward(r, *ops, name, ACTS[name])
    plain = moe.gated_linear(*ops[:3], act=name, bias_gate=ops[3], bias_up=ops[4], **ACTS[name])
    assert plain.gate is None and torch.equal(plain.out, r.out)


def padded(t, pad, fill=float("nan")):
    """The same matrix as a view of a wider one whose other values are `fill`."""
    w = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    w[:, : t.shape[1]] = t
    return w[:, : t.shape[1]], w


@pytest.mark.parametrize("M", [1, 37, 300])
def test_strided_operands_and_outputs(M):
    """Rows apart in every operand, NaN between them; what lies between output rows stays."""
    print(f"[gated] strided M={M}", flush=True)
    x, wg, wu, bg, bu = make(7, M, 136, 200, torch.bfloat16, bias=True)
    want = moe.gated_linear(x, wg, wu, bias_gate=bg, bias_up=bu, save=True)
    outs = [padded(torch.zeros(M, 200, dtype=x.dtype, device=DEV), p, 5.0) for p in (8, 16, 24)]
    moe.gated_linear(padded(x, 8)[0], padded(wg, 16)[0], padded(wu, 24)[0], bias_gate=bg, bias_up=bu, out=outs[0][0],
                     gate=outs[1][0], up=outs[2][0])
    torch.cuda.synchronize()
    for (v, whole), w in zip(outs, want):
        assert torch.equal(v, w) and (whole[:, 200:] == 5.0).all()
    dout = torch.randn(M, 200, device=DEV).bfloat16()
    kw = dict(want_dbias=True)
    ref = moe.gated_linear_backward(dout, x, wg, wu, want.gate, want.up, **kw)
    dx, dxw = padded(torch.zeros_like(x), 8, 5.0)
    dwg, dwgw = padded(torch.zeros_like(wg), 8, 5.0)
    dwu, dwuw = padded(torch.zeros_like(wu), 24, 5.0)
    got = moe.gated_linear_backward(padded(dout, 8)[0], padded(x, 24)[0], padded(wg, 8)[0], padded(wu, 16)[0],
                                    padded(want.gate, 8)[0], padded(want.up, 16)[0], dx=dx, dw_gate=dwg, dw_up=dwu, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert (dxw[:, 136:] == 5).all() and (dwgw[:, 136:] == 5).all() and (dwuw[:, 136:] == 5).all()


def grad_bounds(dout, x, wg, wu, gate, up, name, kw, parts=1):
    dt, (M, I), H = x.dtype, dout.shape, x.shape[1]
    g, u, d = gate.double(), up.double(), dout.double()
    ref = O.gated_grads(dout, x, wg, wu, gate, up, name, **kw)
    dg, du = ref[5:]
    a = kw.get("alpha", 1.0) if name == "swiglu_oai" else 1.0
    # magnitudes of the terms of the derivatives: |f_g| terms 1 + alpha |g|, |f_u| itself
    beta = kw.get("beta", 0.0)
    mag = (u.abs() + beta) if name != "situ" else torch.full_like(u, beta)
    if name == "swiglu_oai":
        mag = torch.minimum(u.abs(), torch.full_like(u, kw["limit"])) + beta
    sg = torch.sigmoid(a * g.clamp(max=kw.get("limit", float("inf"))))
    eg = E * (16 + 2 * a * g.abs()) * d.abs() * mag * sg * (2 + a * g.abs() * (1 - sg))
    eu = E * (16 + 2 * a * g.abs()) * d.abs() * ((g.abs() * sg) if name != "situ" else torch.full_like(u, kw["alpha"]) * sg)
    h = half(dt) ** parts
    rg, ru = eg + h * dg.abs() + tiny(dt), eu + h * du.abs() + tiny(dt)
    ag, au, X = dg.abs() + rg, du.abs() + ru, x.double().abs()
    wga, wua = wg.double().abs(), wu.double().abs()
    bx = rg @ wga + ru @ wua + acc(2 * I, ag @ wga + au @ wua)
    bg = rg.t() @ X + acc(M, ag.t() @ X)
    bu = ru.t() @ X + acc(M, au.t() @ X)
    return ref, bx, bg, bu, (eg.sum(0) + (M + 66) * E * dg.abs().sum(0)), (eu.sum(0) + (M + 66) * E * du.abs().sum(0))


def check_grads(r, dout, x, wg, wu, gate, up, name, kw, old=(0, 0, 0, 0), parts=1):
    dt = x.dtype
    ref, bx, bg, bu, bbg, bbu = grad_bounds(dout, x, wg, wu, gate, up, name, kw, parts)
    rounded = lambda v, b, t: b * (1 + half(t)) + half(t) * v.abs() + tiny(t)  # noqa: E731
    if r.dx is not None:
        check(r.dx, ref[0], rounded(ref[0], bx, dt), "dx")
    for got, want, b, o, what in ((r.dw_gate, ref[1], bg, old[0], "dw_gate"), (r.dw_up, ref[2], bu, old[1], "dw_up"),
                                  (r.dbias_gate, ref[3], bbg, old[2], "dbias_gate"), (r.dbias_up, ref[4], bbu, old[3], "dbias_up")):
        if got is not None:
            check(got, want + o, rounded(want + o, b, got.dtype), what)


def grad_ops(seed, M, H, I, dt, bias=False, gain=1.5):
    x, wg, wu, bg, bu = make(seed, M, H, I, dt, bias, gain)
    _, g, u = O.gated(x, wg, wu, bg, bu)
    d = torch.randn(M, I, generator=torch.Generator(device=DEV).manual_seed(seed + 1), device=DEV) * (0.5 if dt == torch.float16 else 0.02)
    return d.to(dt), x, wg, wu, g.to(dt), u.to(dt)


@pytest.mark.parametrize("M,H,I", SHAPES)
@pytest.mark.parametrize("dt", T16)
def test_backward_shapes(M, H, I, dt):
    name = list(ACTS)[(M + H // 8) % 3]
    print(f"[grad] {M}x{H}x{I} {dt} {name}", flush=True)
    ops = grad_ops(M + 3 * H + I, M, H, I, dt)
    r = moe.gated_linear_backward(*ops, act=name, want_dbias=M % 2 == 1, **ACTS[name])
    torch.cuda.synchronize()
    assert (r.dbias_gate is not None) == (M % 2 == 1)
    check_grads(r, *ops, name, ACTS[name])


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("dt", T16)
def test_backward_float32_weight_gradients_and_accumulation(name, dt):
    print(f"[grad] f32 {name} {dt}", flush=True)
    M, H, I = 77, 264, 136
    ops = grad_ops(5, M, H, I, dt, gain=6.0)
    for t in (torch.float32, dt):
        dw = [torch.empty(I, H, dtype=t, device=DEV) for _ in range(2)]
        db = [torch.empty(I, device=DEV) for _ in range(2)]
        r = moe.gated_linear_backward(*ops, act=name, dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1], **ACTS[name])
        torch.cuda.synchronize()
        assert r.dw_gate is dw[0] and r.dbias_up is db[1]
        check_grads(r, *ops, name, ACTS[name])
        old = [v.double() for v in dw + db]
        moe.gated_linear_backward(*ops, act=name, dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1], accumulate=True,
                                  want_dx=False, **ACTS[name])
        torch.cuda.synchronize()
        check_grads(moe.GatedGrads(None, *dw, *db), *ops, name, ACTS[name], old)


@pytest.mark.parametrize("M,H,I", [(1, 72, 88), (1, 264, 16384), (2, 264, 8), (17, 8200, 960), (63, 136, 72), (64, 2056, 256)])
@pytest.mark.parametrize("dt", T16)
def test_gradients_of_few_values_are_rounded_once(M, H, I, dt):
    """Up to 16384 values (and 64 rows) dg and du are two 16-bit values, the second of at most half a step of the first and itself off by half a step: in
    the bound above r is the square of u."""
    name = list(ACTS)[M % 3]
    print(f"[grad] two parts {M}x{H}x{I} {dt} {name}", flush=True)
    ops = grad_ops(M + H + I, M, H, I, dt)
    r = moe.gated_linear_backward(*ops, act=name, **ACTS[name])
    torch.cuda.synchronize()
    check_grads(r, *ops, name, ACTS[name], parts=2)


def test_backward_parts_alone_and_clamps():
    """Each gradient alone has the bits it has among all; values on a clamp pass gradients, values beyond none."""
    print("[grad] parts", flush=True)
    kw = ACTS["swiglu_oai"]
    d, x, wg, wu, g, u = grad_ops(9, 50, 136, 72, torch.bfloat16)
    g[0], u[0] = 7.0, 7.0
    g[1], u[1] = 7.03125, -7.03125
    g[2], u[2] = -50.0, -7.0
    args = (d, x, wg, wu, g, u)
    r = moe.gated_linear_backward(*args, act="swiglu_oai", want_dbias=True, **kw)
    check_grads(r, *args, "swiglu_oai", kw)
    one = dict(want_dx=False, want_dw=False, want_dbias=False)
    for flag, names in (("want_dx", ["dx"]), ("want_dw", ["dw_gate", "dw_up"]), ("want_dbias", ["dbias_gate", "dbias_up"])):
        s = moe.gated_linear_backward(*args, act="swiglu_oai", **{**one, flag: True}, **kw)
        torch.cuda.synchronize()
        for n in moe.GatedGrads._fields:
            a = getattr(s, n)
            assert (a is not None) == (n in names) and (a is None or torch.equal(a, getattr(r, n)))
    # a row beyond every clamp alone moves nothing
    s = moe.gated_linear_backward(d[1:2], x[1:2], wg, wu, g[1:2], u[1:2], act="swiglu_oai", want_dbias=True, **kw)
    assert all((v == 0).all() for v in s)


@pytest.mark.parametrize("name", list(ACTS))
def test_gradients_against_differences(name):
    """The oracle's formula against central differences of its forward pass in float64, then the kernel against
    the oracle through a loss of the framework's own forward pass."""
    kw = ACTS[name]
    x, wg, wu, bg, bu = [t.double() for t in make(3, 6, 24, 16, torch.bfloat16, bias=True)]
    d = torch.randn(6, 16, device=DEV, dtype=torch.float64)
    loss = lambda *o: (O.gated(*o, name, **kw)[0] * d).sum()  # noqa: E731
    _, g, u = O.gated(x, wg, wu, bg, bu, name, **kw)
    grads = O.gated_grads(d, x, wg, wu, g, u, name, **kw)[:5]
    ops = [x, wg, wu, bg, bu]
    h = 1e-6
    for i, gr in enumerate(grads):
        v = torch.randn_like(ops[i])
        up, dn = [loss(*[o + s * h * v if j == i else o for j, o in enumerate(ops)]) for s in (1, -1)]
        # central differences: h^2 of the third derivative, and 2^-52 of the loss over h
        num = ((up - dn) / (2 * h)).item()
        assert abs(num - (gr * v).sum().item()) <= 1e-6 * (gr.abs() * v.abs()).sum().item() + 1e-7


@pytest.mark.parametrize("M", [0])
def test_no_rows(M):
    x, wg, wu, bg, bu = make(1, 4, 64, 72, torch.bfloat16, bias=True)
    r = moe.gated_linear(x[:0], wg, wu, save=True)
    assert r.out.shape == (0, 72) and r.gate.shape == (0, 72)
    d = torch.empty(0, 72, dtype=x.dtype, device=DEV)
    for t in (torch.bfloat16, torch.float32):
        dw = [torch.full((72, 64), 3.0, dtype=t, device=DEV) for _ in range(2)]
        db = [torch.full((72,), 3.0, device=DEV) for _ in range(2)]
        kw = dict(dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1])
        moe.gated_linear_backward(d, x[:0], wg, wu, d, d, accumulate=True, **kw)
        torch.cuda.synchronize()
        assert all((v == 3).all() for v in dw + db)
        r = moe.gated_linear_backward(d, x[:0], wg, wu, d, d, **kw)
        torch.cuda.synchronize()
        assert r.dx.shape == (0, 64) and all((v == 0).all() for v in dw + db)


@pytest.mark.parametrize("M", [3, 200])
def test_nan_and_infinity_stay_in_their_rows(M):
    print(f"[gated] nan M={M}", flush=True)
    x, wg, wu, _, _ = make(2, M, 136, 264, torch.bfloat16)
    clean = moe.gated_linear(x, wg, wu, save=True)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    bad = moe.gated_linear(x2, wg, wu, act="swiglu_oai", **ACTS["swiglu_oai"])
    ref = moe.gated_linear(x, wg, wu, act="swiglu_oai", **ACTS["swiglu_oai"])
    torch.cuda.synchronize()
    rest = torch.arange(M, device=DEV) != 1
    assert bad.out[1].isnan().all() and torch.equal(bad.out[rest], ref.out[rest])
    d = torch.randn(M, 264, device=DEV).bfloat16()
    r0 = moe.gated_linear_backward(d, x, wg, wu, clean.gate, clean.up)
    d[1, 7] = float("inf")
    r1 = moe.gated_linear_backward(d, x, wg, wu, clean.gate, clean.up)
    torch.cuda.synchronize()
    assert not r1.dx[1].isfinite().all() and torch.equal(r0.dx[rest], r1.dx[rest])
    cols = torch.arange(264, device=DEV) != 7
    assert torch.equal(r0.dw_gate[cols], r1.dw_gate[cols]) and torch.equal(r0.dw_up[cols], r1.dw_up[cols])


def test_repeats_are_bitwise_equal():
    ops = grad_ops(4, 333, 520, 392, torch.bfloat16)
    first = moe.gated_linear_backward(*ops, want_dbias=True)
    f1 = moe.gated_linear(*ops[1:4], save=True)
    for _ in range(3):
        again = moe.gated_linear_backward(*ops, want_dbias=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(a, b) for a, b in zip(f1, moe.gated_linear(*ops[1:4], save=True)))


@pytest.mark.parametrize("M,H,I", GATED_LARGE)
@pytest.mark.parametrize("dt", T16)
def test_many_rows(M, H, I, dt):
    """Sizes that fill the chip with the largest tiles in one direction or all, with ends inside tiles."""
    name = list(ACTS)[(M + H // 8) % 3]
    print(f"[gated, grad] {M}x{H}x{I} {dt} {name}", flush=True)
    ops = make(M + H, M, H, I, dt, bias=M % 2 == 0)
    r = moe.gated_linear(*ops[:3], act=name, bias_gate=ops[3], bias_up=ops[4], save=True, **ACTS[name])
    torch.cuda.synchronize()
    check_forward(r, *ops, name, ACTS[name])
    d = (torch.randn(M, I, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV) * 0.02).to(dt)
    args = (d, *ops[:3], r.gate, r.up)
    s = moe.gated_linear_backward(*args, act=name, want_dbias=True, **ACTS[name])
    torch.cuda.synchronize()
    check_grads(s, *args, name, ACTS[name])


def test_rows_far_apart():
    """Every operand's rows 2^21 elements apart, so that the last ones lie past 2^32: the bits of compact operands."""
    print("[gated, grad] far", flush=True)
    M, H, I, dt = 2057, 72, 2056, torch.bfloat16
    base = torch.empty(2064, 1 << 21, dtype=dt, device=DEV)
    at = iter(range(0, 1 << 21, 4096))

    def far(t):
        v = base[:t.shape[0]].narrow(1, next(at), t.shape[1])
        return v.copy_(t)

    d, x, wg, wu, _, _ = grad_ops(6, M, H, I, dt)
    r = moe.gated_linear(x, wg, wu, save=True)
    s = moe.gated_linear_backward(d, x, wg, wu, r.gate, r.up)
    new = [far(torch.zeros_like(t)) for t in (r.out, r.gate, r.up, s.dx, s.dw_gate, s.dw_up)]
    X, G, U, D = far(x), far(wg), far(wu), far(d)
    for few in (3, M):
        moe.gated_linear(X[:few], G, U, out=new[0][:few], gate=new[1][:few], up=new[2][:few])
        ref = moe.gated_linear(x[:few], wg, wu, save=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a[:few], b) for a, b in zip(new, ref))
        moe.gated_linear_backward(D[:few], X[:few], G, U, new[1][:few], new[2][:few], dx=new[3][:few], dw_gate=new[4], dw_up=new[5])
        ref = moe.gated_linear_backward(d[:few], x[:few], wg, wu, ref.gate, ref.up)
        torch.cuda.synchronize()
        assert torch.equal(new[3][:few], ref.dx) and torch.equal(new[4], ref.dw_gate) and torch.equal(new[5], ref.dw_up)


@pytest.mark.parametrize("dt", T16)
def test_derivatives_of_saturated_values(dt):
    """SiTu's derivatives keep their relative precision where tanh nears 1. One row, so the biases' gradients are dg and
    du themselves, in float32. With y = u / beta (division within 2 e), 4 q r^2, q = exp(-2 |y|) and r = 1 / (1 + q): the
    exponent is off by at most 2 |y| (2 e + e), q by e (6 |y| + 1) of itself, r by 1.5 e, the products by e: e (6 |y| + 5). tanh is
    within 2 e, a sigmoid e (3 |g| + 3), each further product e / 2: together less than e (6 |y| + 3 |g| + 16), and for
    the sum of positive terms that g > 0 gives, e (6 |g| / alpha + 6 |g| + 24)."""
    print(f"[grad] saturated {dt}", flush=True)
    kw = ACTS["situ"]
    I = 512
    g = torch.linspace(0.05, 24, I, device=DEV).to(dt)[None]
    u = (torch.linspace(0.1, 40, I, device=DEV).flip(0) * torch.tensor([1.0, -1.0], device=DEV).repeat(I // 2)).to(dt)[None]
    d = torch.ones_like(g)
    x, w = torch.ones(1, 8, dtype=dt, device=DEV), torch.ones(I, 8, dtype=dt, device=DEV)
    r = moe.gated_linear_backward(d, x, w, w, g, u, act="situ", want_dx=False, want_dw=False, want_dbias=True, **kw)
    torch.cuda.synchronize()
    G, U, a, b = g.double()[0], u.double()[0], kw["alpha"], kw["beta"]
    s, sech2 = torch.sigmoid(G), lambda v: 1 / torch.cosh(v).square()  # noqa: E731
    fg = s * (sech2(G / a) + a * torch.tanh(G / a) * torch.sigmoid(-G)) * b * torch.tanh(U / b)
    fu = a * torch.tanh(G / a) * s * sech2(U / b)
    check(r.dbias_gate, fg, E * (6 * G / a + 6 * G + 24) * fg.abs())
    check(r.dbias_up, fu, E * (6 * U.abs() / b + 3 * G + 16) * fu.abs())
