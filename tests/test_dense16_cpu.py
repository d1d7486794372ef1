"""The dense 16-bit projections without a GPU: the oracle's formulas against other
formulations, and the refusals of the C ABI and of the Python entry points
(checked before anything is enqueued)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
import oracle
from mixture_experts_expert_02_amd import binding as B
from oracle import dense16 as O

OK = 4096  # an address that is never read: every call below is refused first
ACTS = {"silu": dict(), "swiglu_oai": dict(alpha=1.702, beta=1.0, limit=2.0), "situ": dict(alpha=1.5, beta=2.0)}


@pytest.mark.parametrize("name", list(ACTS))
def test_oracle_block_is_the_experts_steps(name):
    """One expert with route weight 1, without its down projection (an identity)."""
    g = torch.Generator().manual_seed(1)
    x, wg, wu = [torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 12), (12, 12), (12, 12))]
    out, _, _ = O.gated(x, wg, wu, name=name, **ACTS[name])
    ref = oracle.experts_forward(x.numpy(), np.zeros((5, 1), np.int32), np.ones((5, 1), np.float32), wg[None].numpy(),
                                 wu[None].numpy(), np.eye(12)[None], act=name, **ACTS[name])
    np.testing.assert_allclose(out.numpy(), ref, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("name", list(ACTS))
def test_oracle_derivatives_by_autograd(name):
    g = torch.Generator().manual_seed(2)
    a, b = [(3 * torch.randn(200, generator=g, dtype=torch.float64)).requires_grad_() for _ in range(2)]
    with torch.no_grad():
        a[0], b[1], b[2] = 2.0, 2.0, -2.0  # on the clamps: both pass gradients there
    O.act(name, a, b, **ACTS[name]).sum().backward()
    fg, fu = O.act_grads(name, a.detach(), b.detach(), **ACTS[name])
    torch.testing.assert_close(fg, a.grad, rtol=1e-12, atol=1e-14)
    torch.testing.assert_close(fu, b.grad, rtol=1e-12, atol=1e-14)


def test_oracle_lora_by_dense_weights():
    """A row of adapter a is a row times the weight with the adapter's product added."""
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, a, b, sc = rn(9, 8), rn(6, 8), rn(3, 4, 8), rn(3, 6, 4), rn(3)
    ids = torch.tensor([0, 2, -1, 1, 3, 0, 2, -7, 1])
    y = O.lora(x, w, a, b, ids, sc)
    for m, i in enumerate(ids.tolist()):
        full = w + (sc[i] * b[i] @ a[i] if 0 <= i < 3 else 0)
        torch.testing.assert_close(y[m], full @ x[m])


# ---------------------------------------------------------------- refusals
def gated(**kw):
    return B.MoeGatedProblem(**{**dict(M=4, H=64, I=72, type=0, act=0, alpha=1.0, beta=0.0, limit=math.inf), **kw})


SIZES = [
    (dict(M=-1), B.MOE_EINVAL), (dict(H=0), B.MOE_EINVAL), (dict(I=0), B.MOE_EINVAL), (dict(type=3), B.MOE_EINVAL),
    (dict(type=-1), B.MOE_EINVAL), (dict(type=2), B.MOE_ENOTSUP), (dict(act=3), B.MOE_EINVAL), (dict(act=-1), B.MOE_EINVAL),
    (dict(act=1, alpha=math.nan), B.MOE_EINVAL), (dict(act=1, beta=math.inf), B.MOE_EINVAL),
    (dict(act=1, limit=math.nan), B.MOE_EINVAL), (dict(act=1, limit=0.0), B.MOE_ENOTSUP), (dict(act=2, beta=0.0), B.MOE_ENOTSUP),
    (dict(act=2, alpha=-1.0, beta=1.0), B.MOE_ENOTSUP), (dict(H=68), B.MOE_ENOTSUP), (dict(I=68), B.MOE_ENOTSUP),
    (dict(M=1 << 24), B.MOE_ENOTSUP), (dict(H=(1 << 20) + 8), B.MOE_ENOTSUP), (dict(I=(1 << 20) + 8), B.MOE_ENOTSUP),
    (dict(H=1 << 17, I=1 << 16), B.MOE_ENOTSUP), (dict(ldx=56), B.MOE_EINVAL), (dict(ldx=-64), B.MOE_EINVAL),
    (dict(ldx=68), B.MOE_ENOTSUP), (dict(ldx=(1 << 21) + 8), B.MOE_ENOTSUP), (dict(ld_wg=56), B.MOE_EINVAL),
    (dict(ld_wu=76), B.MOE_ENOTSUP), (dict(ld_out=64), B.MOE_EINVAL), (dict(ld_out=76), B.MOE_ENOTSUP),
    (dict(ld_gate=64), B.MOE_EINVAL), (dict(ld_up=84), B.MOE_ENOTSUP),
]
FWD = ("x", "w_gate", "w_up", "bias_gate", "bias_up", "out", "gate", "up", "ws", "size")


def call_gated(p, **kw):
    a = {**dict(x=OK, w_gate=OK, w_up=OK, bias_gate=0, bias_up=0, out=OK, gate=0, up=0, ws=OK, size=1 << 40), **kw}
    return B.lib().moe_gated_linear(None if p is None else ctypes.byref(p), *[a[n] for n in FWD], 0)


@pytest.mark.parametrize("kw,code", SIZES)
def test_gated_sizes_are_refused(kw, code):
    assert call_gated(gated(**kw)) == code
    assert B.moe_gated_linear_workspace_bytes(gated(**kw)) == 0
    g = B.MoeGatedGradProblem(gated(**kw), kw.get("type", 0), 0, 0, 0, 0)
    assert call_grad(g) == code
    assert B.moe_gated_linear_backward_workspace_bytes(g) == 0


@pytest.mark.parametrize("ptrs,code", [
    (dict(x=0), B.MOE_EINVAL), (dict(w_gate=0), B.MOE_EINVAL), (dict(w_up=0), B.MOE_EINVAL), (dict(out=0), B.MOE_EINVAL),
    (dict(x=OK + 8), B.MOE_EINVAL), (dict(w_up=OK + 2), B.MOE_EINVAL), (dict(out=OK + 8), B.MOE_EINVAL),
    (dict(gate=OK), B.MOE_EINVAL), (dict(up=OK), B.MOE_EINVAL), (dict(gate=OK + 8, up=OK), B.MOE_EINVAL),
    (dict(bias_gate=OK), B.MOE_EINVAL), (dict(bias_up=OK), B.MOE_EINVAL), (dict(bias_gate=OK + 2, bias_up=OK), B.MOE_EINVAL),
])
def test_gated_pointers_are_refused(ptrs, code):
    assert call_gated(gated(), **ptrs) == code


def test_gated_accepts_no_rows_and_refuses_null():
    assert call_gated(gated(M=0), x=0, out=0) == B.MOE_OK
    assert call_gated(None) == B.MOE_EINVAL
    assert call_grad(None) == B.MOE_EINVAL
    assert call_lora(None) == B.MOE_EINVAL
    for n in ("moe_gated_linear", "moe_gated_linear_backward", "moe_lora_linear"):
        assert getattr(B.lib(), n + "_workspace_bytes")(None) == 0


BWD = ("dout", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up", "ws", "size")


def grad(dw_type=0, accumulate=0, ld_dx=0, ld_dwg=0, ld_dwu=0, **kw):
    return B.MoeGatedGradProblem(gated(**kw), dw_type, accumulate, ld_dx, ld_dwg, ld_dwu)


def call_grad(p, **kw):
    a = {**{n: OK for n in BWD}, "size": 1 << 40, **kw}
    return B.lib().moe_gated_linear_backward(None if p is None else ctypes.byref(p), *[a[n] for n in BWD], 0)


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(dw_type=1), {}, B.MOE_ENOTSUP), (dict(dw_type=3), {}, B.MOE_EINVAL), (dict(accumulate=2), {}, B.MOE_EINVAL),
    (dict(ld_dx=56), {}, B.MOE_EINVAL), (dict(ld_dx=68), {}, B.MOE_ENOTSUP), (dict(ld_dwg=68), {}, B.MOE_ENOTSUP),
    (dict(ld_dwu=66, dw_type=2), {}, B.MOE_ENOTSUP), (dict(ld_dwu=(1 << 40) + 8), {}, B.MOE_ENOTSUP),
    ({}, dict(dout=0), B.MOE_EINVAL), ({}, dict(gate=0), B.MOE_EINVAL), ({}, dict(up=0), B.MOE_EINVAL),
    ({}, dict(x=0), B.MOE_EINVAL), ({}, dict(w_gate=0), B.MOE_EINVAL), ({}, dict(w_up=OK + 8), B.MOE_EINVAL),
    ({}, dict(dw_gate=0), B.MOE_EINVAL), ({}, dict(dw_up=0), B.MOE_EINVAL), ({}, dict(dbias_up=0), B.MOE_EINVAL),
    ({}, dict(dx=OK + 8), B.MOE_EINVAL), ({}, dict(dw_up=OK + 8), B.MOE_EINVAL), ({}, dict(dbias_gate=OK + 2), B.MOE_EINVAL),
    ({}, dict(dx=0, dw_gate=0, dw_up=0, dbias_gate=0, dbias_up=0), B.MOE_EINVAL), ({}, dict(ws=0), B.MOE_EINVAL),
    ({}, dict(ws=OK + 8), B.MOE_EINVAL), ({}, dict(size=0), B.MOE_ENOSPC),
    (dict(M=0, accumulate=1), dict(dout=0, ws=0, size=0), B.MOE_OK),
])
def test_gated_backward_refusals(kw, ptrs, code):
    assert call_grad(grad(**kw), **ptrs) == code


def test_backward_workspace_holds_the_rounded_gradients():
    p = grad(M=100, I=72)
    n = B.moe_gated_linear_backward_workspace_bytes(p)
    assert n >= 2 * 100 * 72 * 2 and call_grad(p, size=n - 1) == B.MOE_ENOSPC


LORA = ("x", "w", "lora_a", "lora_b", "ids", "scales", "bias", "add", "out", "ws", "size")


def call_lora(p, **kw):
    a = {**{n: OK for n in LORA}, "bias": 0, "add": 0, "size": 1 << 40, **kw}
    return B.lib().moe_lora_linear(None if p is None else ctypes.byref(p), *[a[n] for n in LORA], 0)


def lora(**kw):
    return B.MoeLoraProblem(**{**dict(M=4, N=9, K=64, R=16, L=3, type=0), **kw})


@pytest.mark.parametrize("kw,ptrs,code", [
    (dict(M=-1), {}, B.MOE_EINVAL), (dict(N=0), {}, B.MOE_EINVAL), (dict(K=0), {}, B.MOE_EINVAL), (dict(R=0), {}, B.MOE_EINVAL),
    (dict(L=0), {}, B.MOE_EINVAL), (dict(type=3), {}, B.MOE_EINVAL), (dict(type=2), {}, B.MOE_ENOTSUP),
    (dict(M=1 << 24), {}, B.MOE_ENOTSUP), (dict(N=(1 << 20) + 1), {}, B.MOE_ENOTSUP), (dict(K=68), {}, B.MOE_ENOTSUP),
    (dict(K=(1 << 20) + 8), {}, B.MOE_ENOTSUP), (dict(R=12), {}, B.MOE_ENOTSUP), (dict(R=264), {}, B.MOE_ENOTSUP),
    (dict(L=4097), {}, B.MOE_ENOTSUP), (dict(ldx=56), {}, B.MOE_EINVAL), (dict(ldx=68), {}, B.MOE_ENOTSUP),
    (dict(ldw=68), {}, B.MOE_ENOTSUP), (dict(ld_out=8), {}, B.MOE_EINVAL), (dict(ld_add=8), {}, B.MOE_EINVAL),
    (dict(ld_out=(1 << 40) + 1), {}, B.MOE_ENOTSUP),
    ({}, dict(x=0), B.MOE_EINVAL), ({}, dict(x=OK + 8), B.MOE_EINVAL), ({}, dict(w=OK + 8), B.MOE_EINVAL),
    ({}, dict(lora_a=0), B.MOE_EINVAL), ({}, dict(lora_b=OK + 8), B.MOE_EINVAL), ({}, dict(ids=0), B.MOE_EINVAL),
    ({}, dict(ids=OK + 2), B.MOE_EINVAL), ({}, dict(scales=0), B.MOE_EINVAL), ({}, dict(bias=OK + 2), B.MOE_EINVAL),
    ({}, dict(add=OK + 1), B.MOE_EINVAL), ({}, dict(out=0), B.MOE_EINVAL), ({}, dict(out=OK + 1), B.MOE_EINVAL),
    ({}, dict(ws=0), B.MOE_EINVAL), ({}, dict(ws=OK + 8), B.MOE_EINVAL), ({}, dict(size=0), B.MOE_ENOSPC),
    (dict(M=0), dict(x=0, out=0, ws=0, size=0), B.MOE_OK),
])
def test_lora_refusals(kw, ptrs, code):
    assert call_lora(lora(**kw), **ptrs) == code


class OnGpu(torch.Tensor):
    """A tensor without memory that says it is on a GPU: refused for its sizes, or not at all."""

    def get_device(self):
        return 0


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)


X, W, G, D = t(4, 64), t(72, 64), t(4, 72), t(4, 72)
BIG = 2 ** 32 + 64
F32, I32 = torch.float32, torch.int32


@pytest.mark.parametrize("call", [
    lambda: moe.gated_linear(torch.zeros(4, 64).bfloat16(), W, W),
    lambda: moe.gated_linear(t(4, 64, dtype=F32), W, W),
    lambda: moe.gated_linear(X, t(72, 64, dtype=torch.float16), W),
    lambda: moe.gated_linear(X, t(72, 56), W),
    lambda: moe.gated_linear(X, W, t(64, 64)),
    lambda: moe.gated_linear(X, t(64, 72).t(), W),
    lambda: moe.gated_linear(X, W, W, act="gelu"),
    lambda: moe.gated_linear(X, W, W, bias_gate=t(72, dtype=F32)),
    lambda: moe.gated_linear(X, W, W, bias_gate=t(72), bias_up=t(72)),
    lambda: moe.gated_linear(X, W, W, gate=G),
    lambda: moe.gated_linear(X, W, W, out=t(4, 64)),
    lambda: moe.gated_linear(X, W, W, out=t(1, 72).expand(4, 72)),
    lambda: moe.gated_linear(t(BIG, 64), W, W),
    lambda: moe.gated_linear(t(1, BIG), t(72, BIG), t(72, BIG)),
    lambda: moe.gated_linear(X, t(BIG, 64), t(BIG, 64)),
    lambda: moe.gated_linear_backward(t(4, 72, dtype=F32), X, W, W, G, G),
    lambda: moe.gated_linear_backward(D, t(5, 64), W, W, G, G),
    lambda: moe.gated_linear_backward(D, X, W, W, G, t(4, 64)),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, accumulate=True),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, want_dw=False, want_dbias=True, accumulate=True),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, dw_gate=t(72, 64)),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, dw_gate=t(72, 64, dtype=F32), dw_up=t(72, 64)),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, dw_gate=t(72, 64, dtype=torch.float16), dw_up=t(72, 64, dtype=torch.float16)),
    lambda: moe.gated_linear_backward(D, X, W, W, G, G, dbias_gate=t(72, dtype=F32)),
    lambda: moe.gated_linear_backward(t(BIG, 72), t(BIG, 64), W, W, t(BIG, 72), t(BIG, 72)),
    lambda: moe.lora_linear(t(4, 64, dtype=F32), None, t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 8), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 56), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64, dtype=torch.float16), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, t(8, 64), t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 16), t(4, dtype=torch.int64), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 16), t(5, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32), add=t(4, 9, dtype=F32)),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32), out=t(9, 4).t()),
    lambda: moe.lora_linear(X, None, t(3, 16, 64), t(3, BIG, 16), t(4, dtype=I32), t(3, dtype=F32)),
    lambda: moe.lora_linear(t(BIG, 64), None, t(3, 16, 64), t(3, 9, 16), t(BIG, dtype=I32), t(3, dtype=F32)),
])
def test_python_entries_refuse(call):
    with pytest.raises(moe.MoeError):
        call()
