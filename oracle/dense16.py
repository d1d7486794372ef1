"""Float64 oracle of the dense 16-bit projections (test infrastructure only): the
gated block, its gradients, and a projection with low-rank adapters. Torch
tensors in and out, on whatever device they are, all in float64.

Sources: the vLLM page "moonep_experts" (module docstring: gate and up
projections and silu(gate) * up) and "trtllm_mxfp4_moe" (SwiGLU-OAI and SiTu
parameters); the readings of the activations are moe_oracle's. Derivatives and adapters
are formulas of this repository: parity unpinned, checked against differences.
"""
from __future__ import annotations

import torch


def act(name: str, g, u, alpha=1.0, beta=0.0, limit=float("inf")):
    if name == "silu":
        return g * torch.sigmoid(g) * u
    if name == "situ":
        return alpha * torch.tanh(g / alpha) * torch.sigmoid(g) * beta * torch.tanh(u / beta)
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g * torch.sigmoid(alpha * g) * (u + beta)


def act_grads(name: str, g, u, alpha=1.0, beta=0.0, limit=float("inf")):
    """Derivatives of act by g and u; 0 beyond the clamps, the inner ones on them."""
    if name == "silu":
        s = torch.sigmoid(g)
        return u * (s + g * s * (1 - s)), g * s
    if name == "situ":
        s, tg, tu = torch.sigmoid(g), torch.tanh(g / alpha), torch.tanh(u / beta)
        return ((1 - tg ** 2) * s + alpha * tg * s * (1 - s)) * beta * tu, alpha * tg * s * (1 - tu ** 2)
    gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    s = torch.sigmoid(alpha * gc)
    zero = torch.zeros_like(g)
    return (torch.where(g > limit, zero, (uc + beta) * (s + alpha * gc * s * (1 - s))),
            torch.where(u.abs() > limit, zero, gc * s))


def gated(x, wg, wu, bg=None, bu=None, name="silu", **kw):
    """(out, gate, up)."""
    x = x.double()
    g, u = x @ wg.double().t(), x @ wu.double().t()
    if bg is not None:
        g, u = g + bg.double(), u + bu.double()
    return act(name, g, u, **kw), g, u


def gated_grads(dout, x, wg, wu, gate, up, name="silu", **kw):
    """(dx, dw_gate, dw_up, dbias_gate, dbias_up, dg, du)."""
    fg, fu = act_grads(name, gate.double(), up.double(), **kw)
    dg, du = dout.double() * fg, dout.double() * fu
    x = x.double()
    return dg @ wg.double() + du @ wu.double(), dg.t() @ x, du.t() @ x, dg.sum(0), du.sum(0), dg, du


def lora(x, w, a, b, ids, scales, bias=None, add=None):
    x = x.double()
    y = x.new_zeros(x.shape[0], b.shape[1])
    if w is not None:
        y = y + x @ w.double().t()
    for i in range(a.shape[0]):
        m = (ids == i).nonzero().flatten()
        y[m] += scales[i].double() * (x[m] @ a[i].double().t()) @ b[i].double().t()
    if bias is not None:
        y = y + bias.double()
    return y if add is None else y + add.double()
