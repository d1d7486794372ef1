"""SwiGLU's derivatives where alpha times the gate leaves float32: the sigmoid is 0 or 1 there, its slope 0, and no infinity
times 0 comes in between. One row, so the biases' gradients are dg and du themselves, in float32."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from oracle import dense16 as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("dt,alpha,top", [(torch.bfloat16, 1.702, 3.3e38), (torch.bfloat16, -4.0, 2e38), (torch.float16, 1e35, 6e4)])
@pytest.mark.parametrize("limit", [7.0, float("inf")])
def test_products_beyond_float32(dt, alpha, top, limit):
    print(f"[grad] range {dt} alpha={alpha} limit={limit}", flush=True)
    g = torch.tensor([top, -top, 0.75 * top, -0.75 * top, 3.0, -3.0, 0.0, 1.0], device=DEV).to(dt).repeat(2)[None]
    u = torch.tensor([0.5, -2.0], device=DEV).to(dt).repeat_interleave(8)[None]
    d = torch.full_like(g, 0.5)
    x, w = torch.ones(1, 8, dtype=dt, device=DEV), torch.ones(16, 8, dtype=dt, device=DEV)
    kw = dict(act="swiglu_oai", alpha=alpha, beta=1.0, limit=limit)
    r = moe.gated_linear_backward(d, x, w, w, g, u, want_dx=False, want_dw=False, want_dbias=True, **kw)
    torch.cuda.synchronize()
    alpha = torch.tensor(alpha, dtype=torch.float32).double().item()  # as the call takes it
    G, U, D = g.double()[0], u.double()[0], d.double()[0]
    fg, fu = O.act_grads("swiglu_oai", G, U, alpha=alpha, beta=1.0, limit=limit)
    # sigmoid, its argument within 2 e of |alpha g| <= 12 where it is not 0 or 1, and five products: far below 128 e; terms of opposite
    # sign, at |alpha g| <= 12, are at most 13 times |u + beta| / 2
    e = 2.0 ** -23
    for got, ref in ((r.dbias_gate, D * fg), (r.dbias_up, D * fu)):
        assert torch.isfinite(got).all(), got
        b = 128 * e * ref.abs() + (13 * 1.5 * 128 * e if got is r.dbias_gate else 0) * (alpha * G).abs().le(12).double()
        assert ((got.double() - ref).abs() <= b).all(), (got, ref)
