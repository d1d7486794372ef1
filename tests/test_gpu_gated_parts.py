"""How exactly dg and du enter the products of moe_gated_linear_backward. Bounds: test_gpu_gated_linear.py, with r = u^2
of |dg| where both parts are kept."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from mixture_experts_expert_02_amd import binding as B
from oracle import dense16 as O
from test_gpu_gated_linear import ACTS, DEV, E, T16, check_grads, grad_ops, half, padded, tiny

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,H,I", [(65, 72, 8), (100, 72, 88), (129, 136, 120), (200, 264, 72), (256, 1032, 64), (512, 72, 32), (2048, 264, 8)])
@pytest.mark.parametrize("dt", T16)
def test_few_values_of_many_rows_are_rounded_once(M, H, I, dt):
    """Up to 16384 values dg and du are in two parts whatever the number of rows."""
    assert M > 64 and M * I <= 16384
    name = list(ACTS)[M % 3]
    print(f"[grad] two parts {M}x{H}x{I} {dt} {name}", flush=True)
    ops = grad_ops(M + H + I, M, H, I, dt)
    r = moe.gated_linear_backward(*ops, act=name, want_dbias=True, **ACTS[name])
    torch.cuda.synchronize()
    check_grads(r, *ops, name, ACTS[name], parts=2)


MANY = [(64, 2056, 264), (65, 136, 264), (128, 1032, 520), (129, 8, 200), (300, 64, 2048), (600, 1032, 64), (1023, 512, 768), (4099, 2056, 2088),
        (8200, 72, 2120), (8200, 1528, 1496), (2048, 2880, 2880), (1000, 1040, 7168), (6000, 520, 264)]


def excess(dt, K, s2, other2):
    """How far a sum of K products with dg, of root sum of squares s = sqrt(s2), may be off, as a root mean square, but for its own last
    rounding. Errors of terms in however many places have no common sign: the second part is off by at most u^2 of each dg
    (or half float16's smallest step, of products with other2's root), dg's float32 evaluation by less than 64 e, and each of K + 66
    additions by e of a partial sum of at most s in root mean square. Twice that."""
    u = half(dt)
    return 2 * (s2.sqrt() * (u * u + (64 + (K + 66) ** 0.5) * E) + tiny(dt) * other2.sqrt())


@pytest.mark.parametrize("M,H,I", MANY)
@pytest.mark.parametrize("dt", T16)
def test_two_parts_on_request(M, H, I, dt):
    """Of more than 16384 values, in every tile, with and without K ranges: float32 weight gradients within the error of float32 sums, and dx
    rounded otherwise than the exact one only where that error reaches a tie."""
    assert M * I > 16384
    name = list(ACTS)[(M + I // 8) % 3]
    print(f"[grad] two parts on request {M}x{H}x{I} {dt} {name}", flush=True)
    ops = grad_ops(M + H + I, M, H, I, dt)
    dw = [torch.empty(I, H, device=DEV) for _ in range(2)]
    kw = dict(act=name, want_dbias=True, **ACTS[name])
    r = moe.gated_linear_backward(*ops, dw_gate=dw[0], dw_up=dw[1], two_parts=True, **kw)
    torch.cuda.synchronize()
    check_grads(r, *ops, name, ACTS[name], parts=2)
    d, x, wg, wu, g, u = ops
    dx, dwg, dwu, _, _, dg, du = O.gated_grads(*ops, name, **ACTS[name])
    X = x.double().square()
    for got, ref, v in ((r.dw_gate, dwg, dg), (r.dw_up, dwu, du)):
        b = excess(dt, M, v.square().t() @ X, X.sum(0))
        assert (got.double() - ref).square().mean().sqrt() <= b.square().mean().sqrt()
    G, U = wg.double().square(), wu.double().square()
    b = excess(dt, 2 * I, dg.square() @ G + du.square() @ U, G.sum(0) + U.sum(0))
    # ties are at least u |dx| apart
    most = (2 * b / (half(dt) * dx.abs())).clamp(max=1).mean().item()
    assert (r.dx != dx.to(dt)).double().mean().item() <= most
    # 16-bit results are the float32 ones rounded, and biases' sums are what they are without
    s = moe.gated_linear_backward(*ops, two_parts=True, **kw)
    one = moe.gated_linear_backward(*ops, **kw)
    torch.cuda.synchronize()
    assert torch.equal(s.dx, r.dx) and torch.equal(s.dw_gate, r.dw_gate.to(dt)) and torch.equal(s.dw_up, r.dw_up.to(dt))
    assert torch.equal(one.dbias_gate, r.dbias_gate) and torch.equal(one.dbias_up, r.dbias_up)


@pytest.mark.parametrize("M,H,I", [(50, 136, 72), (200, 264, 72), (1, 72, 88)])
def test_few_values_are_in_two_parts_anyway(M, H, I):
    ops = grad_ops(M, M, H, I, torch.bfloat16)
    a, b = [moe.gated_linear_backward(*ops, want_dbias=True, two_parts=t) for t in (False, True)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, w) for v, w in zip(a, b))


@pytest.mark.parametrize("M,H,I", [(40, 264, 520), (100, 264, 520), (900, 264, 520)])
def test_two_parts_accumulated_captured_and_in_their_workspace(M, H, I):
    """Rows apart, gradients added to earlier ones, a workspace of exactly the size between other bytes, replays of a graph."""
    print(f"[grad] two parts captured {M}x{H}x{I}", flush=True)
    ops = grad_ops(1, M, H, I, torch.bfloat16)
    p = B.MoeGatedGradProblem(B.MoeGatedProblem(M, H, I, 0, 0, 1.0, 0.0, float("inf")), B.MOE_T_FP32, 1, 0, 0, 0, 1)
    n = moe.moe_gated_linear_backward_workspace_bytes(p)
    held = torch.full((n + 4352,), 0x7F, dtype=torch.uint8, device=DEV)
    held[:256], held[-4096:] = 0x5A, 0x5A
    ws = held[256: 256 + n]
    wide = [padded(t, 8 * i + 8)[0] for i, t in enumerate(ops)]
    dx, dw, db = torch.empty(M, H, dtype=torch.bfloat16, device=DEV), [torch.empty(I, H, device=DEV) for _ in range(2)], [torch.empty(I, device=DEV) for _ in range(2)]

    def run():
        moe.gated_linear_backward(*wide, dx=dx, dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1], accumulate=True, two_parts=True,
                                  workspace=ws)

    def fill():
        for t in dw + db:
            t.fill_(0.25)
    fill()
    run()
    torch.cuda.synchronize()
    old = [torch.full_like(t, 0.25).double() for t in dw + db]
    check_grads(moe.GatedGrads(dx, *dw, *db), *ops, "silu", {}, old, parts=2)
    want = [t.clone() for t in (dx, *dw, *db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        fill()
        held[256: 256 + n] = 0xFF
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, *dw, *db), want))
        fill()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, *dw, *db), want))
    assert (held[:256] == 0x5A).all() and (held[-4096:] == 0x5A).all()
