"""moe_gated_linear_backward's gradients of weights and biases added to earlier ones, and in float32, beyond the few rows whose
kernel holds all of them at once: tiles of 128 and 256 rows, with and without ranges of rows, and column sums of one
workgroup and of several. Bounds: test_gpu_gated_linear.py."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from dense16_accumulate_cases import ACCUMULATE
from test_gpu_gated_linear import ACTS, DEV, T16, check_grads, grad_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,H,I", ACCUMULATE)
@pytest.mark.parametrize("dt", T16)
@pytest.mark.parametrize("f32", [True, False])
def test_accumulation(M, H, I, dt, f32):
    """Two steps, the second one added to the first; rows apart in the gradients, and what lies between them stays."""
    name = list(ACTS)[(M + H // 8) % 3]
    print(f"[grad, accumulated] {M}x{H}x{I} {dt} f32={f32} {name}", flush=True)
    t = torch.float32 if f32 else dt
    whole = [torch.full((I, H + p), 5.0, dtype=t, device=DEV) for p in ((4, 12) if f32 else (8, 16))]
    dw = [v[:, :H] for v in whole]
    db = [torch.full((I,), 5.0, device=DEV) for _ in range(2)]
    kw = dict(act=name, dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1], **ACTS[name])
    old = (0, 0, 0, 0)
    for step in range(2):
        ops = grad_ops(M + step, M, H, I, dt)
        r = moe.gated_linear_backward(*ops, accumulate=step == 1, **kw)
        torch.cuda.synchronize()
        assert r.dw_gate is dw[0] and r.dbias_up is db[1]
        check_grads(r, *ops, name, ACTS[name], old)
        assert all((v[:, H:] == 5).all() for v in whole)
        old = [v.double() for v in dw + db]


@pytest.mark.parametrize("M,H,I", [(300, 264, 136), (8200, 72, 2120)])
def test_accumulated_steps_repeat_bit_for_bit(M, H, I):
    print(f"[grad, accumulated] repeats {M}x{H}x{I}", flush=True)
    ops = grad_ops(3, M, H, I, torch.bfloat16)
    got = []
    for _ in range(3):
        dw, db = [torch.ones(I, H, device=DEV) for _ in range(2)], [torch.ones(I, device=DEV) for _ in range(2)]
        moe.gated_linear_backward(*ops, want_dx=False, accumulate=True, dw_gate=dw[0], dw_up=dw[1], dbias_gate=db[0], dbias_up=db[1])
        torch.cuda.synchronize()
        got.append(dw + db)
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(g, got[0]))
