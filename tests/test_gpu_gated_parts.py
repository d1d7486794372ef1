"""How exactly dg and du enter the products of moe_gated_linear_backward. Bounds: test_gpu_gated_linear.py, with r = u^2
of |dg| where both parts are kept."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from test_gpu_gated_linear import ACTS, T16, check_grads, grad_ops

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
