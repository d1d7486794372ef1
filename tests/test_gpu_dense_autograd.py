"""Dense 16-bit projections on tensors that require gradients: the bits of the same call without, a warning, no graph; and inside a
torch.autograd.Function of the user's own, where autograd is off, the gradients of the formulas and no warning."""
import warnings

import pytest
import torch

import mixture_experts_expert_02_amd as moe
from test_gpu_gated_linear import DEV, check_grads, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 90])
def test_calls_warn_and_give_the_same_bits(M):
    x, wg, wu, _, _ = make(1, M, 72, 136, torch.bfloat16)
    want = moe.gated_linear(x, wg, wu).out
    a, b = wg[:16].reshape(2, 8, 72).contiguous(), wu[:, :8].reshape(1, 136, 8).repeat(2, 1, 1).contiguous()
    ids, sc = torch.zeros(M, dtype=torch.int32, device=DEV), torch.ones(2, device=DEV)
    lora = moe.lora_linear(x, wg, a, b, ids, sc)
    with pytest.warns(UserWarning, match="records no autograd graph"):
        got = moe.gated_linear(x, wg.requires_grad_(), wu).out
    with pytest.warns(UserWarning, match="records no autograd graph"):
        got_lora = moe.lora_linear(x, wg, a, b, ids, sc)
    assert not got.requires_grad and torch.equal(got, want) and torch.equal(got_lora, lora)


class Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wg, wu):
        r = moe.gated_linear(x, wg, wu, save=True)
        ctx.save_for_backward(x, wg, wu, r.gate, r.up)
        return r.out

    @staticmethod
    def backward(ctx, d):
        r = moe.gated_linear_backward(d.contiguous(), *ctx.saved_tensors)
        return r.dx, r.dw_gate, r.dw_up


@pytest.mark.parametrize("M", [5, 200])
def test_inside_a_function_of_the_users_own(M):
    leaves = [t.requires_grad_() for t in make(2, M, 136, 264, torch.bfloat16)[:3]]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        d = torch.randn(M, 264, device=DEV).bfloat16()
        Block.apply(*leaves).backward(d)
    x, wg, wu = [t.detach() for t in leaves]
    r = moe.gated_linear(x, wg, wu, save=True)
    check_grads(moe.GatedGrads(*[t.grad for t in leaves], None, None), d, x, wg, wu, r.gate, r.up, "silu", {})
