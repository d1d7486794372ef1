"""Tensors that ask for gradients: the dense 16-bit projections record no graph and say so. Without a GPU: every call below is
refused for another reason (an unknown activation, a workspace in host memory) behind the warning."""
import warnings

import pytest
import torch

import mixture_experts_expert_02_amd as moe
from test_dense16_cpu import F32, I32, W, X, t

A, B, IDS, S = t(3, 16, 64), t(3, 9, 16), t(4, dtype=I32), t(3, dtype=F32)


def leaf(*shape, dtype=torch.bfloat16):
    return t(*shape, dtype=dtype).requires_grad_()


def gated(*a, **kw):
    return moe.gated_linear(*a, act="gelu", **kw)


def lora(*a, **kw):
    return moe.lora_linear(*a, workspace=torch.empty(64, dtype=torch.uint8), **kw)


CALLS = [
    lambda: gated(leaf(4, 64), W, W),
    lambda: gated(X, W, leaf(72, 64)),
    lambda: gated(X, W, W, bias_gate=t(72, dtype=F32), bias_up=leaf(72, dtype=F32)),
    lambda: lora(leaf(4, 64), None, A, B, IDS, S),
    lambda: lora(X, leaf(9, 64), A, B, IDS, S),
    lambda: lora(X, None, A, leaf(3, 9, 16), IDS, S),
    lambda: lora(X, None, A, B, IDS, S, add=leaf(4, 9)),
]


@pytest.mark.parametrize("call", CALLS)
def test_a_call_that_autograd_would_record_warns(call):
    with pytest.warns(UserWarning, match="records no autograd graph"), pytest.raises(moe.MoeError):
        call()


@pytest.mark.parametrize("call", CALLS)
def test_none_without_a_graph(call):
    with warnings.catch_warnings(), torch.no_grad(), pytest.raises(moe.MoeError):
        warnings.simplefilter("error")
        call()


@pytest.mark.parametrize("call", [lambda: gated(X, W, W), lambda: lora(X, None, A, B, IDS, S)])
def test_none_without_leaves(call):
    with warnings.catch_warnings(), pytest.raises(moe.MoeError):
        warnings.simplefilter("error")
        call()
