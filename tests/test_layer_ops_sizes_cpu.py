"""Sizes past 32 bits in the operators around the experts step: refused by the
Python entry points, whose problem structures hold 32-bit sizes and would
keep the low bits of a larger one. Tensors without memory stand in for those sizes."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe

BIG = 2 ** 32 + 64                                              # 64 to a 32-bit field


class OnGpu(torch.Tensor):
    def get_device(self):
        return 0


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)


def u8(*shape):
    return t(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("call", [
    lambda: moe.mx_quantize(t(BIG, 32)),
    lambda: moe.mx_quantize(t(1, BIG)),
    lambda: moe.mx_quantize(t(BIG, 64)[:, :32]),
    lambda: moe.mx_dequantize(u8(BIG, 32), u8(BIG, 1), "mxfp8"),
    lambda: moe.mx_dequantize(u8(1, BIG), u8(1, BIG // 32), "mxfp8"),
    lambda: moe.mx_dequantize(u8(1, BIG // 2), u8(1, BIG // 32), "mxfp4"),
    lambda: moe.add_rmsnorm(t(BIG, 8), t(8)),
    lambda: moe.add_rmsnorm(t(1, BIG), t(BIG), mx="mxfp8"),
    lambda: moe.mx_linear(u8(BIG, 32), u8(BIG, 1), u8(4, 16), u8(4, 1)),
    lambda: moe.mx_linear(u8(4, 32), u8(4, 1), u8(BIG, 16), u8(BIG, 1)),
    lambda: moe.mx_linear(u8(1, BIG // 2), u8(1, BIG // 32), u8(4, BIG // 2), u8(4, BIG // 32), a_fmt="mxfp4"),
    lambda: moe.route_topk(t(BIG, 8), 2),
    lambda: moe.route_topk(t(4, BIG), 2),
    lambda: moe.route_topk(t(4, 8), 2 ** 32 + 2),
    lambda: moe.route_topk(t(4, 8), 2, n_group=2 ** 32),
    lambda: moe.route_topk(t(4, 8), 2, n_group=4, topk_group=2 ** 32 + 2),
    lambda: moe.route_topk(t(4, 8), 2, n_group=2.0, topk_group=1),
])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(moe.MoeError):
        call()
