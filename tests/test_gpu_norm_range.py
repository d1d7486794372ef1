"""moe_add_rmsnorm on the GPU where its values are large, small or next to a
rounding border, against the float64 oracle."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FMTS = ["mxfp8", "mxfp4"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h,w,rest", [
    (1.0, 3e38, 0.0),       # h * w is finite, the root (8) takes the product past float32
    (-1.0, 3e38, 0.0),
    (8.0, 1e38, 0.5),       # h * w itself is past it
    (-8.0, 1e38, 0.5),
])
def test_overflowing_y_is_a_nan_block(h, w, rest, dtype, fmt):
    """y past float32 is an infinity; its block is scale 255 and codes 0, the other block as ever."""
    x = torch.full((2, 64), rest)
    x[0, 3], x[1, 40] = h, -h
    weight = torch.ones(64)
    weight[3] = weight[40] = w
    o = moe.add_rmsnorm(x.to(dtype).to(DEV), weight.to(DEV), eps=0.0, mx=fmt)
    torch.cuda.synchronize()
    y, sc, codes = o.y.cpu().float(), o.scales.cpu(), o.codes.cpu()
    inf = float("inf")
    assert y[0, 3] == (inf if h > 0 else -inf) and y[1, 40] == (-inf if h > 0 else inf)
    assert sc[0, 0] == 255 and sc[1, 1] == 255
    half = codes.shape[1] // 2
    assert (codes[0, :half] == 0).all() and (codes[1, half:] == 0).all()
    ref = L.rmsnorm(x.to(dtype).double().numpy(), weight.double().numpy(), 0.0)
    for row, blk in ((0, 1), (1, 0)):
        _, _, want = L.mx_quantize(ref[row, 32 * blk:32 * blk + 32], fmt)
        assert sc[row, blk] == want[0]
    v = L.mx_values(codes.numpy(), sc.numpy(), fmt)
    assert np.isfinite(v[0, 32:]).all() and np.isfinite(v[1, :32]).all()
