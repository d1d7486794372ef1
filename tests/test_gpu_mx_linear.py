"""moe_mx_linear on the GPU against the float64 oracle.

Tolerance: the products are exact (4 by 2 significant bits and a power of two),
so the error is the accumulation's. Whatever the order, a sum of K terms is K - 1
additions of partial sums that are at most S = sum |a||w| in magnitude; an fp32
addition that truncates (the block-scaled MFMA is not documented to round each of
the additions inside it to nearest) is off by less than 2^-23 of its result,
so the sum is within K * 2^-23 * S (|alpha| S with alpha). At most 16 partial sums
are joined, and alpha, bias and add round once each: 20 more such terms; then
half a step of the output type. (K / 64 in place of K, one rounding per block product
of 64, was the first reading and is too small by this count: one case came
to 2.2 times it.)"""
import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def operands(seed, M, N, K, fmt):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    ws = torch.randint(118, 126, (N, K // 32), generator=g, dtype=torch.uint8)
    if fmt == "mxfp4":
        a = torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8)
    else:
        a = torch.randn(M, K, generator=g).mul(60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    sc = torch.randint(117, 125, (M, K // 32), generator=g, dtype=torch.uint8)
    return a, sc, w, ws


def reference(a, sc, w, ws, fmt, **kw):
    A, W = L.mx_values(a.numpy(), sc.numpy(), fmt), L.mx_values(w.numpy(), ws.numpy(), "mxfp4")
    ref = L.mx_linear(A, W, **kw)
    return ref, np.abs(A) @ np.abs(W).T


def check(out, ref, S, K, alpha=1.0, extra=0.0):
    dt = out.dtype
    u = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * u
    got = out.double().cpu().numpy()
    acc = (K + 20) * 2.0 ** -23 * (abs(alpha) * S + extra)
    bound = np.abs(ref) * u + acc * (1 + u) + tiny
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), (err / bound).max()


SHAPES = [(1, 16, 32), (1, 1, 32), (1, 7168, 2048), (2, 17, 96), (5, 100, 160), (16, 33, 2880), (17, 300, 416),
          (29, 2895, 2880), (32, 64, 7168), (33, 70, 608), (64, 64, 256), (65, 129, 288), (100, 1000, 1056),
          (130, 257, 4128), (300, 513, 544), (513, 640, 1024)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, fmt):
    print(f"[mx_linear] {M}x{N}x{K} {fmt}", flush=True)
    ops = operands(M * 7 + N + K, M, N, K, fmt)
    out = moe.mx_linear(*[t.to(DEV) for t in ops], a_fmt=fmt, dtype=TYPES[(M + N) % 3])
    torch.cuda.synchronize()
    ref, S = reference(*ops, fmt)
    check(out, ref, S, K)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(4096, 1040, 320), (2050, 6400, 288), (1500, 1600, 544)])
def test_many_tiles(M, N, K, fmt):
    """Sizes that take the larger tiles, with ends inside tiles in every direction; checked on the GPU in float64."""
    print(f"[mx_linear] {M}x{N}x{K} {fmt}", flush=True)
    ops = operands(3, M, N, K, fmt)
    out = moe.mx_linear(*[t.to(DEV) for t in ops], a_fmt=fmt, dtype=torch.float32)
    A = torch.from_numpy(L.mx_values(ops[0].numpy(), ops[1].numpy(), fmt)).to(DEV)
    W = torch.from_numpy(L.mx_values(ops[2].numpy(), ops[3].numpy(), "mxfp4")).to(DEV)
    ref = (A @ W.t().contiguous()).cpu().numpy()
    S = (A.abs() @ W.abs().t().contiguous()).cpu().numpy()
    check(out, ref, S, K)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(3, 50, 128), (20, 64, 352), (70, 131, 256), (300, 512, 512)])
def test_alpha_bias_add(M, N, K, fmt, dtype):
    print(f"[mx_linear] epilogue {M}x{N}x{K} {fmt} {dtype}", flush=True)
    ops = operands(11, M, N, K, fmt)
    g = torch.Generator().manual_seed(12)
    bias, add = torch.randn(N, generator=g), (3 * torch.randn(M, N, generator=g)).to(dtype)
    kw = dict(a_fmt=fmt, bias=bias.to(DEV), alpha=-0.37)
    ref, S = reference(*ops, fmt, bias=bias.double().numpy(), add=add.double().numpy(), alpha=np.float64(np.float32(-0.37)))
    extra = np.abs(bias.double().numpy()) + np.abs(add.double().numpy())
    dev = [t.to(DEV) for t in ops]
    out = moe.mx_linear(*dev, add=add.to(DEV), dtype=dtype, **kw)
    torch.cuda.synchronize()
    check(out, ref, S, K, 0.37, extra)
    acc = add.to(DEV).clone()                                   # added in place
    r = moe.mx_linear(*dev, add=acc, out=acc, **kw)
    torch.cuda.synchronize()
    assert r.data_ptr() == acc.data_ptr() and torch.equal(acc, out)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(9, 40, 160), (90, 200, 480)])
def test_strided(M, N, K, fmt):
    print(f"[mx_linear] strided {M}x{N}x{K} {fmt}", flush=True)
    a, sc, w, ws = operands(21, M, N, K, fmt)
    plain = moe.mx_linear(a.to(DEV), sc.to(DEV), w.to(DEV), ws.to(DEV), a_fmt=fmt)
    aw = torch.full((M, a.shape[1] + 48), 0x7F, dtype=torch.uint8, device=DEV)
    aw[:, 16:16 + a.shape[1]] = a.to(DEV)
    sw = torch.full((M, sc.shape[1] + 7), 255, dtype=torch.uint8, device=DEV)
    sw[:, 3:3 + sc.shape[1]] = sc.to(DEV)
    out = torch.full((M + 2, N + 9), 5.0, dtype=torch.bfloat16, device=DEV)
    moe.mx_linear(aw[:, 16:16 + a.shape[1]], sw[:, 3:3 + sc.shape[1]], w.to(DEV), ws.to(DEV), a_fmt=fmt,
                  out=out[1:M + 1, 4:4 + N])
    torch.cuda.synchronize()
    assert torch.equal(out[1:M + 1, 4:4 + N], plain)
    out[1:M + 1, 4:4 + N] = 5.0
    assert (out == 5.0).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M", [4, 200])
def test_nan_scale_stays_in_its_row_and_column(M, fmt):
    N, K = 70, 96
    a, sc, w, ws = operands(31, M, N, K, fmt)
    sc[2, 1] = 255
    ws[69, 2] = 255
    out = moe.mx_linear(a.to(DEV), sc.to(DEV), w.to(DEV), ws.to(DEV), a_fmt=fmt).cpu()
    bad = torch.isnan(out)
    assert bad[2].all() and bad[:, 69].all()
    bad[2] = False
    bad[:, 69] = False
    assert not bad.any()


def test_extreme_scales():
    """Scales at both ends of their range: products that over- or underflow in a
    half of them, exact ones in the others."""
    a, sc, w, ws = operands(41, 4, 32, 128, "mxfp8")
    sc[:], ws[:] = 254, 1
    sc[1], ws[:, 0] = 0, 254
    out = moe.mx_linear(a.to(DEV), sc.to(DEV), w.to(DEV), ws.to(DEV), dtype=torch.float32).cpu()
    A, W = L.mx_values(a.numpy(), sc.numpy(), "mxfp8"), L.mx_values(w.numpy(), ws.numpy(), "mxfp4")
    ref = A @ W.T
    S = np.abs(A) @ np.abs(W).T
    row = 1                                                     # 2^-127 times 2^-126 and 2^127
    check(out[row:row + 1], ref[row:row + 1], S[row:row + 1], 128)


def test_repeat_is_bitwise_the_same_and_rows_are_independent():
    a, sc, w, ws = [t.to(DEV) for t in operands(51, 40, 96, 1024, "mxfp4")]
    one = moe.mx_linear(a, sc, w, ws, a_fmt="mxfp4")
    for _ in range(3):
        assert torch.equal(moe.mx_linear(a, sc, w, ws, a_fmt="mxfp4"), one)
    a2 = a.clone()
    a2[7] ^= 0x33
    two = moe.mx_linear(a2, sc, w, ws, a_fmt="mxfp4")
    keep = torch.arange(40, device=DEV) != 7
    assert torch.equal(one[keep], two[keep])


def test_refusals():
    a, sc, w, ws = [t.to(DEV) for t in operands(61, 4, 32, 128, "mxfp8")]
    bad = [
        ((a, sc, w, ws), dict(a_fmt="mxfp4")), ((a[:, :64], sc, w, ws), {}), ((a, sc[:, :2], w, ws), {}),
        ((a, sc, w, ws[:8]), {}), ((a, sc, w[:, :60], ws), {}), ((a.float(), sc, w, ws), {}),
        ((a, sc, w, ws), dict(bias=torch.zeros(31, device=DEV))), ((a, sc, w, ws), dict(bias=torch.zeros(32))),
        ((a, sc, w, ws), dict(add=torch.zeros(4, 32, device=DEV))),            # float32 beside a bf16 result
        ((a, sc, w, ws), dict(out=torch.zeros(4, 31, device=DEV))), ((a, sc, w, ws), dict(dtype=torch.float64)),
        ((a, sc, w.t().contiguous().t(), ws), {}), ((a.cpu(), sc, w, ws), {}), ((a, sc, w, ws), dict(alpha=float("nan"))),
    ]
    for args, kw in bad:
        with pytest.raises(moe.MoeError):
            moe.mx_linear(*args, **kw)
    assert moe.mx_linear(a[:0], sc[:0], w, ws).shape == (0, 32)
