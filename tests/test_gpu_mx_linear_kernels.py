"""Every kernel of moe_mx_linear at sizes that fill its loops, checked on the
GPU in float64.

Tolerance per value: as derived in test_gpu_mx_linear.py. It grows with K, the worst
order of K additions, so the error's root mean square is bounded beside it. A float32
sum of K products of one size, one after the other, each addition off by at most 2^-24
of its partial sum (of size sqrt(i) after i of them), is off by at most
sqrt(sum of i) 2^-24 = K 2^-24 / sqrt(2) in the mean, where the sum itself is of size sqrt(K): below
sqrt(K) 2^-24 relative. Float32 results have to be as good as that; products that are cut (1.5e-5) or left out
are not. 16-bit results round by at most half a step u on top, and MXFP8 rows beside them lose up to 2^-13 of
the largest of eight products (three times their mean size) from each product: 2^-11 covers it."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
import mx_linear_cases as C
from oracle import layer_ops as L
from test_gpu_mx_linear import cut, operands

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


class Product:
    """Operands on the GPU, their float64 product and what the tolerance counts."""

    def __init__(self, seed, M, N, K, fmt):
        ops = operands(seed, M, N, K, fmt)
        A, W = L.mx_values(ops[0].numpy(), ops[1].numpy(), fmt), L.mx_values(ops[2].numpy(), ops[3].numpy(), "mxfp4")
        a, w = torch.from_numpy(A).to(DEV), torch.from_numpy(W).to(DEV).t().contiguous()
        self.dev, self.fmt, self.K = [t.to(DEV) for t in ops], fmt, K
        self.ref, self.S = a @ w, a.abs() @ w.abs()
        self._host = (A, W, ops[0], ops[1], ops[3])
        self._lost = None

    @property
    def lost(self):
        if self._lost is None:
            self._lost = torch.from_numpy(cut(*self._host)).to(DEV) if self.fmt == "mxfp8" else torch.zeros_like(self.S)
        return self._lost

    def check(self, out, alpha=1.0, bias=None, add=None, exact=False):
        dt = out.dtype
        cuts = self.fmt == "mxfp8" and dt != torch.float32 and not exact
        u, tiny = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
        ref, extra = alpha * self.ref, 0.0
        for t in (bias, add):
            if t is not None:
                ref, extra = ref + t.double(), extra + t.double().abs()
        bound = (self.K + 20) * 2.0 ** -23 * (abs(alpha) * self.S + extra)
        if cuts:
            bound = bound + abs(alpha) * self.lost
        bound = ref.abs() * u + bound * (1 + u) + tiny
        err = (out.double() - ref).abs()
        assert torch.isfinite(out).all()
        assert (err <= bound).all(), (err / bound).max().item()
        rms = lambda t: t.square().mean().sqrt().item()  # noqa: E731
        # bias and addend add their own roundings: two more of the result's size
        rel = (self.K ** 0.5 + 2) * 2.0 ** -24 + (2.0 ** -11 if cuts else 0.0)
        limit = rel * (rms(alpha * self.ref) + rms(ref)) + (u * rms(ref) + tiny if dt != torch.float32 else 0.0)
        assert rms(err) <= limit, rms(err) / limit


@pytest.mark.parametrize("fmt,M,N,K", [(f, *s) for f in C.LARGEST for s in C.LARGEST[f]])
def test_largest_tiles(fmt, M, N, K):
    p = Product(M + N + K, M, N, K, fmt)
    for dtype in TYPES[:2] if fmt == "mxfp8" else TYPES:
        print(f"[mx_linear] largest tile {M}x{N}x{K} {fmt} {dtype}", flush=True)
        out = moe.mx_linear(*p.dev, a_fmt=fmt, dtype=dtype)
        torch.cuda.synchronize()
        p.check(out)
