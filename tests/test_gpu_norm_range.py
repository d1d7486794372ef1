"""moe_add_rmsnorm on the GPU where its values are large, small or next to a
rounding border, against the float64 oracle, with the tolerances of a kernel that
takes squares, their sum and the root in doubles and carries the products' roundings along.

EPS64 bounds the noise on both sides: a sum of H <= 16384 squares is off by
at most H 2^-53 < 2e-12 relative (halved by the root); the carried roundings are themselves off by a
few 2^-48. A float32 y is then within half a step (2^-24). A 16-bit y comes from h w (exact
beside a 16-bit weight, else 2^-24), the root rounded to float32 (2^-24) and their product (2^-24): 3 2^-24, then its own
half step. A microscaled element is the nearest one to y (ties aside): off by half an element step and no more than
EPS64 |y| beyond it."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FMTS = ["mxfp8", "mxfp4"]
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS64 = 2e-12


def check_y(y, ref):
    f32 = np.abs(ref) * ((1 if y.dtype == torch.float32 else 3.001) * 2.0 ** -24 + EPS64) + 2.0 ** -150
    u, tiny = torch.finfo(y.dtype).eps / 2, torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps / 2
    bound = f32 if y.dtype == torch.float32 else f32 + (np.abs(ref) + f32) * u + tiny
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bound).all(), (err / bound).max()


def check_mx(codes, scales, ref, fmt):
    """Scales equal, elements nearest to ref but for values within EPS64 of a border."""
    sc = scales.cpu().numpy().astype(np.int64)
    _, _, want = L.mx_quantize(ref, fmt)
    top = np.abs(ref).reshape(ref.shape[0], -1, 32).max(-1)
    frac = np.where(top > 0, top / np.ldexp(1.0, np.frexp(top)[1] - 1), 1.5)
    assert ((sc == want) | (np.minimum(frac - 1, 2 - frac) < 2 * EPS64)).all()
    X = np.ldexp(1.0, (sc - 127).astype(np.int32))[..., None]
    got = L.mx_values(codes.cpu().numpy(), scales.cpu().numpy(), fmt).reshape(*X.shape[:2], 32) / X
    v = np.clip(ref.reshape(got.shape) / X, -L.TOP[fmt], L.TOP[fmt])
    over = np.abs(got - v) - L.element_spacing(v, fmt) / 2
    assert (over <= np.abs(v) * EPS64).all(), (over / np.abs(v)).max()


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


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", [(1, 7168), (3, 32), (600, 2880), (530, 5120), (2, 16384), (515, 8224)])
def test_rounded_once(T, H, dtype, fmt):
    g = torch.Generator().manual_seed(T + H)
    x = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dtype)
    w = 1 + 0.3 * torch.randn(H, generator=g)                   # float32: h * w has up to 48 bits
    o = moe.add_rmsnorm(x.to(DEV), w.to(DEV), mx=fmt)
    torch.cuda.synchronize()
    ref = L.rmsnorm(x.double().numpy(), w.double().numpy(), float(np.float32(1e-6)))
    check_y(o.y, ref)
    check_mx(o.codes, o.scales, ref, fmt)


@pytest.mark.parametrize("T", [2, 520])
@pytest.mark.parametrize("size,dtype", [(1e20, torch.float32), (1e20, torch.bfloat16), (1e38, torch.float32),
                                        (1e38, torch.bfloat16), (1e-25, torch.float32), (1e-25, torch.bfloat16),
                                        (1e-37, torch.float32), (1e-40, torch.float32), (1e-38, torch.bfloat16),
                                        (2e4, torch.float16), (1e-6, torch.float16)])
def test_rows_near_the_ends_of_the_range(size, dtype, T):
    """Squares past float32's range, or below it, do not reach y; nor does h * w past it."""
    H = 2080
    g = torch.Generator().manual_seed(T)
    x = (size * torch.randn(T, H, generator=g).clamp(-3, 3)).to(dtype)
    w = 1 + 0.3 * torch.randn(H, generator=g)
    w[5], w[77] = 40.0, 1e-3
    x[0, 5], x[1, 5] = 3 * size, -3 * size
    assert torch.isfinite(x).all() and (x != 0).any(1).all()
    for fmt in FMTS:
        o = moe.add_rmsnorm(x.to(DEV), w.to(DEV), eps=0.0, mx=fmt)
        torch.cuda.synchronize()
        ref = L.rmsnorm(x.double().numpy(), w.double().numpy(), 0.0)
        check_y(o.y, ref)
        check_mx(o.codes, o.scales, ref, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_elements_beside_their_borders(dtype, fmt):
    """Products within 2^-24 of a midpoint between two elements, on either side of it: a y rounded to float32
    before would fall on the midpoint itself, or on its other side."""
    T, H = 24, 256
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.uniform(0.3, 3.0, (T, H)) * rng.choice([-1.0, 1.0], (T, H))).to(dtype)
    grid = np.unique(np.abs(L.E2M1 if fmt == "mxfp4" else L.e4m3_values()[:127]))
    mid = (grid[1:] + grid[:-1])[grid[1:] >= 2.0 ** -6] / 2
    h = x.double().numpy()
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True))
    near = 0
    for t in range(T):                                          # a weight for each row: one call each
        want = rng.choice(mid, H) * 0.25
        want[::32] = 0.25 * 0.8 * 2 * L.TOP[fmt] / 1.75         # fixes the scale of every block
        w = (want / (np.abs(h[t]) * r[t])).astype(np.float32)
        o = moe.add_rmsnorm(x[t:t + 1].to(DEV), torch.from_numpy(w).to(DEV), eps=0.0, mx=fmt)
        torch.cuda.synchronize()
        y = h[t] * w.astype(np.float64) * r[t]
        off = np.abs(np.abs(y) / want - 1)
        assert (off <= 2.0 ** -24 * 1.01).all()
        sure = off > 1e-13
        near += int((sure & (off < 2.0 ** -25)).sum())
        _, elem, code = L.mx_quantize(y[None], fmt)
        assert np.array_equal(o.scales.cpu().numpy(), code)
        c = o.codes.cpu().numpy()[0]
        got = np.stack([L.E2M1[c & 15], L.E2M1[c >> 4]], -1).reshape(-1) if fmt == "mxfp4" else L.e4m3_values()[c]
        assert np.array_equal(got[sure], elem[0][sure])
    assert near > T * H // 4


@pytest.mark.parametrize("T,H", [(2 ** 22 + 5, 8224), (2 ** 23 + 1, 64)])
def test_more_rows_than_a_grid_dimension_holds(T, H):
    """Rows times threads pass 32 bits, offsets too; the rows around the borders are looked at."""
    print(f"[norm] {T}x{H}", flush=True)
    need = T * H * 2.6
    if torch.cuda.mem_get_info()[0] < 1.2 * need:
        pytest.skip("not enough memory")
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    at = [r for b in (0, 2 ** 21, 2 ** 22, T) for r in (b - 2, b - 1, b, b + 1) if 0 <= r < T]
    rows = torch.randn(len(at), H, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[at] = rows.to(DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    o = moe.add_rmsnorm(x, w, want_y=False, mx="mxfp4")
    torch.cuda.synchronize()
    want = moe.add_rmsnorm(rows.to(DEV), w, want_y=False, mx="mxfp4")
    assert torch.equal(o.codes[at], want.codes) and torch.equal(o.scales[at], want.scales)
    check_mx(want.codes, want.scales, L.rmsnorm(rows.double().numpy(), np.ones(H), float(np.float32(1e-6))), "mxfp4")
