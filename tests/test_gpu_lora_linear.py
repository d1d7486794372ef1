"""moe_lora_linear on the GPU against the float64 oracle.

Tolerance, element by element, u = half a step of the type, e = 2^-23. Sums as in
test_gpu_gated_linear.py: within acc(K, S) = (K + 66) e S of S = sum |a||b|. An adapter's x A^T is within acc(K, |x||A|),
gets its scale (one rounding) and is carried in two parts of the type over the row's power of two, the second of
which is rounded to half a step of a value that is half a step of the first: p = u^2 of the row's largest for
bfloat16, and for float16 at least its smallest step, 2^-25 of it, as well. The second product adds
acc(2 R, |t||B|). The row's power of two and the additions of the parts, bias and add: 8 more roundings of everything's
magnitude. Then the last rounding."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from dense16_cases import LORA, LORA_LARGE
from oracle import dense16 as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
E = 2.0 ** -23
T16 = [torch.bfloat16, torch.float16]


def make(seed, M, K, N, R, L, dt, w=True, bias=False, add=False, ids="token"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if ids == "token":
        i = torch.randint(-1, L, (M,), generator=g, device=DEV)
    else:
        i = torch.randint(-1, L, (1 + M // 50,), generator=g, device=DEV).repeat_interleave(50)[:M].contiguous()
    return dict(x=rn(M, K).to(dt), w=(rn(N, K) / K ** 0.5).to(dt) if w else None, lora_a=(rn(L, R, K) / K ** 0.5).to(dt),
                lora_b=(0.3 * rn(L, N, R) / R ** 0.5).to(dt), ids=i.to(torch.int32),
                scales=0.25 + 2 * torch.rand(L, generator=g, device=DEV), bias=rn(N) if bias else None,
                add=rn(M, N).to(dt) if add else None)


def bound(c):
    x, dt = c["x"], c["x"].dtype
    M, K = x.shape
    R = c["lora_a"].shape[1]
    u = torch.finfo(dt).eps / 2
    X = x.double().abs()
    y = X.new_zeros(M, c["lora_b"].shape[1])
    mag = y.clone()
    for i in range(c["lora_a"].shape[0]):
        m = (c["ids"] == i).nonzero().flatten()
        s, B = c["scales"][i].double(), c["lora_b"][i].double().abs()
        T = s * (X[m] @ c["lora_a"][i].double().abs().t())
        top = (s * (x[m].double() @ c["lora_a"][i].double().t())).abs().amax(-1, keepdim=True)
        part = u * u * 2 * top + (2.0 ** -24 * top if dt == torch.float16 else 0)
        y[m] += ((K + 67) * E * T + part) @ B.t() + (2 * R + 66) * E * (T @ B.t())
        mag[m] += T @ B.t()
    if c["w"] is not None:
        S = X @ c["w"].double().abs().t()
        y += (K + 66) * E * S
        mag += S
    if c["bias"] is not None:
        mag += c["bias"].double().abs()
    if c["add"] is not None:
        mag += c["add"].double().abs()
    return y + 8 * E * mag


def check(got, c):
    dt = c["x"].dtype
    u = torch.finfo(dt).eps / 2
    ref = O.lora(c["x"], c["w"], c["lora_a"], c["lora_b"], c["ids"], c["scales"], c["bias"], c["add"])
    b = bound(c) * (1 + u) + u * ref.abs() + torch.finfo(dt).smallest_normal * u
    assert torch.isfinite(got).all()
    r = ((got.double() - ref).abs() / b).max().item()
    assert r <= 1, r


SHAPES = LORA


@pytest.mark.parametrize("M,K,N,R,L", SHAPES)
@pytest.mark.parametrize("dt", T16)
def test_shapes(M, K, N, R, L, dt):
    print(f"[lora] {M}x{K}x{N} R={R} L={L} {dt}", flush=True)
    c = make(M + K + N, M, K, N, R, L, dt, w=(M + R // 8) % 3 != 0, bias=N % 2 == 0, add=M % 2 == 1,
             ids="run" if R % 16 == 0 and M % 2 == 0 else "token")
    out = moe.lora_linear(**c)
    torch.cuda.synchronize()
    check(out, c)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("w", [True, False])
def test_in_place_addend_and_strides(M, w):
    """out is add; rows apart in x, w, out and add; what lies between output rows stays."""
    print(f"[lora] strides M={M} w={w}", flush=True)
    K, N = 136, 203
    c = make(11, M, K, N, 16, 5, torch.bfloat16, w=w, bias=True, add=True)
    want = moe.lora_linear(**c)
    check(want, c)

    def wide(t, pad):
        v = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        v[:, : t.shape[1]] = t
        return v[:, : t.shape[1]], v
    for pad in (5, 6, 21):
        o, whole = wide(c["add"], pad)
        s = {**c, "x": wide(c["x"], 8)[0], "w": wide(c["w"], 16)[0] if w else None, "add": o}
        got = moe.lora_linear(**s, out=o)
        torch.cuda.synchronize()
        assert got is o and torch.equal(o, want) and whole[:, N:].isnan().all()


def test_ids_outside_and_no_adapter_at_all():
    print("[lora] ids", flush=True)
    c = make(3, 70, 264, 136, 16, 4, torch.bfloat16, add=True)
    none = {**c, "ids": torch.full_like(c["ids"], -1)}
    base = moe.lora_linear(**none)
    check(base, none)
    ids = c["ids"].clone()
    ids[::5] = 4
    ids[1::5] = -2 ** 31
    ids[2::5] = 2 ** 31 - 1
    c["ids"] = ids
    got = moe.lora_linear(**c)
    torch.cuda.synchronize()
    out = (ids < 0) | (ids >= 4)
    assert torch.equal(got[out], base[out])
    check(got, c)


@pytest.mark.parametrize("M", [5, 90, 400])
def test_a_broken_adapter_stays_with_its_rows(M):
    """Infinities and NaN in one adapter, and in rows without one."""
    print(f"[lora] broken M={M}", flush=True)
    c = make(4, M, 264, 200, 16, 3, torch.bfloat16)
    ref = moe.lora_linear(**c)
    b = {**c, "lora_a": c["lora_a"].clone(), "lora_b": c["lora_b"].clone(), "scales": c["scales"].clone()}
    b["lora_b"][1, ::3] = float("inf")
    b["lora_b"][1, 1::3] = float("nan")
    b["lora_a"][1, 3] = float("nan")
    got = moe.lora_linear(**b)
    torch.cuda.synchronize()
    mine = c["ids"] == 1
    assert torch.equal(got[~mine], ref[~mine])
    assert got[mine].isnan().all()
    unused = {**c, "ids": torch.where(mine, -1, c["ids"])}
    ref = moe.lora_linear(**unused)
    got = moe.lora_linear(**{**b, "ids": unused["ids"]})
    assert torch.equal(got, ref)


def test_float16_parts_hold_large_and_small_products():
    """x A^T beyond float16's ends: its row's power of two carries it."""
    print("[lora] range", flush=True)
    c = make(6, 40, 264, 136, 24, 3, torch.float16)
    for up in (2.0 ** 8, 2.0 ** -8):
        s = {**c, "x": (c["x"].float() * up).half(), "lora_a": (c["lora_a"].float() * up).half(), "w": None, "scales": c["scales"] / up ** 2}
        check(moe.lora_linear(**s), s)
        t = {**s, "scales": c["scales"], "lora_b": (c["lora_b"].float() * 2.0 ** -6).half() if up > 1 else c["lora_b"]}
        check(moe.lora_linear(**t), t)


def test_rows_do_not_depend_on_their_batch():
    """A row's bits are the same whichever adapters the other rows of the call have."""
    print("[lora] batch", flush=True)
    c = make(8, 300, 512, 264, 32, 7, torch.bfloat16)
    whole = moe.lora_linear(**c)
    perm = torch.randperm(300, device=DEV)
    got = moe.lora_linear(**{**c, "x": c["x"][perm].contiguous(), "ids": c["ids"][perm].contiguous()})
    torch.cuda.synchronize()
    assert torch.equal(got, whole[perm])
    for _ in range(3):
        assert torch.equal(moe.lora_linear(**c), whole)


@pytest.mark.parametrize("M,K,N,R,L", LORA_LARGE)
@pytest.mark.parametrize("dt", T16)
@pytest.mark.parametrize("ids", ["token", "run"])
def test_many_rows(M, K, N, R, L, dt, ids):
    print(f"[lora] {M}x{K}x{N} R={R} L={L} {dt} {ids}", flush=True)
    c = make(M + K + N, M, K, N, R, L, dt, w=N != 1100, bias=N % 2 == 0, add=M % 2 == 0, ids=ids)
    out = moe.lora_linear(**c)
    torch.cuda.synchronize()
    check(out, c)


@pytest.mark.parametrize("w", [True, False])
def test_rows_far_apart(w):
    """Rows 2^21 elements apart, so that the last ones lie past 2^32; x then goes in parts of fewer rows."""
    print(f"[lora] far {w}", flush=True)
    M, K, N, dt = 2057, 72, 2056, torch.bfloat16
    base = torch.empty(2064, 1 << 21, dtype=dt, device=DEV)
    at = iter(range(0, 1 << 21, 4096))
    c = make(8, M, K, N, 16, 5, dt, w=w, add=True, bias=True)
    far = {k: None if c[k] is None else base[:c[k].shape[0]].narrow(1, next(at), c[k].shape[1]).copy_(c[k]) for k in ("x", "w", "add")}
    out = base[:M].narrow(1, next(at), N)
    for m in (7, M):
        part = {k: c[k][:m] for k in ("x", "add", "ids")}
        moe.lora_linear(**{**c, **far, "x": far["x"][:m], "add": far["add"][:m], "ids": c["ids"][:m]}, out=out[:m])
        torch.cuda.synchronize()
        check(out[:m], {**c, **part})


@pytest.mark.parametrize("M", [5, 70, 700])
def test_adapters_far_apart(M):
    """Factors of more than 2^32 bytes (of 2^31 values); adapters that no row names hold whatever the memory held."""
    print(f"[lora] large factors {M}", flush=True)
    L, R, K, N, dt = 600, 256, 16392, 14424, torch.float16
    c = make(9, M, K, N, R, 3, dt)
    a, b = [torch.empty(L, *c[k].shape[1:], dtype=dt, device=DEV) for k in ("lora_a", "lora_b")]
    assert a.numel() > 1 << 31 and b.numel() > 1 << 31
    use = torch.tensor([0, 311, L - 1, -1], device=DEV)
    for i in range(3):
        a[use[i]], b[use[i]] = c["lora_a"][i], c["lora_b"][i]
    scales = torch.full((L,), float("nan"), device=DEV)
    scales[use[:3]] = c["scales"]
    got = moe.lora_linear(**{**c, "lora_a": a, "lora_b": b, "scales": scales, "ids": use[c["ids"].long()].to(torch.int32)})
    torch.cuda.synchronize()
    check(got, c)


@pytest.mark.parametrize("M,K,N,R,L", [(1, 2048, 7168, 16, 8), (1, 2048, 7168, 32, 8), (2, 1024, 4500, 16, 3), (2, 2056, 4500, 16, 3),
                                       (1, 4096, 4096, 32, 4), (8, 520, 129, 8, 5), (4, 1000, 200, 16, 2), (4, 8, 4100, 8, 64),
                                       (8, 8, 4100, 8, 64), (1, 72, 5000, 24, 2), (1, 2048, 33, 64, 2), (1, 8, 1, 256, 1)])
@pytest.mark.parametrize("dt", T16)
def test_few_rows_with_their_own_first_products(M, K, N, R, L, dt):
    """Both sides of the rule by which few rows' first products take no launch: rows without an adapter among them, an addend in
    place, and a broken adapter that reaches its own rows alone."""
    print(f"[lora] own {M}x{K}x{N} R={R} {dt}", flush=True)
    c = make(M + K + N + R, M, K, N, R, L, dt, bias=True, add=True)
    c["ids"] = (torch.arange(M, device=DEV, dtype=torch.int32) * 3) % L
    out = moe.lora_linear(**c)
    torch.cuda.synchronize()
    check(out, c)
    o = c["add"].clone()
    moe.lora_linear(**{**c, "add": o}, out=o)
    torch.cuda.synchronize()
    assert torch.equal(o, out)
    ids = c["ids"].clone()
    ids[M // 2:] = torch.tensor([-1, L, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV).repeat(2)[: M - M // 2]
    some = {**c, "ids": ids}
    got = moe.lora_linear(**some)
    torch.cuda.synchronize()
    check(got, some)
    assert torch.equal(got[: M // 2], out[: M // 2])
    if L > 1 and M > 1:
        broken = {**c, "lora_a": c["lora_a"].clone(), "lora_b": c["lora_b"].clone(), "scales": c["scales"].clone()}
        bad = int(c["ids"][0])
        broken["lora_a"][bad], broken["lora_b"][bad], broken["scales"][bad] = float("nan"), float("inf"), float("inf")
        got = moe.lora_linear(**broken)
        torch.cuda.synchronize()
        mine = c["ids"] == bad
        assert torch.equal(got[~mine], out[~mine]) and got[mine].isnan().all()


@pytest.mark.parametrize("M", [70, 700, 2100])
@pytest.mark.parametrize("N", [201, 330, 515])
@pytest.mark.parametrize("w", [True, False])
def test_rows_that_begin_anywhere(M, N, w):
    """Outputs and addends whose rows begin at multiples of 2, 4 and 16 bytes give the same bits, in place too, and what lies
    between the rows stays."""
    print(f"[lora] rows {M}x{N} w={w}", flush=True)
    c = make(M + N, M, 136, N, 24, 5, torch.bfloat16, w=w, bias=True, add=True)
    out = moe.lora_linear(**c)
    torch.cuda.synchronize()
    check(out, c)
    for ld, at in ((N + 8 - N % 8, 0), (N + 2 - N % 2, 0), (N + 4 - N % 2, 2), (N + 5 - N % 2, 1)):
        whole = torch.full((M, ld), float("nan"), dtype=torch.bfloat16, device=DEV)
        o = whole[:, at: at + N]
        o.copy_(c["add"])
        moe.lora_linear(**{**c, "add": o}, out=o)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and whole[:, :at].isnan().all() and whole[:, at + N:].isnan().all()
