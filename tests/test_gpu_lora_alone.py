"""moe_lora_linear without a projection on every way through its two products, and the sorts of many adapters, against the
float64 oracle with the bounds of test_gpu_lora_linear.py."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from lora_alone_cases import ALONE
from test_gpu_lora_linear import DEV, E, T16, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,R,L", ALONE)
@pytest.mark.parametrize("dt", T16)
@pytest.mark.parametrize("ids", ["token", "run"])
@pytest.mark.parametrize("more", [False, True])
def test_adapters_alone(M, K, N, R, L, dt, ids, more):
    """With and without bias and addend (then to a multiple of 8 columns, too); twice, for the same bits."""
    print(f"[lora alone] {M}x{K}x{N} R={R} L={L} {dt} {ids} {more}", flush=True)
    for n in {N, (N + 7) // 8 * 8 if more else N}:
        c = make(M + K + n, M, K, n, R, L, dt, w=False, bias=more, add=more, ids=ids)
        out = moe.lora_linear(**c)
        again = moe.lora_linear(**c)
        torch.cuda.synchronize()
        check(out, c)
        assert torch.equal(out, again)
        if more:
            o = c["add"].clone()
            moe.lora_linear(**{**c, "add": o}, out=o)
            torch.cuda.synchronize()
            assert torch.equal(o, out)


@pytest.mark.parametrize("M,K,N,R,L", [(256, 7168, 264, 64, 3), (1000, 2056, 203, 136, 3), (2100, 4104, 136, 64, 3), (2048, 2056, 330, 128, 3)])
def test_a_broken_adapter_stays_with_its_rows(M, K, N, R, L):
    print(f"[lora alone] broken {M}x{K}x{N} R={R}", flush=True)
    c = make(M, M, K, N, R, L, torch.bfloat16, w=False)
    ref = moe.lora_linear(**c)
    b = {**c, "lora_a": c["lora_a"].clone(), "lora_b": c["lora_b"].clone(), "scales": c["scales"].clone()}
    b["lora_a"][1], b["lora_b"][1], b["scales"][1] = float("nan"), float("inf"), float("inf")
    got = moe.lora_linear(**b)
    torch.cuda.synchronize()
    mine = c["ids"] == 1
    assert torch.equal(got[~mine], ref[~mine]) and got[mine].isnan().all()


def check_rows(got, c):
    """test_gpu_lora_linear.py's bound with every row's own factors gathered: no turn for each of thousands of adapters."""
    x, dt = c["x"].double(), c["x"].dtype
    L, R, K = c["lora_a"].shape
    u = torch.finfo(dt).eps / 2
    on = (c["ids"] >= 0) & (c["ids"] < L)
    a = torch.where(on, c["ids"], 0).long()
    s = torch.where(on, c["scales"][a].double(), 0.0)[:, None]
    A, B = c["lora_a"][a].double(), c["lora_b"][a].double()
    t = s * (x[:, None, :] * A).sum(-1)
    ref = (t[:, None, :] * B).sum(-1)
    T = s * (x[:, None, :] * A).abs().sum(-1)
    top = t.abs().amax(-1, keepdim=True)
    part = u * u * 2 * top + (2.0 ** -24 * top if dt == torch.float16 else 0)
    TB = (T[:, None, :] * B.abs()).sum(-1)
    b = ((((K + 67) * E * T + part)[:, None, :] * B.abs()).sum(-1) + (2 * R + 66) * E * TB) + 8 * E * TB
    if c["w"] is not None:
        W, w = x.abs() @ c["w"].double().abs().t(), x @ c["w"].double().t()
        ref, b = ref + w, b + (K + 66 + 8) * E * W
    b = b * (1 + u) + u * ref.abs() + torch.finfo(dt).smallest_normal * u
    r = ((got.double() - ref).abs() / b).max().item()
    assert torch.isfinite(got).all() and r <= 1, r


@pytest.mark.parametrize("M,L", [(70, 4096), (1000, 319), (1000, 4096), (1024, 512), (1025, 319), (1100, 320), (2000, 1000), (4096, 4096),
                                 (9000, 4095), (9000, 1)])
@pytest.mark.parametrize("w", [True, False])
@pytest.mark.parametrize("ids", ["any", "sorted", "last", "few"])
def test_sorts_of_many_adapters(M, L, w, ids):
    """Both sorts at numbers of adapters around those at which a further wave holds counters, up to the largest: adapters
    all over, in order, the last ones alone, or a few of them far apart."""
    print(f"[lora sort] M={M} L={L} w={w} {ids}", flush=True)
    c = make(M + L, M, 64, 24, 8, L, torch.bfloat16, w=w)
    g = torch.Generator(device=DEV).manual_seed(M * L)
    draw = lambda lo, hi: torch.randint(lo, hi, (M,), generator=g, device=DEV)  # noqa: E731
    i = draw(-1, L + 1)
    if ids == "sorted":
        i = i.sort().values
    elif ids == "last":
        i = draw(max(0, L - 3), L + 1)
    elif ids == "few":
        i = torch.tensor([0, L // 3, L // 2, L - 1], device=DEV)[draw(0, 4)]
    c["ids"] = i.to(torch.int32)
    out = moe.lora_linear(**c)
    again = moe.lora_linear(**c)
    torch.cuda.synchronize()
    check_rows(out, c)
    assert torch.equal(out, again)
