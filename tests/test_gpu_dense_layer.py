"""The dense 16-bit projections run together as a layer uses them: a shared expert whose down projection
has adapters of many requests, added to the routed experts' output, and a training step through the gated block;
each stage against the float64 oracle of its inputs with the operators' own tolerances, then captured, replayed, on
other streams, at once and on shared workspaces, bit for bit."""
import pytest
import torch

import mixture_experts_expert_02_amd as moe
from mixture_experts_expert_02_amd import binding as B
from oracle import dense16 as O
from test_gpu_gated_linear import ACTS, check_forward, check_grads
from test_gpu_lora_linear import check as check_lora

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
H, I, E, K, R, L = 320, 264, 8, 2, 16, 5
ACT = dict(act="swiglu_oai", **ACTS["swiglu_oai"])


class Weights:
    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(3)
        rn = lambda *s, sd: (sd * torch.randn(*s, generator=g, device=DEV)).bfloat16()  # noqa: E731
        self.gate, self.up, self.down = rn(I, H, sd=H ** -0.5), rn(I, H, sd=H ** -0.5), rn(H, I, sd=I ** -0.5)
        self.experts = [rn(E, 192, H, sd=H ** -0.5), rn(E, 192, H, sd=H ** -0.5), rn(E, H, 192, sd=192 ** -0.5)]
        self.a, self.b = rn(L, R, I, sd=I ** -0.5), rn(L, H, R, sd=0.1)
        self.scales = 0.5 + torch.rand(L, generator=g, device=DEV)
        self.bias = [0.2 * torch.randn(I, generator=g, device=DEV) for _ in range(2)]


def ws_of(size):
    return B.alloc_workspace(size, DEV)


class Layer:
    """Buffers of a step; run() makes no tensor whose address a replay would not know."""

    def __init__(self, w: Weights, T: int, share=None):
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.w, self.T = w, T
        self.x, self.d = e(T, H), e(T, I)
        self.ids, self.topk, self.wt = e(T, dtype=torch.int32), e(T, K, dtype=torch.int32), e(T, K, dtype=torch.float32)
        self.routed, self.hid, self.g, self.u, self.out = e(T, H), e(T, I), e(T, I), e(T, I), e(T, H)
        self.dx, self.dwg, self.dwu = e(T, H), e(I, H, dtype=torch.float32), e(I, H, dtype=torch.float32)
        self.db = [e(I, dtype=torch.float32) for _ in range(2)]
        p = moe.problem(T, H, 192, E, K)
        self.ws = ws_of(moe.moe_experts_workspace_bytes(p))
        f = B.MoeGatedProblem(T, H, I, 0, 1, *[ACT[n] for n in ("alpha", "beta", "limit")])
        sizes = [moe.moe_gated_linear_workspace_bytes(f),
                 moe.moe_gated_linear_backward_workspace_bytes(B.MoeGatedGradProblem(f, B.MOE_T_FP32, 0, 0, 0, 0)),
                 moe.moe_lora_linear_workspace_bytes(B.MoeLoraProblem(T, H, I, R, L, 0))]
        self.dense_ws = share.dense_ws if share is not None else ws_of(max(sizes))

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g))
        self.d.copy_(0.05 * torch.randn(self.d.shape, generator=g))
        self.ids.copy_(torch.randint(-1, L + 1, self.ids.shape, generator=g))
        self.topk.copy_(torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(self.T)]))
        self.wt.copy_(torch.rand(self.wt.shape, generator=g))
        return self

    def run(self):
        w, ws = self.w, self.dense_ws
        kw = dict(bias_gate=w.bias[0], bias_up=w.bias[1])
        moe.experts_forward(self.x, self.topk, self.wt, *w.experts, out=self.routed, workspace=self.ws)
        moe.gated_linear(self.x, w.gate, w.up, out=self.hid, gate=self.g, up=self.u, workspace=ws, **kw, **ACT)
        moe.lora_linear(self.hid, w.down, w.a, w.b, self.ids, w.scales, add=self.routed, out=self.out, workspace=ws)
        moe.gated_linear_backward(self.d, self.x, w.gate, w.up, self.g, self.u, dx=self.dx, dw_gate=self.dwg, dw_up=self.dwu,
                                  dbias_gate=self.db[0], dbias_up=self.db[1], workspace=ws, **ACT)

    def results(self):
        return [t.clone() for t in (self.routed, self.hid, self.g, self.u, self.out, self.dx, self.dwg, self.dwu, *self.db)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


SIZES = [1, 7, 40, 90, 700]


@pytest.mark.parametrize("T", SIZES)
def test_stage_by_stage(T):
    print(f"[dense layer] T={T}", flush=True)
    w = Weights()
    lay = Layer(w, T).fill(T)
    lay.run()
    torch.cuda.synchronize()
    kw = {n: ACT[n] for n in ("alpha", "beta", "limit")}
    check_forward(moe.GatedOut(lay.hid, lay.g, lay.u), lay.x, w.gate, w.up, *w.bias, ACT["act"], kw)
    check_lora(lay.out, dict(x=lay.hid, w=w.down, lora_a=w.a, lora_b=w.b, ids=lay.ids, scales=w.scales, bias=None, add=lay.routed))
    check_grads(moe.GatedGrads(lay.dx, lay.dwg, lay.dwu, *lay.db), lay.d, lay.x, w.gate, w.up, lay.g, lay.u, ACT["act"], kw)


@pytest.mark.parametrize("T", SIZES)
def test_replays_equal_eager_calls(T):
    """New inputs for each replay, eager work on the same weights between replays."""
    print(f"[dense layer] graph T={T}", flush=True)
    w = Weights()
    cap, eager = Layer(w, T).fill(1), Layer(w, T)
    cap.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap.run()
    for seed in range(4):
        eager.fill(seed).run()
        torch.cuda.synchronize()
        want = eager.results()
        cap.fill(seed)
        g.replay()
        eager.fill(seed + 50).run()
        torch.cuda.synchronize()
        assert same(cap.results(), want), f"replay {seed}"


@pytest.mark.parametrize("T", [40, 700])
def test_graphs_that_share_a_workspace_replay_in_turn(T):
    w = Weights()
    one = Layer(w, T)
    lays, want, graphs = [one, Layer(w, T, share=one)], [], []
    for i, lay in enumerate(lays):
        lay.fill(i).run()
        torch.cuda.synchronize()
        want.append(lay.results())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lay.run()
        graphs.append(g)
    for _ in range(3):
        for lay in lays:
            lay.out.fill_(float("nan"))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(same(lay.results(), r) for lay, r in zip(lays, want))


@pytest.mark.parametrize("T", [16, 300])
def test_two_streams_and_two_graphs_at_once(T):
    w = Weights()
    lays, want, graphs = [Layer(w, T) for _ in range(2)], [], []
    for i, lay in enumerate(lays):
        lay.fill(i).run()
        torch.cuda.synchronize()
        want.append(lay.results())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lay.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for by_graph in (True, False):
            for lay in lays:
                lay.out.fill_(float("nan"))
                lay.dwg.fill_(float("nan"))
            torch.cuda.synchronize()
            for s, lay, g in zip(streams, lays, graphs):
                with torch.cuda.stream(s):
                    g.replay() if by_graph else lay.run()
            torch.cuda.synchronize()
            assert all(same(lay.results(), r) for lay, r in zip(lays, want)), by_graph


def test_calls_run_on_the_current_stream():
    """Inputs that a busy stream writes late: a call on another stream would read what was there before."""
    w, T = Weights(), 90
    lay = Layer(w, T).fill(3)
    lay.run()
    torch.cuda.synchronize()
    want = lay.results()
    x, d, ids = lay.x.clone(), lay.d.clone(), lay.ids.clone()
    lay.x.zero_(), lay.d.zero_(), lay.ids.zero_()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(10):
            busy @ busy
        lay.x.copy_(x), lay.d.copy_(d), lay.ids.copy_(ids)
        lay.run()
    side.synchronize()
    assert same(lay.results(), want)


@pytest.mark.parametrize("T", SIZES)
def test_workspaces_hold_nothing_and_are_kept_to(T):
    """Workspaces of exactly the asked-for size between bytes of another pattern, of any contents before the call."""
    print(f"[dense layer] workspace T={T}", flush=True)
    w = Weights()
    lay = Layer(w, T).fill(5)
    lay.run()
    torch.cuda.synchronize()
    want = lay.results()
    f = B.MoeGatedProblem(T, H, I, 0, 1, *[ACT[n] for n in ("alpha", "beta", "limit")])
    sizes = dict(fwd=moe.moe_gated_linear_workspace_bytes(f),
                 bwd=moe.moe_gated_linear_backward_workspace_bytes(B.MoeGatedGradProblem(f, B.MOE_T_FP32, 0, 0, 0, 0)),
                 lora=moe.moe_lora_linear_workspace_bytes(B.MoeLoraProblem(T, H, I, R, L, 0)))
    for byte in (0, 0xFF, 0x7F):
        held = {n: torch.full((256 + s + 4096,), byte, dtype=torch.uint8, device=DEV) for n, s in sizes.items()}
        ws = {n: v[256:256 + sizes[n]] for n, v in held.items()}
        for v in held.values():
            v[:256] = 0x5A
            v[-4096:] = 0x5A
        kw = dict(bias_gate=w.bias[0], bias_up=w.bias[1])
        moe.gated_linear(lay.x, w.gate, w.up, out=lay.hid, gate=lay.g, up=lay.u, workspace=ws["fwd"], **kw, **ACT)
        moe.lora_linear(lay.hid, w.down, w.a, w.b, lay.ids, w.scales, add=lay.routed, out=lay.out, workspace=ws["lora"])
        moe.gated_linear_backward(lay.d, lay.x, w.gate, w.up, lay.g, lay.u, dx=lay.dx, dw_gate=lay.dwg, dw_up=lay.dwu,
                                  dbias_gate=lay.db[0], dbias_up=lay.db[1], workspace=ws["bwd"], **ACT)
        torch.cuda.synchronize()
        assert same(lay.results(), want), byte
        assert all((v[:256] == 0x5A).all() and (v[-4096:] == 0x5A).all() for v in held.values())


def test_too_small_a_workspace_is_refused_before_anything_runs():
    w, T = Weights(), 90
    lay = Layer(w, T).fill(5)
    lay.out.fill_(7.0)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for call in (lambda: moe.lora_linear(lay.x[:, :I], w.down, w.a, w.b, lay.ids, w.scales, out=lay.out, workspace=small),
                 lambda: moe.gated_linear_backward(lay.d, lay.x, w.gate, w.up, lay.d, lay.d, workspace=small)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == B.MOE_ENOSPC
    torch.cuda.synchronize()
    assert (lay.out == 7.0).all()


def test_a_training_step_lowers_the_loss_by_its_gradient():
    """The gradients of a loss of the block's output against differences of the loss along them, in the framework's own
    forward pass (float16, large enough a step that roundings of the output do not hide it)."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T = 64
    x = torch.randn(T, H, generator=g, device=DEV).half()
    wg, wu = [(torch.randn(I, H, generator=g, device=DEV) / H ** 0.5).half() for _ in range(2)]
    d = torch.randn(T, I, generator=g, device=DEV).half()
    r = moe.gated_linear(x, wg, wu, save=True)
    s = moe.gated_linear_backward(d, x, wg, wu, r.gate, r.up)
    loss = lambda a, b, c: (O.gated(a, b, c)[0] * d.double()).sum().item()  # noqa: E731
    for i, gr in enumerate((s.dx, s.dw_gate, s.dw_up)):
        v = gr.double() / gr.double().norm()
        ops = [t.double() for t in (x, wg, wu)]
        h = 1e-4
        up, dn = ([o + t * h * v if j == i else o for j, o in enumerate(ops)] for t in (1, -1))
        num, want = (loss(*up) - loss(*dn)) / (2 * h), (gr.double() * v).sum().item()
        # gate, up, dg, du and the gradients are rounded to 2^-11 of their values, and the difference's own error is h^2
        assert abs(num - want) <= 5 * 2.0 ** -11 * abs(want)
