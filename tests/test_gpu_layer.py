"""The operators around the experts step, run together as one layer: row norm with
its MXFP8 output, router logits, routing, routed experts, a shared expert
beside them added into the output. Each stage against the float64 oracle of
its inputs, with the tolerances derived in the operators' own tests; then the
same calls captured, replayed, on other streams and at once, bit for bit."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_02_amd as moe
import oracle
from helpers import TOL, rel_err, to_np
from oracle import layer_ops as L
from test_gpu_forward import ACT_PARAMS, make_problem
from test_gpu_mx_linear import check as check_linear, sums
from test_gpu_norm import check_mx, check_y
from test_gpu_route_topk import TOL as ROUTE_TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
E, K, H, I = 24, 4, 320, 192
ACT = dict(act="swiglu_oai", **ACT_PARAMS["swiglu_oai"], act_fmt="mxfp8")


class Weights:
    def __init__(self):
        g = torch.Generator().manual_seed(5)
        _, _, _, W, S = make_problem(61, 1, H, I, E, K, "mxfp4")
        self.W, self.S = [t.to(DEV) for t in W], [t.to(DEV) for t in S]
        self.norm = (1 + 0.2 * torch.randn(H, generator=g)).bfloat16().to(DEV)
        rows = lambda n, k: (torch.randn(n, k, generator=g) / k ** 0.5).to(DEV)  # noqa: E731
        self.router, self.up, self.down = [moe.mx_quantize(rows(n, k), "mxfp4") for n, k in ((E, H), (I, H), (H, I))]
        self.router_bias = (0.1 * torch.randn(E, generator=g)).to(DEV)
        self.pick_bias = (0.05 * torch.randn(E, generator=g)).to(DEV)


class Layer:
    """One layer's buffers; run() makes no tensor whose address a replay would not know."""

    def __init__(self, w: Weights, T: int):
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
        u8 = lambda *s: e(*s, dtype=torch.uint8)  # noqa: E731
        self.w, self.x, self.res = w, e(T, H), e(T, H)
        self.y, self.codes, self.sc = e(T, H), u8(T, H), u8(T, H // 32)
        self.logits, self.wt = e(T, E, dtype=torch.float32), e(T, K, dtype=torch.float32)
        self.ids = e(T, K, dtype=torch.int32)
        self.hid, self.hc, self.hs = e(T, I), u8(T, I), u8(T, I // 32)
        self.routed, self.out = e(T, H), e(T, H)
        p = moe.problem(T, H, I, E, K, "mxfp4", ACT["act"], ACT["alpha"], ACT["beta"], ACT["limit"], act_fmt="mxfp8")
        self.ws = moe.binding.alloc_workspace(moe.moe_experts_workspace_bytes(p), DEV)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g))
        self.res.copy_(torch.randn(self.x.shape, generator=g))
        return self

    def run(self):
        w = self.w
        moe.add_rmsnorm(self.x, w.norm, residual=self.res, residual_out=self.res, mx="mxfp8", y=self.y, codes=self.codes,
                        scales=self.sc)
        moe.mx_linear(self.codes, self.sc, *w.router, bias=w.router_bias, out=self.logits)
        moe.route_topk(self.logits, K, "sigmoid", bias=w.pick_bias, n_group=4, topk_group=2, routed_scaling_factor=1.5,
                       ids=self.ids, weights=self.wt)
        moe.experts_forward(self.y, self.ids, self.wt, *w.W, scales=w.S, out=self.routed, workspace=self.ws, **ACT)
        moe.mx_linear(self.codes, self.sc, *w.up, out=self.hid)
        moe.mx_quantize(self.hid, "mxfp8", codes=self.hc, scales=self.hs)
        moe.mx_linear(self.hc, self.hs, *w.down, add=self.routed, alpha=0.5, out=self.out)

    def results(self):
        return [t.clone() for t in (self.res, self.y, self.logits, self.ids, self.wt, self.out)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def values(codes, sc, fmt):
    return L.mx_values(codes.cpu().numpy(), sc.cpu().numpy(), fmt)


def check_product(out, a, sc, pair, **kw):
    A, W = values(a, sc, "mxfp8"), values(*pair, "mxfp4")
    extra = sum(np.abs(kw[n]) for n in ("bias", "add") if n in kw)
    check_linear(out, L.mx_linear(A, W, **kw), sums(A, W, a.cpu(), sc.cpu(), pair[0].cpu(), pair[1].cpu(), "mxfp8"),
                 A.shape[1], kw.get("alpha", 1.0), extra)


@pytest.mark.parametrize("T", [1, 7, 33, 700])
def test_stage_by_stage(T):
    print(f"[layer] T={T}", flush=True)
    w = Weights()
    lay = Layer(w, T).fill(T)
    h = (lay.x.float() + lay.res.float()).bfloat16()
    lay.run()
    torch.cuda.synchronize()
    assert torch.equal(lay.res, h)
    y = L.rmsnorm(h.double().cpu().numpy(), w.norm.double().cpu().numpy(), 1e-6)
    check_y(lay.y, y, torch.bfloat16)
    check_mx(lay.codes, lay.sc, y, "mxfp8")
    check_product(lay.logits, lay.codes, lay.sc, w.router, bias=w.router_bias.double().cpu().numpy())
    ids, wt = L.route_topk(lay.logits.cpu().numpy(), K, "sigmoid", bias=w.pick_bias.cpu().numpy(), n_group=4, topk_group=2,
                           routed_scaling_factor=1.5)
    assert np.array_equal(lay.ids.cpu().numpy(), ids)
    assert (np.abs(lay.wt.double().cpu().numpy() - wt) <= ROUTE_TOL * np.abs(wt)).all()
    ref = oracle.experts_forward(to_np(lay.y), ids, wt.astype(np.float32),
                                 *[(c.cpu().numpy(), s.cpu().numpy()) for c, s in zip(w.W, w.S)], **ACT)
    assert rel_err(to_np(lay.routed), ref) <= TOL
    check_product(lay.hid, lay.codes, lay.sc, w.up)
    check_product(lay.out, lay.hc, lay.hs, w.down, alpha=0.5, add=lay.routed.double().cpu().numpy())


@pytest.mark.parametrize("T", [3, 40, 700])
def test_replays_equal_eager_calls(T):
    """A captured layer with new inputs for each replay, eager work of another one between replays."""
    print(f"[layer] graph T={T}", flush=True)
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
        eager.fill(seed + 50).run()                             # on the same weights, behind the replay
        torch.cuda.synchronize()
        assert same(cap.results(), want), f"replay {seed}"


def test_two_graphs_and_two_streams_at_once():
    w = Weights()
    T = 60
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
    for rounds in range(3):
        for by_graph in (True, False):
            for i, lay in enumerate(lays):
                lay.fill(i)
                lay.out.fill_(float("nan"))
            torch.cuda.synchronize()
            for s, lay, g in zip(streams, lays, graphs):
                with torch.cuda.stream(s):
                    g.replay() if by_graph else lay.run()
            torch.cuda.synchronize()
            assert all(same(lay.results(), r) for lay, r in zip(lays, want)), (rounds, by_graph)


def test_calls_run_on_the_current_stream():
    """Inputs that a busy stream writes late: a call on another stream would read what was there before."""
    w, T = Weights(), 16
    lay = Layer(w, T).fill(3)
    lay.run()
    torch.cuda.synchronize()
    want = lay.results()
    lay.fill(3)
    x, res = lay.x.clone(), lay.res.clone()
    lay.x.zero_(), lay.res.zero_()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(10):
            busy @ busy
        lay.x.copy_(x), lay.res.copy_(res)
        lay.run()
    side.synchronize()
    assert same(lay.results(), want)
