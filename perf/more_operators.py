"""Cases of the 16-bit dense projections beside the routed experts: the gated
feed-forward block (gated_linear), its backward pass (gated_linear_backward) and
a projection with low-rank adapters of many requests (lora_linear). Each case
runs either in plain torch operations or, with `own`, through the package's calls
on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
ACT = {"silu": dict(act="silu"), "swiglu_oai": dict(act="swiglu_oai", alpha=1.702, beta=1.0, limit=7.0),
       "situ": dict(act="situ", alpha=1.5, beta=2.0)}


def listed():
    return [
        # a fine-grained layer's shared expert, one token in a decode step
        dict(name="gated_one_token", op="gated", M=1, H=7168, I=2048, dtype="bf16", act="silu", bias=False, save=False),
        # a decode batch with clamped activation and biases, widths that end inside tiles
        dict(name="gated_decode_ragged", op="gated", M=29, H=2880, I=2880, dtype="fp16", act="swiglu_oai", bias=True,
             save=False),
        # a chunk of a prompt: too few large tiles to fill the card
        dict(name="gated_chunk", op="gated", M=300, H=7168, I=2048, dtype="bf16", act="silu", bias=False, save=False),
        # the forward half of a training step on a wide layer: the pre-activations are kept
        dict(name="gated_train", op="gated", M=4096, H=4096, I=14336, dtype="bf16", act="silu", bias=False, save=True),
        # the backward pass of one short sequence, with gradients of the biases
        dict(name="grad_short", op="grad", M=77, H=2880, I=2880, dtype="fp16", act="swiglu_oai", bias=True),
        # a ragged batch through a shared expert
        dict(name="grad_ragged", op="grad", M=1023, H=7168, I=2048, dtype="bf16", act="situ", bias=False),
        # the backward half of the training step
        dict(name="grad_train", op="grad", M=4096, H=4096, I=14336, dtype="bf16", act="silu", bias=False),
        # the down projection of a shared expert for one request with an adapter, added to the routed experts' output
        dict(name="lora_one_token", op="lora", M=1, K=2048, N=7168, R=16, L=8, ids="token", dtype="bf16", w=True,
             bias=False, add=True),
        # a decode batch, a request with an adapter of its own to each token
        dict(name="lora_decode", op="lora", M=64, K=2880, N=2895, R=32, L=32, ids="token", dtype="fp16", w=True,
             bias=True, add=False),
        # adapters alone, onto the result of a projection whose weights are in MXFP4
        dict(name="lora_beside", op="lora", M=256, K=7168, N=7168, R=64, L=16, ids="run", dtype="bf16", w=False,
             bias=False, add=True),
        # tokens of many adapters mixed, and a rank that is no power of two
        dict(name="lora_mixed", op="lora", M=1000, K=4096, N=4096, R=24, L=64, ids="token", dtype="bf16", w=True,
             bias=False, add=False),
        # the prompts of several requests in one prefill
        dict(name="lora_prefill", op="lora", M=8192, K=2048, N=7168, R=64, L=16, ids="run", dtype="bf16", w=True,
             bias=False, add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "grad", "lora", "lora"))
    dtype = rng.choice(("bf16", "fp16"))
    if op != "lora":
        M, H, I = _log(rng, 1, 8192), 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 2048)
        while M * H * I > 4096 * 4096 * 14336:
            M = max(1, M // 2)
        c = dict(op=op, M=M, H=H, I=I, dtype=dtype, act=rng.choice(tuple(ACT)), bias=rng.random() < 0.4)
        if op == "gated":
            c["save"] = rng.random() < 0.4
        return c
    M, K, N = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024), _log(rng, 16, 14336)
    L = _log(rng, 1, 64)
    R = min(rng.choice((8, 16, 24, 32, 64, 128)), 4096 // L // 8 * 8)
    w = rng.random() < 0.75
    while M * (N * K * w + L * R * (N + K)) > 16384 * 2048 * 7168 or M * max(N, L * R) > 8192 * 14336:
        M = max(1, M // 2)
    return dict(op="lora", M=M, K=K, N=N, R=R, L=L, ids=rng.choice(("token", "run")), dtype=dtype, w=w,
                bias=rng.random() < 0.3, add=not w or rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6271 + 29)
    return g


def _rows(g, rows, width, sd=1.0):
    """Normalised hidden rows: normal values, each row at a size of its own, a few channels larger than the rest."""
    x = torch.randn(rows, width, generator=g, device=DEV)
    x *= sd * torch.exp(0.3 * torch.randn(rows, 1, generator=g, device=DEV))
    big = torch.rand(1, width, generator=g, device=DEV) < 0.005
    return torch.where(big, x * 8, x)


def _weights(g, rows, width, dt, gain=1.0):
    return (torch.randn(rows, width, generator=g, device=DEV) * (gain / width ** 0.5)).to(dt)


def _ids(g, case):
    """An adapter to each token, or to each of a few runs of tokens (the requests' prompts); about one in eight has none."""
    M, L = case["M"], case["L"]
    n = M if case["ids"] == "token" else min(M, 2 * L)
    of = torch.randint(-1, L, (n,), generator=g, device=DEV) if L > 6 else torch.randint(0, L, (n,), generator=g, device=DEV)
    of = torch.where(torch.rand(n, generator=g, device=DEV) < (0.1 if n > 1 else 0.0), -1, of.clamp(min=0 if n == 1 else -1))
    if n < M:
        start = torch.randint(0, M, (n - 1,), generator=g, device=DEV).sort().values
        of = of[torch.searchsorted(start, torch.arange(M, device=DEV), right=True)]
    return of.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    dt, M = DT[case["dtype"]], case["M"]
    if case["op"] == "lora":
        K, N, R, L = case["K"], case["N"], case["R"], case["L"]
        return dict(case=case, x=_rows(g, M, K).to(dt), w=_weights(g, N, K, dt) if case["w"] else None,
                    a=_weights(g, L * R, K, dt).view(L, R, K), b=_weights(g, L * N, R, dt, 0.3).view(L, N, R),
                    ids=_ids(g, case), scales=2.0 * torch.rand(L, generator=g, device=DEV) + 0.25,
                    bias=0.3 * torch.randn(N, generator=g, device=DEV) if case["bias"] else None,
                    add=torch.randn(M, N, generator=g, device=DEV).to(dt) if case["add"] else None)
    H, I = case["H"], case["I"]
    s = dict(case=case, x=_rows(g, M, H).to(dt), wg=_weights(g, I, H, dt, 1.5), wu=_weights(g, I, H, dt, 1.5),
             bg=0.3 * torch.randn(I, generator=g, device=DEV) if case["bias"] else None,
             bu=0.3 * torch.randn(I, generator=g, device=DEV) if case["bias"] else None)
    if case["op"] == "grad":
        # what the forward pass kept, and gradients of a loss (scaled up for float16)
        x = s["x"].float()
        s["gate"], s["up"] = [(x @ w.float().t() + (0 if b is None else b)).to(dt)
                              for w, b in ((s["wg"], s["bg"]), (s["wu"], s["bu"]))]
        s["dout"] = _rows(g, M, I, 0.5 if dt == torch.float16 else 0.01).to(dt)
    return s


# ------------------------------------------------------------------ plain forms
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _tanh(v):
    return 1 - 2 / (torch.exp(2 * v) + 1)


def _f(c, g, u):
    a = ACT[c["act"]]
    if c["act"] == "silu":
        return g * _sigmoid(g) * u
    if c["act"] == "situ":
        return a["alpha"] * _tanh(g / a["alpha"]) * _sigmoid(g) * (a["beta"] * _tanh(u / a["beta"]))
    g, u = g.clamp(max=a["limit"]), u.clamp(-a["limit"], a["limit"])
    return g * _sigmoid(a["alpha"] * g) * (u + a["beta"])


def _df(c, g, u):
    """Derivatives of _f by g and by u."""
    a = ACT[c["act"]]
    if c["act"] == "silu":
        s = _sigmoid(g)
        return u * s * (1 + g * (1 - s)), g * s
    if c["act"] == "situ":
        s, tg, tu = _sigmoid(g), _tanh(g / a["alpha"]), _tanh(u / a["beta"])
        return s * (1 - tg * tg + a["alpha"] * tg * (1 - s)) * a["beta"] * tu, a["alpha"] * tg * s * (1 - tu * tu)
    gc, uc = g.clamp(max=a["limit"]), u.clamp(-a["limit"], a["limit"])
    s = _sigmoid(a["alpha"] * gc)
    return ((uc + a["beta"]) * s * (1 + a["alpha"] * gc * (1 - s)) * (g <= a["limit"]),
            gc * s * (u.abs() <= a["limit"]))


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if c["bias"]:
        g, u = g + s["bg"], u + s["bu"]
    out = dict(out=_f(c, g, u).to(s["x"].dtype))
    if c["save"]:
        out.update(gate=g.to(s["x"].dtype), up=u.to(s["x"].dtype))
    return out


def _plain_grad(s):
    c, dt = s["case"], s["x"].dtype
    fg, fu = _df(c, s["gate"].float(), s["up"].float())
    dout, x = s["dout"].float(), s["x"].float()
    dg, du = dout * fg, dout * fu
    out = dict(dx=(dg @ s["wg"].float() + du @ s["wu"].float()).to(dt), dw_gate=(dg.t() @ x).to(dt),
               dw_up=(du.t() @ x).to(dt))
    if c["bias"]:
        out.update(dbias_gate=dg.sum(0), dbias_up=du.sum(0))
    return out


def _plain_lora(s):
    c = s["case"]
    M, N, L, R = c["M"], c["N"], c["L"], c["R"]
    x = s["x"].float()
    t = (x @ s["a"].float().reshape(L * R, -1).t()).view(M, L, R)
    mine = (s["ids"][:, None] == torch.arange(L, device=x.device)).float() * s["scales"]
    y = (t * mine[:, :, None]).view(M, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, N)
    if s["w"] is not None:
        y = y + x @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["x"].dtype)


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return _plain_gated(state) if op == "gated" else _plain_grad(state) if op == "grad" else _plain_lora(state)
    import mixture_experts_expert_02_amd as moe
    if op == "gated":
        r = moe.gated_linear(state["x"], state["wg"], state["wu"], bias_gate=state["bg"], bias_up=state["bu"],
                             save=c["save"], **ACT[c["act"]])
        out = dict(out=r.out)
        if c["save"]:
            out.update(gate=r.gate, up=r.up)
        return out
    if op == "grad":
        r = moe.gated_linear_backward(state["dout"], state["x"], state["wg"], state["wu"], state["gate"], state["up"],
                                      want_dbias=c["bias"], **ACT[c["act"]])
        out = dict(dx=r.dx, dw_gate=r.dw_gate, dw_up=r.dw_up)
        if c["bias"]:
            out.update(dbias_gate=r.dbias_gate, dbias_up=r.dbias_up)
        return out
    return moe.lora_linear(state["x"], state["w"], state["a"], state["b"], state["ids"], state["scales"],
                           bias=state["bias"], add=state["add"])


def work(case):
    M = case["M"]
    if case["op"] == "lora":
        K, N, R, L = case["K"], case["N"], case["R"], case["L"]
        used = min(L, M)
        moved = 2 * (M * K + N * K * case["w"] + used * R * (K + N) + M * N * (2 if case["add"] else 1))
        return {"bytes": moved + 4 * M + 4 * N * case["bias"], "flops": 2 * M * N * K * case["w"] + 2 * M * R * (K + N)}
    H, I = case["H"], case["I"]
    if case["op"] == "gated":
        return {"bytes": 2 * (M * H + 2 * I * H + M * I * (3 if case["save"] else 1)) + 8 * I * case["bias"],
                "flops": 4 * M * H * I + 8 * M * I}
    return {"bytes": 2 * (3 * M * I + 2 * M * H + 4 * I * H) + 8 * I * case["bias"], "flops": 8 * M * H * I + 16 * M * I}


# ------------------------------------------------------------------ 64 bits
def _exact_act(case, g, u):
    """Value and derivatives from the hyperbolic forms, in 64 bits."""
    a = ACT[case["act"]]
    half = lambda v: (1 + torch.tanh(v / 2)) / 2  # noqa: E731
    if case["act"] == "silu":
        p = half(g)
        return g * p * u, (p + g * p * half(-g)) * u, g * p
    if case["act"] == "situ":
        A, B = a["alpha"], a["beta"]
        p, q, r = half(g), torch.tanh(g / A), torch.tanh(u / B)
        return (A * q * p * B * r, (p / torch.cosh(g / A).square() + A * q * p * half(-g)) * B * r,
                A * q * p / torch.cosh(u / B).square())
    top = a["limit"]
    ming, midu = torch.where(g > top, top, g), torch.where(u > top, top, torch.where(u < -top, -top, u))
    p, n = half(a["alpha"] * ming), half(-a["alpha"] * ming)
    in_g, in_u = ~(g > top), ~((u > top) | (u < -top))
    return (ming * p * (midu + a["beta"]), torch.where(in_g, (p + a["alpha"] * ming * p * n) * (midu + a["beta"]), 0.0),
            torch.where(in_u, ming * p, 0.0))


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "gated":
        g, u = [torch.mm(x, w.double().t().contiguous()) for w in (s["wg"], s["wu"])]
        if case["bias"]:
            g, u = g + s["bg"].double(), u + s["bu"].double()
        out = dict(out=_exact_act(case, g, u)[0])
        if case["save"]:
            out.update(gate=g, up=u)
        return out
    if case["op"] == "grad":
        _, fg, fu = _exact_act(case, s["gate"].double(), s["up"].double())
        dgu = torch.cat((fg, fu), 1) * s["dout"].double().repeat(1, 2)
        dw = torch.mm(dgu.t().contiguous(), x)
        out = dict(dx=torch.mm(dgu, torch.cat((s["wg"], s["wu"])).double()), dw_gate=dw[: case["I"]], dw_up=dw[case["I"]:])
        if case["bias"]:
            out.update(dbias_gate=dgu[:, : case["I"]].sum(0), dbias_up=dgu[:, case["I"]:].sum(0))
        return out
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=x.device)
    if s["w"] is not None:
        y += torch.mm(x, s["w"].double().t().contiguous())
    for a in range(case["L"]):
        rows = torch.nonzero(s["ids"] == a).flatten()
        t = torch.mm(x[rows], s["a"][a].double().t().contiguous()) * s["scales"][a].double()
        y.index_add_(0, rows, torch.mm(t, s["b"][a].double().t().contiguous()))
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["add"] is not None:
        y += s["add"].double()
    return y
