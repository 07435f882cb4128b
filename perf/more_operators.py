"""The operators of a dense feed-forward block around the linear layers, as they are measured.

Three operators that such a block runs one after another:

* norms before and after a block, in one pass over the residual stream with the block's gate and
  the residual's scale, and their gradient;
* the gated projection: both projections of a feed-forward block, the activation and the product,
  and their gradient, from the projections that the forward call kept or from the inputs alone;
* a linear layer with a low-rank adapter of its own for every token (requests of many adapters in
  one batch), with the shared projection in the same call or added to another one's output.

``own`` false computes the operators in elementary torch operations in 32 bits; ``own`` true
calls this repository's operators.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one decoded token between two blocks: the block's output normed, gated and added to the residual
        # stream, the sum normed for the next block (latency counts)
        dict(name="norm_step", op="norm", tokens=1, hidden=7168, post=True, gate="channel", scale=1.0, dtype="bf16"),
        # a large prefill batch there
        dict(name="norm_prefill", op="norm", tokens=16384, hidden=7168, post=True, gate="channel", scale=1.0,
             dtype="bf16"),
        # a training step's gradient there: both norms' weights, the gate, the block's output and the stream
        dict(name="norm_grad", op="norm_grad", tokens=4096, hidden=7168, post=True, gate="channel", scale=1.0,
             dtype="bf16"),
        # the same in fp32 with a gate per token (a conditioned block), a scaled residual, sizes that fill no tile
        dict(name="norm_grad_odd", op="norm_grad", tokens=2047, hidden=1091, post=True, gate="token", scale=0.7071,
             dtype="f32"),
        # one decoded token through an expert-sized gated projection
        dict(name="gated_step", op="gated", tokens=1, k=7168, f=2048, act="silu", keep=False, dtype="bf16"),
        # a prefill batch through it
        dict(name="gated_prefill", op="gated", tokens=8192, k=7168, f=2048, act="silu", keep=False, dtype="bf16"),
        # a small training batch in fp32 out with the projections kept, sizes that fill no tile
        dict(name="gated_odd", op="gated", tokens=333, k=1096, f=1000, act="gelu", keep=True, dtype="f32"),
        # a training step's gradient with the projections kept
        dict(name="gated_grad", op="gated_grad", tokens=4096, k=7168, f=2048, act="silu", keep=True, dtype="bf16"),
        # and from the inputs alone (activations not kept), an odd number of tokens
        dict(name="gated_grad_again", op="gated_grad", tokens=1021, k=1536, f=4096, act="gelu", keep=False,
             dtype="bf16"),
        # a decode batch whose requests use 32 adapters
        dict(name="adapters_step", op="adapters", tokens=48, k=7168, n=7168, rank=16, adapters=32, run=1, add=False,
             bias=False, dtype="bf16"),
        # a prefill batch of packed sequences, each with its request's adapter
        dict(name="adapters_prefill", op="adapters", tokens=8192, k=7168, n=7168, rank=64, adapters=8, run=700,
             add=False, bias=True, dtype="bf16"),
        # adapters beside a projection that another operator computed (8-bit weights), odd sizes
        dict(name="adapters_add", op="adapters", tokens=1021, k=7168, n=1533, rank=24, adapters=12, run=90, add=True,
             bias=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated_grad", "adapters", "adapters"])
    if op in ("norm", "norm_grad"):
        return dict(op=op, tokens=_log(rng, 1, 16384 if op == "norm" else 4096), hidden=_log(rng, 100, 7168),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]),
                    scale=rng.choice([1.0, 0.7071]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gated":
        return dict(op=op, tokens=_log(rng, 1, 8192), k=8 * _log(rng, 16, 896), f=8 * _log(rng, 16, 256),
                    act=rng.choice(["silu", "gelu"]), keep=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gated_grad":
        return dict(op=op, tokens=_log(rng, 16, 4096), k=8 * _log(rng, 16, 896), f=8 * _log(rng, 16, 256),
                    act=rng.choice(["silu", "gelu"]), keep=rng.random() < 0.5, dtype="bf16")
    run = rng.choice([1, 1, _log(rng, 2, 1000)])
    add = rng.random() < 0.3
    return dict(op=op, tokens=_log(rng, 1, 512 if run == 1 else 8192), k=8 * _log(rng, 16, 896),
                n=_log(rng, 100, 7168), rank=8 * rng.randint(1, 8), adapters=_log(rng, 1, 32), run=run, add=add,
                bias=not add and rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f32"]))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _requests(g, tokens, adapters, run):
    """Each token's adapter, -1 for none: sequences of some `run` tokens (1: a decode batch), one in eight of
    which has none."""
    n = max(1, tokens // run)
    ends = torch.randint(0, tokens + 1, (n - 1,), generator=g, device=DEV).sort().values if run > 1 else None
    of = torch.randint(0, adapters, (n if run > 1 else tokens,), generator=g, device=DEV)
    of = torch.where(torch.rand(of.shape, generator=g, device=DEV) < 0.125, -1, of).to(torch.int32)
    return of[torch.searchsorted(ends, torch.arange(tokens, device=DEV), right=True)] if run > 1 else of


def prepare(case, seed):
    g = _gen(seed)
    c = case
    T, dt = c["tokens"], TYPES[c["dtype"]]
    if c["op"] in ("norm", "norm_grad"):
        H = c["hidden"]
        # a residual stream with a few large channels, and weights around 1
        large = 1.0 + 20.0 * (torch.rand(H, generator=g, device=DEV) < 0.002)
        s = dict(case=c, x=(_randn(g, T, H) * large).to(dt), y=(0.5 * _randn(g, T, H)).to(dt),
                 weight=1.0 + 0.1 * _randn(g, H), post=1.0 + 0.1 * _randn(g, H) if c["post"] else None, gate=None)
        if c["gate"] != "none":
            s["gate"] = 0.5 + 0.2 * _randn(g, H) if c["gate"] == "channel" else (0.5 + 0.2 * _randn(g, T, H)).to(dt)
        if c["op"] == "norm_grad":     # (x stands for the stream after the addition, as the forward call returned it)
            s |= dict(dt=_randn(g, T, H).to(dt), dz=_randn(g, T, H).to(dt))
        return s
    K = c["k"]
    x = _randn(g, T, K).to(torch.bfloat16)
    if c["op"] in ("gated", "gated_grad"):
        F = c["f"]
        s = dict(case=c, x=x, w=(_randn(g, 2 * F, K) * K ** -0.5).to(torch.bfloat16))
        if c["op"] == "gated_grad":
            s |= dict(dh=_randn(g, T, F).to(torch.bfloat16), gu=None)
            if c["keep"]:
                s["gu"] = (s["x"].float() @ s["w"].float().t()).to(torch.bfloat16)
        return s
    N, r, L = c["n"], c["rank"], c["adapters"]
    s = dict(case=c, x=x, ids=_requests(g, T, L, c["run"]), a=(_randn(g, L, r, K) * K ** -0.5).to(torch.bfloat16),
             b=(0.2 * _randn(g, L, N, r)).to(torch.bfloat16), scales=(0.5 + torch.rand(L, generator=g, device=DEV)),
             w=None, y=None, bias=_randn(g, N) if c["bias"] else None)
    if c["add"]:
        s["y"] = _randn(g, T, N).to(dt)
    else:
        s["w"] = (_randn(g, N, K) * K ** -0.5).to(torch.bfloat16)
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import fp8_act_quant_amd as fq
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return fq.residual_norm(s["x"], s["y"], s["weight"], post=s["post"], gate=s["gate"], scale=c["scale"], eps=EPS)
    if op == "norm_grad":
        return fq.residual_norm_backward(s["dt"], s["dz"], s["x"], s["y"], s["weight"], post=s["post"], gate=s["gate"],
                                         scale=c["scale"], eps=EPS)
    if op == "gated":
        return fq.gated_linear(s["x"], s["w"], act=c["act"], keep=c["keep"], out_dtype=TYPES[c["dtype"]])
    if op == "gated_grad":
        return fq.gated_linear_backward(s["dh"], s["x"], s["w"], s["gu"], act=c["act"], dw_dtype=torch.bfloat16)
    if c["add"]:
        return fq.adapter_add(s["y"], s["x"], s["a"], s["b"], s["ids"], s["scales"])
    return fq.adapter_linear(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scales"], bias=s["bias"],
                             out_dtype=TYPES[c["dtype"]])


def _inverse_rms(v):
    return torch.rsqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)


def _act(a, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-a))
        return a * p, p * (1.0 + a * (1.0 - p))
    p = 0.5 * torch.erfc(a * -math.sqrt(0.5))
    return a * p, p + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op == "norm":
        y = s["y"].float()
        if s["post"] is not None:
            y = y * _inverse_rms(y) * s["post"]
        if s["gate"] is not None:
            y = y * s["gate"].float()
        t = c["scale"] * s["x"].float() + y
        return t.to(dt), (t * _inverse_rms(t) * s["weight"]).to(dt)
    if op == "norm_grad":
        t, y, dz, gate = s["x"].float(), s["y"].float(), s["dz"].float(), s["gate"]
        r = _inverse_rms(t)
        that = t * r
        dthat = dz * s["weight"]
        d = s["dt"].float() + r * (dthat - that * (dthat * that).mean(-1, keepdim=True))
        dweight = (dz * that).sum(0)
        dpost = dgate = None
        yhat = n = y
        if s["post"] is not None:
            q = _inverse_rms(y)
            yhat = y * q
            n = yhat * s["post"]
        dn = d
        if gate is not None:
            dn = d * gate.float()
            dgate = d * n
            dgate = dgate.to(dt) if gate.dim() == 2 else dgate.sum(0)
        dy = dn
        if s["post"] is not None:
            dpost = (dn * yhat).sum(0)
            dyhat = dn * s["post"]
            dy = q * (dyhat - yhat * (dyhat * yhat).mean(-1, keepdim=True))
        return (c["scale"] * d).to(dt), dy.to(dt), dweight, dpost, dgate
    x = s["x"].float()
    if op in ("gated", "gated_grad"):
        w = s["w"].float()
        gu = x @ w.t() if op == "gated" or s["gu"] is None else s["gu"].float()
        a, b = gu[:, :c["f"]], gu[:, c["f"]:]
        p, dp = _act(a, c["act"])
        if op == "gated":
            h = (p * b).to(dt)
            return (h, gu.to(torch.bfloat16)) if c["keep"] else h
        dh = s["dh"].float()
        d = torch.cat([dh * b * dp, dh * p], -1)
        return (d @ w).to(torch.bfloat16), (d.t() @ x).to(torch.bfloat16)
    L, r, T = c["adapters"], c["rank"], c["tokens"]
    # every adapter's ranks for every token, of which the token's own are kept
    mine = s["ids"][:, None] == torch.arange(L, device=DEV)
    u = (x @ s["a"].float().view(L * r, -1).t()).view(T, L, r)
    u = torch.where(mine[..., None], u * s["scales"][:, None], 0.0)
    y = u.view(T, L * r) @ s["b"].float().permute(0, 2, 1).reshape(L * r, -1)
    if s["y"] is not None:
        return (s["y"].float() + y).to(dt)
    y = y + x @ s["w"].float().t()
    return (y if s["bias"] is None else y + s["bias"]).to(dt)


def work(case):
    c = case
    T, op, size = c["tokens"], c["op"], SIZE[c["dtype"]]
    if op in ("norm", "norm_grad"):
        n = T * c["hidden"]
        vectors = 1 + (1 if c["post"] else 0) + (1 if c["gate"] == "channel" else 0)
        rows = (4 if op == "norm" else 6) + ((1 if op == "norm" else 2) if c["gate"] == "token" else 0)
        return dict(bytes=rows * n * size + 4 * c["hidden"] * vectors * (1 if op == "norm" else 2),
                    flops=(10 if op == "norm" else 24) * n)
    K = c["k"]
    if op == "gated":
        F = c["f"]
        return dict(bytes=2 * T * K + 4 * F * K + T * F * (size + (4 if c["keep"] else 0)), flops=4 * T * F * K)
    if op == "gated_grad":
        F = c["f"]
        return dict(bytes=2 * (T * F + 2 * T * K + 4 * F * K) + (4 * T * F if c["keep"] else 0),
                    flops=(8 if c["keep"] else 12) * T * F * K)
    N, r, L = c["n"], c["rank"], c["adapters"]
    met = L * (1.0 - (1.0 - 0.875 / L) ** max(1, T // c["run"]))     # the adapters that some token uses
    return dict(bytes=2 * T * K + T * N * size * (2 if c["add"] else 1) + 2 * met * r * (K + N) + 4 * T
                + (0 if c["add"] else 2 * N * K) + (4 * N if c["bias"] else 0),
                flops=2 * T * r * (K + N) * 0.875 + (0 if c["add"] else 2 * T * N * K))


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    c, op = case, case["op"]

    def wide(name):
        return None if s[name] is None else s[name].double()

    if op in ("norm", "norm_grad"):
        x, y, weight, post, gate = (wide(n) for n in ("x", "y", "weight", "post", "gate"))
        if op == "norm":
            n = y if post is None else post * y / (y.square().mean(-1, keepdim=True) + EPS).sqrt()
            t = c["scale"] * x + (n if gate is None else gate * n)
            return t, weight * t / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
        # the chain of derivatives, by torch: of the second norm at the stream x, then of what was added to it
        leaves = [v.requires_grad_() for v in (x, y, weight, post, gate) if v is not None]
        z = weight * x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        dx, dweight = torch.autograd.grad(z, (x, weight), s["dz"].double())
        d = dx + s["dt"].double()
        n = y if post is None else post * y / (y.square().mean(-1, keepdim=True) + EPS).sqrt()
        n = n if gate is None else gate * n
        of = [v for v in (y, post, gate) if v is not None]
        got = dict(zip(map(id, of), torch.autograd.grad(n, of, d)))
        del leaves
        return c["scale"] * d, got[id(y)], dweight, got.get(id(post)), got.get(id(gate))
    x = s["x"].double()
    if op in ("gated", "gated_grad"):
        act = torch.nn.functional.silu if c["act"] == "silu" else torch.nn.functional.gelu
        gu = torch.nn.functional.linear(x, s["w"].double()) if op == "gated" or s["gu"] is None else s["gu"].double()
        if op == "gated":
            a, b = gu.chunk(2, dim=-1)
            return (act(a) * b, gu) if c["keep"] else act(a) * b
        gu = gu.requires_grad_()
        a, b = gu.chunk(2, dim=-1)
        d, = torch.autograd.grad(act(a) * b, gu, s["dh"].double())
        return d @ s["w"].double(), d.t() @ x
    # adapter by adapter, its own tokens
    y = s["y"].double() if c["add"] else torch.nn.functional.linear(x, s["w"].double())
    if s["bias"] is not None:
        y = y + s["bias"].double()
    for e in range(c["adapters"]):
        at = (s["ids"] == e).nonzero()[:, 0]
        if at.numel():
            y[at] += s["scales"][e].double() * ((x[at] @ s["a"][e].double().t()) @ s["b"][e].double().t())
    return y
