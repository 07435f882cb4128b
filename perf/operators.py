"""The operators of a routed-expert layer next to the FP8 linear layers, as they are measured.

Three operators that a mixture-of-experts layer runs one after another:

* routing: the gate's logits to each token's experts and their weights, and the gradient;
* placement: the rows (token, expert) put into expert order, and the experts' outputs added
  up per token again, with the gradient;
* products in 8-bit integers, with one scale per token and one per output channel: of one
  weight, and of every expert's weight with its own rows.

``own`` false computes the operators in elementary torch operations in 32 bits; ``own`` true
calls this repository's operators.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decoded token's routing: 256 experts in 8 groups of which 4 are kept, top 8,
        # sigmoid scores with a balance bias (latency counts)
        dict(name="route_one", op="route", tokens=1, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype="f32"),
        # a prefill batch through the same gate
        dict(name="route_prefill", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_score="top2", renormalize=True, scale=2.5, dtype="f32"),
        # softmax scores without groups or bias, bf16 logits, counts that fill no wave or tile
        dict(name="route_softmax_odd", op="route", tokens=5003, experts=72, top_k=6, score="softmax", bias=False,
             groups=1, topk_groups=1, group_score="max", renormalize=False, scale=1.0, dtype="bf16"),
        # a training step's gradient of the gate
        dict(name="route_grad", op="route_grad", tokens=16384, experts=256, top_k=8, score="softmax",
             renormalize=True, scale=2.5, dtype="f32"),
        # a decode batch's rows put into expert order
        dict(name="place_step", op="place", tokens=48, experts=256, top_k=8, first=0, local=256),
        # a prefill batch's, for one GPU's 32 of 256 experts
        dict(name="place_prefill", op="place", tokens=16384, experts=256, top_k=8, first=64, local=32),
        # a prefill batch's expert outputs weighted and added up per token
        dict(name="combine_prefill", op="combine", tokens=8192, experts=256, top_k=8, local=256, hidden=7168,
             dtype="bf16"),
        # its gradient in training, an odd number of tokens
        dict(name="combine_grad", op="combine_grad", tokens=2047, experts=64, top_k=6, hidden=7168, dtype="bf16"),
        # one decoded token through a linear layer with 8-bit weights
        dict(name="linear_one", op="linear", tokens=1, n=7168, k=7168, bias=False, dtype="bf16"),
        # a large prefill batch through it
        dict(name="linear_prefill", op="linear", tokens=16384, n=7168, k=7168, bias=True, dtype="bf16"),
        # a decode batch through the experts' up-projections (expert hidden size 2048, two of them)
        dict(name="experts_step", op="experts", tokens=16, experts=64, top_k=6, n=4096, k=7168, dtype="bf16"),
        # a prefill batch through the experts' up-projections
        dict(name="experts_prefill", op="experts", tokens=2048, experts=64, top_k=6, n=4096, k=7168, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "place", "combine", "combine_grad", "linear", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = rng.randint(8, 32 if groups > 1 else 160)
        topk_groups = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=groups * per, top_k=rng.randint(1, 8),
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_score=rng.choice(["top2", "max"]),
                    renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
    if op == "route_grad":
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=rng.randint(8, 256), top_k=rng.randint(1, 8),
                    score=rng.choice(["sigmoid", "softmax"]), renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
    if op == "place":
        experts = rng.randint(8, 256)
        local = experts if rng.random() < 0.5 else rng.randint(1, experts)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, top_k=rng.randint(1, 8),
                    first=rng.randint(0, experts - local), local=local)
    if op == "combine":
        experts = rng.randint(8, 256)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, top_k=rng.randint(1, 8),
                    local=experts if rng.random() < 0.5 else rng.randint(1, experts), hidden=_log(rng, 100, 7168),
                    dtype=rng.choice(["f32", "bf16"]) if rng.random() < 0.3 else "bf16")
    if op == "combine_grad":
        return dict(op=op, tokens=_log(rng, 1, 2047), experts=rng.randint(8, 256), top_k=rng.randint(1, 6),
                    hidden=_log(rng, 100, 7168), dtype=rng.choice(["f32", "bf16"]) if rng.random() < 0.3 else "bf16")
    if op == "linear":
        return dict(op=op, tokens=_log(rng, 1, 16384), n=_log(rng, 100, 7168), k=16 * _log(rng, 8, 448),
                    bias=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))
    return dict(op=op, tokens=_log(rng, 1, 2048), experts=rng.randint(8, 64), top_k=rng.randint(1, 6),
                n=_log(rng, 100, 4096), k=16 * _log(rng, 8, 448), dtype=rng.choice(["f32", "bf16"]))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _assign(g, tokens, experts, top_k):
    """Each token's experts, [tokens, top_k]: some experts are more popular than others."""
    popular = 0.5 * _randn(g, 1, experts)
    return (_randn(g, tokens, experts) + popular).topk(top_k, dim=-1).indices.to(torch.int32)


def _placement(assigned, experts, first, local):
    """Rows in expert order (tokens ascending within an expert) for experts first .. first +
    local - 1: the rows' bounds by expert, each row's token, each (token, choice)'s row; -1
    where there is none."""
    tokens, top_k = assigned.shape
    flat = assigned.reshape(-1).to(torch.int64) - first
    flat = torch.where((flat < 0) | (flat >= local), torch.full_like(flat, local), flat)
    by, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by, torch.arange(local + 1, device=DEV))
    at = torch.arange(tokens * top_k, device=DEV)
    placed = by < local
    rows = torch.where(placed, order // top_k, -1).to(torch.int32)
    slots = torch.empty(tokens * top_k, dtype=torch.int32, device=DEV)
    slots[order] = torch.where(placed, at, -1).to(torch.int32)
    return offsets, rows, slots.view(tokens, top_k)


def _channel_codes(g, *shape):
    """8-bit weights as a quantiser leaves them (normal, the largest of a channel at 127) and
    their channels' scales."""
    w = _randn(g, *shape).to(torch.bfloat16)
    top = w.abs().amax(-1, keepdim=True).clamp(min=1e-3)
    q = (w * (127.0 / top)).round_().clamp_(-127, 127).to(torch.int8)
    return q, (0.02 / 127.0) * top.squeeze(-1).float()


def prepare(case, seed):
    g = _gen(seed)
    c = case
    T, E = c["tokens"], c.get("experts")
    if c["op"] == "route":
        logits = _randn(g, T, E).to(TYPES[c["dtype"]])
        bias = 0.1 * _randn(g, E) if c["bias"] else None
        return dict(case=c, logits=logits, bias=bias)
    if c["op"] == "route_grad":
        return dict(case=c, logits=_randn(g, T, E).to(TYPES[c["dtype"]]), experts=_assign(g, T, E, c["top_k"]),
                    dweights=_randn(g, T, c["top_k"]))
    if c["op"] == "place":
        return dict(case=c, experts=_assign(g, T, E, c["top_k"]))
    if c["op"] in ("combine", "combine_grad"):
        k, H, dt = c["top_k"], c["hidden"], TYPES[c["dtype"]]
        _, _, slots = _placement(_assign(g, T, E, k), E, 0, c.get("local", E))
        weights = torch.softmax(_randn(g, T, k), -1)
        state = dict(case=c, h=_randn(g, T * k, H).to(dt), slots=slots, weights=weights)
        if c["op"] == "combine_grad":
            state["dy"] = _randn(g, T, H).to(dt)
        return state
    x = _randn(g, T, c["k"]).to(torch.bfloat16)
    if c["op"] == "linear":
        w, ws = _channel_codes(g, c["n"], c["k"])
        return dict(case=c, x=x, w=w, ws=ws, bias=_randn(g, c["n"]) if c["bias"] else None)
    w = torch.empty((E, c["n"], c["k"]), dtype=torch.int8, device=DEV)
    ws = torch.empty((E, c["n"]), device=DEV)
    for e in range(E):
        w[e], ws[e] = _channel_codes(g, c["n"], c["k"])
    assigned = _assign(g, T, E, c["top_k"])
    offsets, rows, _ = _placement(assigned, E, 0, E)
    most = int((offsets[1:] - offsets[:-1]).max())
    return dict(case=c, x=x, w=w, ws=ws, offsets=offsets, rows=rows, most=most)


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import fp8_act_quant_amd as fq
    c = s["case"]
    op = c["op"]
    if op == "route":
        return fq.moe_route(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                            topk_groups=c["topk_groups"], group_score=c["group_score"],
                            renormalize=c["renormalize"], scale=c["scale"])
    if op == "route_grad":
        return fq.moe_route_backward(s["dweights"], s["logits"], s["experts"], score=c["score"],
                                     renormalize=c["renormalize"], scale=c["scale"])
    if op == "place":
        return fq.moe_place(s["experts"], c["local"], first=c["first"])
    if op == "combine":
        return fq.moe_combine(s["h"], s["slots"], s["weights"])
    if op == "combine_grad":
        return fq.moe_combine_backward(s["dy"], s["h"], s["slots"], s["weights"])
    if op == "linear":
        return fq.int8_linear(s["x"], s["w"], s["ws"], s["bias"], out_dtype=TYPES[c["dtype"]])
    q, qs = fq.int8_quant(s["x"])
    return fq.int8_grouped_gemm(q, qs, s["w"], s["ws"], s["offsets"], rows=s["rows"], out_dtype=TYPES[c["dtype"]])


def _scores(logits, kind):
    x = logits.float()
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    # the sum is taken in 64 bits and rounded once, so that no selection depends on its order
    return e / e.double().sum(-1, keepdim=True).float()


def _best(v, k):
    """Indices of the k largest along the last dimension, largest first, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        score = _scores(s["logits"], c["score"])
        choice = score if s["bias"] is None else score + s["bias"]
        if c["groups"] > 1:
            grouped = choice.view(c["tokens"], c["groups"], -1)
            top = torch.sort(grouped, dim=-1, descending=True).values
            value = top[..., 0] + top[..., 1] if c["group_score"] == "top2" else top[..., 0]
            kept = _best(value, c["topk_groups"])
            mask = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
            choice = torch.where(mask[..., None], grouped, float("-inf")).view_as(choice)
        experts = _best(choice, c["top_k"])
        w = score.gather(1, experts)
        if c["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
        return w * c["scale"], experts.to(torch.int32)
    if op == "route_grad":
        score = _scores(s["logits"], c["score"])
        at = s["experts"].long()
        sel, dw = score.gather(1, at), s["dweights"] * c["scale"]
        if c["renormalize"]:
            total = sel.sum(-1, keepdim=True)
            dw = (dw - (dw * sel).sum(-1, keepdim=True) / total) / total
        if c["score"] == "sigmoid":
            dx = torch.zeros_like(score).scatter_(1, at, dw * sel * (1.0 - sel))
        else:
            dx = torch.zeros_like(score).scatter_(1, at, dw)
            dx = score * (dx - (dw * sel).sum(-1, keepdim=True))
        return dx.to(s["logits"].dtype)
    if op == "place":
        return _placement(s["experts"], c["experts"], c["first"], c["local"])
    if op == "combine":
        there = s["slots"] >= 0
        h = s["h"][s["slots"].clamp(min=0).long()].float()
        w = torch.where(there, s["weights"], 0.0)
        return (h * w[..., None]).sum(1).to(s["h"].dtype)
    if op == "combine_grad":
        at = s["slots"].long()
        dy = s["dy"].float()[:, None]
        dweights = (dy * s["h"][at].float()).sum(-1)
        dh = torch.empty_like(s["h"])
        dh[at] = (s["weights"][..., None] * dy).to(dh.dtype)
        return dh, dweights
    x = s["x"].float()
    scale = x.abs().amax(-1, keepdim=True) / 127.0
    q = torch.round(x / torch.where(scale > 0, scale, 1.0))
    if op == "linear":
        y = (q @ s["w"].float().t()) * scale * s["ws"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(TYPES[c["dtype"]])
    # every expert's rows padded to the longest expert's
    offsets, rows, most = s["offsets"], s["rows"].long(), s["most"]
    at = (offsets[:-1, None] + torch.arange(most, device=DEV)).clamp(max=rows.numel() - 1)
    padded = torch.bmm(q[rows[at]], s["w"].float().transpose(1, 2))
    row = torch.arange(rows.numel(), device=DEV)
    e = torch.searchsorted(offsets, row, right=True) - 1
    return (padded[e, row - offsets[e]] * scale[rows] * s["ws"][e]).to(TYPES[c["dtype"]])


def work(case):
    c = case
    T, op = c["tokens"], c["op"]
    if op == "route":
        n = T * c["experts"]
        return dict(bytes=n * SIZE[c["dtype"]] + (4 * c["experts"] if c["bias"] else 0) + 8 * T * c["top_k"],
                    flops=12 * n)
    if op == "route_grad":
        n = T * c["experts"]
        read = n if c["score"] == "softmax" else T * c["top_k"]
        return dict(bytes=(read + n) * SIZE[c["dtype"]] + 8 * T * c["top_k"], flops=12 * read)
    if op == "place":
        return dict(bytes=12 * T * c["top_k"] + 8 * (c["local"] + 1), flops=4 * T * c["top_k"])
    if op == "combine":
        n = T * c["top_k"] * c["local"] // c["experts"] * c["hidden"]
        return dict(bytes=(n + T * c["hidden"]) * SIZE[c["dtype"]] + 8 * T * c["top_k"], flops=2 * n)
    if op == "combine_grad":
        n = T * c["top_k"] * c["hidden"]
        return dict(bytes=(2 * n + T * c["hidden"]) * SIZE[c["dtype"]] + 12 * T * c["top_k"], flops=3 * n)
    if op == "linear":
        return dict(bytes=2 * T * c["k"] + c["n"] * (c["k"] + 4) + T * c["n"] * SIZE[c["dtype"]],
                    flops=2 * T * c["n"] * c["k"])
    rows = T * c["top_k"]
    # the experts that some token picks, were all equally popular
    met = c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** T)
    return dict(bytes=2 * T * c["k"] + met * c["n"] * (c["k"] + 4) + rows * (c["n"] * SIZE[c["dtype"]] + 4),
                flops=2 * rows * c["n"] * c["k"])


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "place":
        return None
    if op in ("route", "route_grad"):
        x = s["logits"].double()
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    if op == "route":
        T, G = c["tokens"], c["groups"]
        choice = p if s["bias"] is None else p + s["bias"].double()
        value = choice.view(T, G, -1).topk(2 if c["group_score"] == "top2" else 1, dim=-1).values.sum(-1)
        out = torch.ones((T, G), dtype=torch.bool, device=DEV).scatter_(1, value.topk(c["topk_groups"]).indices, False)
        choice = choice.masked_fill(out.repeat_interleave(choice.shape[1] // G, dim=1), -math.inf)
        w = p.gather(1, torch.argsort(-choice, dim=-1, stable=True)[:, :c["top_k"]])
        return (c["scale"] * w / (w.sum(-1, keepdim=True) if c["renormalize"] else 1.0), None)
    if op == "route_grad":
        # through the derivative of each step: dL/dp, then dL/dx
        at = s["experts"].long()
        sel, dw = p.gather(1, at), c["scale"] * s["dweights"].double()
        if c["renormalize"]:
            total = sel.sum(-1, keepdim=True)
            jac = torch.eye(c["top_k"], device=DEV, dtype=torch.float64) / total[..., None] \
                - sel[..., None] / (total * total)[..., None]
            dw = (dw[:, None, :] @ jac)[:, 0]
        dp = torch.zeros_like(p).scatter_(1, at, dw)
        if c["score"] == "sigmoid":
            return dp * p * torch.sigmoid(-x)
        return dp * p - p * (dp * p).sum(-1, keepdim=True)
    if op == "combine":
        y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=DEV)
        for j in range(c["top_k"]):
            at = s["slots"][:, j].long()
            y += torch.where(at >= 0, s["weights"][:, j], 0.0).double()[:, None] * s["h"][at.clamp(min=0)].double()
        return y
    if op == "combine_grad":
        dy = s["dy"].double()
        dh = torch.zeros(s["h"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
        for j in range(c["top_k"]):
            at = s["slots"][:, j].long()
            dh.index_copy_(0, at, s["weights"][:, j, None].double() * dy)
            dw[:, j] = torch.linalg.vecdot(dy, s["h"][at].double())
        return dh, dw
    # codes and scales as the 8-bit format defines them: the scale is a 32-bit number, the code
    # the nearest whole number (ties to even) to the 32-bit quotient
    x = s["x"].float()
    scale = x.abs().max(dim=-1, keepdim=True).values / 127.0
    q = torch.where(scale > 0, x / scale, 0.0).round().double()
    a = q * scale.double()
    if op == "linear":
        y = a @ (s["w"].double() * s["ws"].double()[:, None]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    y = torch.empty((s["rows"].numel(), c["n"]), dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    for e in range(c["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            y[lo:hi] = a[s["rows"][lo:hi].long()] @ (s["w"][e].double() * s["ws"][e].double()[:, None]).t()
    return y
