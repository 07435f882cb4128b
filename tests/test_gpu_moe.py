"""GPU parity of the routed-expert operators (moe_route, moe_place, moe_combine and their
gradients) against plain implementations in 64 bits.

Tolerances. u = 2^-24 is fp32's unit roundoff. A bf16 result is the rounding of an fp32 one:
where that lies within some bound of the 64-bit value, the result lies between the bf16
roundings of the value's bounds (rounding is monotonic), which is what `within` checks.
  * scores: expf within 2 ulp, an addition and a division: 6 u. Weights: the sum of at most 32
    scores adds 5 levels of u, then a division and a product: within 24 u of the 64-bit value.
  * a choice s + b is within 6 u |s| + u |s + b| of the 64-bit one, so the selection is the
    64-bit selection wherever values differ by more than 1e-6 (scores <= 1, |b| <= 1); where
    they do not, what is selected may differ by no more than that. Equal inputs have equal
    choices in both, and their order is checked exactly.
  * gradients: every term is within 48 u of its magnitude, and the bound sums magnitudes.
  * combine: k products and sums in fp32: within (k + 1) u of sum |w h|.
"""
import numpy as np
import pytest
import torch

import fp8_act_quant_amd as fq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(y, ref, bound):
    """y is (the rounding to its type of) a value within bound of ref."""
    bound = bound + 1e-37
    lo, hi = (ref - bound).to(y.dtype).double(), (ref + bound).to(y.dtype).double()
    if y.dtype == torch.float32:
        lo, hi = ref - bound, ref + bound
    return bool(((y.double() >= lo) & (y.double() <= hi)).all())


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def scores64(x, kind):
    x = x.double()
    if kind == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(-1, keepdim=True)
    e = torch.where(torch.isneginf(x), 0.0, torch.exp(x - torch.where(torch.isneginf(top), 0.0, top)))
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / torch.where(total > 0, total, 1.0), 0.0)


def order64(v, k):
    """The k largest, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def group_value64(c, groups, group_score):
    g = c.view(c.shape[0], groups, -1)
    n = 2 if group_score == "top2" and g.shape[-1] > 1 else 1
    return torch.sort(g, dim=-1, descending=True).values[..., :n].sum(-1)


def weights64(s, idx, renormalize, scale):
    w = s.gather(1, idx.long())
    if renormalize:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return w * scale


def check_route(logits, bias, w, e, top_k, score, groups, topk_groups, group_score, renormalize, scale):
    T, E = logits.shape
    s = scores64(logits, score)
    c = s if bias is None else s + bias.double()
    assert e.dtype == torch.int32 and w.dtype == torch.float32 and e.shape == w.shape == (T, top_k)
    assert int(e.min()) >= 0 and int(e.max()) < E
    assert (torch.sort(e, dim=-1).values.diff(dim=-1) > 0).all(), "an expert twice"
    tol = 1e-6
    if groups > 1:
        value = group_value64(c, groups, group_score)
        limit = torch.sort(value, dim=-1, descending=True).values[:, topk_groups - 1:topk_groups]
        used = value.gather(1, e.long() // (E // groups))
        assert (used >= limit - 2 * tol).all(), "an expert of a group that is not among the best"
        # compare within the groups that are certainly in, where the bound is clear
        nxt = torch.sort(value, dim=-1, descending=True).values
        clear = (nxt[:, topk_groups - 1] - nxt[:, topk_groups] > 2 * tol) if topk_groups < groups else \
            torch.ones(T, dtype=torch.bool, device=c.device)
        kept = (value >= limit).repeat_interleave(E // groups, dim=1)
        c = torch.where(kept, c, -torch.inf)[clear]
        got = e[clear]
    else:
        got = e
    best = torch.sort(c, dim=-1, descending=True).values[:, :top_k]
    mine = c.gather(1, got.long())
    same_inf = torch.isneginf(best) & torch.isneginf(mine)
    assert (same_inf | ((best - mine).abs() <= tol)).all(), float((best - mine).abs().max())
    ref = weights64(s, e, renormalize, scale)
    assert ((w.double() - ref).abs() <= 24 * U * ref.abs() + 1e-37).all(), float(((w - ref).abs() / ref.abs()).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,topk_groups,group_score,biased", [
    (1, 256, 8, 8, 4, "top2", True),
    (1, 1, 1, 1, 1, "max", False),
    (3, 2, 2, 2, 2, "top2", False),
    (67, 72, 6, 1, 1, "max", False),
    (130, 160, 6, 8, 3, "max", False),
    (65, 100, 7, 5, 2, "top2", True),
    (33, 1024, 32, 1, 1, "max", True),
    (9, 1023, 32, 33, 4, "top2", True),
    (257, 64, 4, 64, 5, "top2", False),
    (12, 999, 3, 3, 1, "top2", True),
])
def test_route(T, E, k, groups, topk_groups, group_score, biased, score, dtype):
    g = rng(T * E + k)
    logits = randn(g, T, E).to(DT[dtype])
    bias = 0.2 * randn(g, E).clamp(-4, 4) if biased else None
    for renormalize, scale in ((True, 2.5), (False, 1.0)):
        w, e = fq.moe_route(logits, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups,
                            group_score=group_score, renormalize=renormalize, scale=scale)
        check_route(logits, bias, w, e, k, score, groups, topk_groups, group_score, renormalize, scale)


MANY = [
    # T, E, k, groups, topk_groups, group_score, biased: many tokens, no whole number of waves
    (8193, 256, 8, 8, 4, "top2", True), (8205, 256, 16, 1, 1, "max", False), (4098, 72, 6, 1, 1, "max", False),
    (6147, 160, 6, 8, 3, "max", False), (6150, 130, 7, 2, 1, "top2", True), (2049, 64, 8, 16, 5, "top2", True),
    (2050, 16, 16, 16, 16, "max", False), (2051, 3, 2, 1, 1, "max", True), (6145, 100, 7, 5, 2, "top2", True),
    (8192, 241, 9, 1, 1, "max", True), (2048, 33, 3, 11, 4, "max", False), (4099, 36, 6, 9, 3, "top2", True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,topk_groups,group_score,biased", MANY)
def test_route_many(T, E, k, groups, topk_groups, group_score, biased, score, dtype):
    """Also bit for bit what a few of the tokens alone give (bf16 logits tie often)."""
    g = rng(T * E + k)
    logits = randn(g, T, E).to(DT[dtype])
    bias = 0.2 * randn(g, E).clamp(-4, 4) if biased else None
    kw = dict(score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_score=group_score)
    for renormalize, scale in ((True, 2.5), (False, 1.0)):
        w, e = fq.moe_route(logits, k, renormalize=renormalize, scale=scale, **kw)
        check_route(logits, bias, w, e, k, score, groups, topk_groups, group_score, renormalize, scale)
        for part in (slice(0, 100), slice(T - 37, T)):
            wp, ep = fq.moe_route(logits[part].contiguous(), k, renormalize=renormalize, scale=scale, **kw)
            assert torch.equal(e[part], ep)
            assert torch.equal(w[part], wp)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bits", [0xFFFFFFFF, 0x7FC00000, 0x7F800000])
@pytest.mark.parametrize("T", [9, 8195])
def test_route_experts_in_range_whatever_the_logits(T, bits, score):
    logits = randn(rng(6), T, 250)
    logits.view(torch.int32)[::2] = bits if bits < 1 << 31 else bits - (1 << 32)
    for k, groups, topk_groups, group_score in ((8, 1, 1, "max"), (10, 10, 2, "top2"), (16, 10, 3, "max")):
        _, e = fq.moe_route(logits, k, score=score, groups=groups, topk_groups=topk_groups, group_score=group_score)
        assert 0 <= int(e.min()) and int(e.max()) < 250
        assert bool((torch.sort(e, dim=-1).values.diff(dim=-1) > 0).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_many_masked_and_tied(score):
    """Experts at -inf, rows of one value, large logits and rows with many ties beside ordinary rows."""
    T, E, k = 8195, 256, 8
    logits = randn(rng(5), T, E)
    logits[::7, 40:] = float("-inf")
    logits[1::7] = 0.25
    logits[2::7, 200] = float("inf") if score == "sigmoid" else 50.0
    logits[3::7] = torch.round(logits[3::7])
    logits[4::7] = -100.0
    for groups, topk_groups in ((1, 1), (8, 4)):
        w, e = fq.moe_route(logits, k, score=score, groups=groups, topk_groups=topk_groups)
        for part in (slice(0, 200), slice(T - 300, T)):
            wp, ep = fq.moe_route(logits[part].contiguous(), k, score=score, groups=groups, topk_groups=topk_groups)
            assert torch.equal(e[part], ep) and torch.equal(w[part], wp)
        assert bool((e[1::7] == torch.arange(k, device="cuda", dtype=torch.int32)).all())
        assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_route_ties_go_to_the_lowest_index(groups, topk_groups, score):
    """Logits and biases from a few values far apart: the order is exact, ties and all."""
    g = rng(5)
    T, E, k = 300, 96, 8
    logits = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 8
    w, e = fq.moe_route(logits, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_score="max")
    # scores differ by far more than roundoff, so integer ranks order them: bias first, then logit
    rank = (bias * 10).long() + logits.long()
    if groups > 1:
        per = E // groups
        value = rank.view(T, groups, per).amax(-1)
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order64(value, topk_groups), True)
        rank = torch.where(keep.repeat_interleave(per, dim=1), rank, -1000)
    assert torch.equal(e.long(), order64(rank, k))


def test_route_one_value_everywhere():
    w, e = fq.moe_route(torch.zeros((5, 256), device="cuda"), 8, groups=8, topk_groups=4)
    assert torch.equal(e, torch.arange(8, device="cuda", dtype=torch.int32).expand(5, 8))
    assert torch.equal(w, torch.full((5, 8), 0.125, device="cuda"))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_masked_experts(score):
    """Logits of -inf: score 0, behind every other expert; rows with fewer numbers than top_k
    and with none; the type's lowest value is a number like any other."""
    T, E, k = 6, 20, 4
    logits = randn(rng(1), T, E)
    logits[1, 3:] = -torch.inf
    logits[2] = -torch.inf
    logits[3, ::2] = torch.finfo(torch.float32).min
    logits[4] = torch.finfo(torch.float32).min
    w, e = fq.moe_route(logits, k, score=score)
    check_route(logits, None, w, e, k, score, 1, 1, "max", True, 1.0)
    assert torch.isfinite(w).all()
    assert set(e[1, :3].tolist()) == {0, 1, 2} and e[1, 3] == 3 and w[1, 3] == 0
    assert e[2].tolist() == [0, 1, 2, 3] and (w[2] == 0).all()
    if score == "softmax":
        assert (w[4] == 0.25).all()
    # switched off by the bias instead
    bias = torch.zeros(E, device="cuda")
    bias[:15] = -torch.inf
    w, e = fq.moe_route(randn(rng(2), T, E), k, score=score, bias=bias)
    assert int(e.min()) >= 15
    # NaN is outside the contract, but the experts stay in range and distinct
    logits[:, 5] = torch.nan
    _, e = fq.moe_route(logits, k, score=score)
    assert int(e.min()) >= 0 and int(e.max()) < E


def grad64(logits, idx, dw, score, renormalize, scale):
    """(gradient, bound's magnitude) by the formulas, in 64 bits."""
    s = scores64(logits, score)
    at = idx.long()
    sel, g = s.gather(1, at), dw.double() * scale
    mag = g.abs()
    if renormalize:
        total = sel.sum(-1, keepdim=True)
        mag = (mag + (mag * sel).sum(-1, keepdim=True) / total) / total
        g = (g - (g * sel).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, at, g)
    dm = torch.zeros_like(s).scatter_(1, at, mag)
    if score == "sigmoid":
        return ds * s * (1 - s), dm * s
    return s * (ds - (g * sel).sum(-1, keepdim=True)), s * (dm + (mag * sel).sum(-1, keepdim=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 64, 6), (130, 65, 1), (67, 256, 8), (9, 511, 32), (3, 1024, 16)])
def test_route_backward(T, E, k, score, renormalize, scale, dtype):
    g = rng(T + E)
    logits = randn(g, T, E).to(DT[dtype])
    _, idx = fq.moe_route(logits, k, score=score)
    dw = randn(g, T, k)
    dx = fq.moe_route_backward(dw, logits, idx, score=score, renormalize=renormalize, scale=scale)
    assert dx.dtype == logits.dtype and dx.shape == logits.shape
    ref, mag = grad64(logits, idx, dw, score, renormalize, scale)
    assert within(dx, ref, 48 * U * mag)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(4097, 256, 8), (4098, 255, 8), (4099, 130, 16), (4100, 64, 6), (4111, 7, 3),
                                   (5000, 192, 1)])
def test_route_backward_many(T, E, k, score, dtype):
    """Bit for bit what a few of the tokens alone give (those are checked against the formula)."""
    g = rng(T * E + k)
    logits = randn(g, T, E).to(DT[dtype])
    dw = randn(g, T, k)
    _, idx = fq.moe_route(logits, k, score=score)
    idx[5, 0] = -1
    for renormalize in (True, False):
        dx = fq.moe_route_backward(dw, logits, idx, score=score, renormalize=renormalize, scale=2.5)
        for part in (slice(0, 64), slice(T - 31, T)):
            few = fq.moe_route_backward(dw[part].contiguous(), logits[part].contiguous(), idx[part].contiguous(),
                                        score=score, renormalize=renormalize, scale=2.5)
            assert torch.equal(dx[part], few)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward_against_differences(score):
    """Central differences of the forward pass in 64 bits, selection held: error h^2 f''' / 6
    plus 2^-53 / h, far below the 1e-6 allowed beside the kernel's fp32 bound."""
    T, E, k, h = 4, 24, 5, 1e-4
    logits = randn(rng(3), T, E)
    _, idx = fq.moe_route(logits, k, score=score)
    dw = randn(rng(4), T, k)
    dx = fq.moe_route_backward(dw, logits, idx, score=score, renormalize=True, scale=1.7)

    def loss(x):
        return (weights64(scores64(x, score), idx, True, 1.7) * dw.double()).sum(-1)
    for i in range(E):
        d = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        d[:, i] = h
        num = (loss(logits.double() + d) - loss(logits.double() - d)) / (2 * h)
        assert ((dx[:, i].double() - num).abs() <= 1e-6 + 1e-5 * num.abs()).all()


def test_route_backward_ignores_experts_out_of_range():
    logits = randn(rng(6), 3, 16)
    idx = torch.tensor([[1, 2], [-1, 5], [16, -7]], dtype=torch.int32, device="cuda")
    dx = fq.moe_route_backward(torch.ones((3, 2), device="cuda"), logits, idx, renormalize=False)
    s = torch.sigmoid(logits.double())
    ref = torch.zeros_like(s)
    for t, i in ((0, 1), (0, 2), (1, 5)):
        ref[t, i] = s[t, i] * (1 - s[t, i])
    assert torch.allclose(dx.double(), ref, rtol=1e-5, atol=0)
    assert (dx[2] == 0).all()


def place_ref(assigned, n, first):
    T, k = assigned.shape
    flat = assigned.reshape(-1).astype(np.int64) - first
    ok = (flat >= 0) & (flat < n)
    pairs = np.nonzero(ok)[0]
    order = pairs[np.argsort(flat[pairs], kind="stable")]
    rows = np.full(T * k, -1, np.int32)
    rows[:len(order)] = order // k
    slots = np.full(T * k, -1, np.int32)
    slots[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[pairs], minlength=n))])
    return offsets, rows, slots.reshape(T, k)


@pytest.mark.parametrize("T,k,E,n,first", [
    (1, 1, 1, 1, 0), (1, 8, 256, 256, 0), (48, 8, 256, 256, 0), (511, 8, 256, 32, 64), (513, 8, 1024, 1024, 0),
    (4097, 1, 3, 3, 0), (1366, 3, 37, 12, 20), (5000, 32, 1024, 1000, 24), (16384, 8, 256, 32, 64),
    (70000, 8, 300, 300, 0), (100, 4, 64, 8, 64),
])
def test_place(T, k, E, n, first):
    """Token counts around the single-workgroup limit, chunks that end inside a wave, experts
    nobody picks, choices that are not placed."""
    assigned = torch.randint(0, E, (T, k), generator=rng(T + k), device="cuda", dtype=torch.int32)
    offsets, rows, slots = fq.moe_place(assigned, n, first=first)
    ro, rr, rs = place_ref(assigned.cpu().numpy(), n, first)
    assert offsets.dtype == torch.int64 and rows.dtype == slots.dtype == torch.int32
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(rows.cpu().numpy(), rr)
    assert np.array_equal(slots.cpu().numpy(), rs)


@pytest.mark.parametrize("T", [20, 3000])
def test_place_edge_assignments(T):
    """All pairs of one expert; none placed; negative and huge ids; no tokens."""
    for fill in (0, 7, 8, -1, 2 ** 31 - 1, -2 ** 31):
        assigned = torch.full((T, 3), fill, dtype=torch.int32, device="cuda")
        assigned[T // 2, 1] = 5
        got = fq.moe_place(assigned, 8)
        for a, b in zip(got, place_ref(assigned.cpu().numpy(), 8, 0)):
            assert np.array_equal(a.cpu().numpy(), b)
    offsets, rows, slots = fq.moe_place(torch.empty((0, 3), dtype=torch.int32, device="cuda"), 8)
    assert (offsets == 0).all() and rows.numel() == 0 and slots.shape == (0, 3)


def placed(g, T, k, E, n=None, first=0):
    assigned = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=-1).indices.to(torch.int32)
    return fq.moe_place(assigned, E if n is None else n, first=first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,H,E,n", [(1, 1, 8, 4, 4), (1, 8, 7168, 256, 256), (37, 6, 100, 64, 64), (5, 3, 1, 8, 8),
                                       (19, 9, 2056, 32, 10), (3, 32, 300, 40, 40), (130, 2, 4097, 8, 3), (7, 3, 7, 8, 8), (20, 4, 3, 8, 5),
                                       (300, 3, 1001, 16, 16), (1100, 2, 515, 8, 8)])
def test_combine(T, k, H, E, n, dtype):
    g = rng(T + H)
    _, _, slots = placed(g, T, k, E, n)
    h = randn(g, T * k, H).to(DT[dtype])
    # rows that no slot names are never read
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[slots[slots >= 0].long()] = True
    h[~named] = torch.nan
    for w in (torch.rand((T, k), generator=g, device="cuda"), None):
        y = fq.moe_combine(h, slots, w)
        hs = torch.where(slots[..., None] >= 0, h.double()[slots.clamp(min=0).long()], 0.0)
        wd = torch.ones_like(hs[..., 0]) if w is None else w.double()
        ref = (hs * wd[..., None]).sum(1)
        assert y.dtype == h.dtype and y.shape == (T, H)
        assert within(y, ref, (k + 1) * U * (hs * wd[..., None]).abs().sum(1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,H,E,n", [(1, 1, 8, 4, 4), (37, 6, 7168, 64, 64), (5, 3, 1, 8, 8), (19, 9, 2056, 32, 10),
                                       (3, 32, 300, 40, 40), (130, 2, 4097, 8, 8), (7, 3, 7, 8, 8), (20, 4, 3, 8, 5),
                                       (300, 3, 1001, 16, 16), (1100, 2, 515, 8, 8)])
def test_combine_backward(T, k, H, E, n, dtype):
    g = rng(T + H + 1)
    _, _, slots = placed(g, T, k, E, n)
    h, dy = randn(g, T * k, H).to(DT[dtype]), randn(g, T, H).to(DT[dtype])
    w = torch.rand((T, k), generator=g, device="cuda")
    dh, dw = fq.moe_combine_backward(dy, h, slots, w)
    there = slots >= 0
    hs = torch.where(there[..., None], h.double()[slots.clamp(min=0).long()], 0.0)
    ref_w = (hs * dy.double()[:, None]).sum(-1)
    assert ((dw.double() - ref_w).abs() <= (H + 1) * U * (hs * dy.double()[:, None]).abs().sum(-1) + 1e-37).all()
    ref_h = w.double()[..., None] * dy.double()[:, None]
    assert within(dh[slots[there].long()], ref_h[there], U * ref_h[there].abs())
    # and against differences of the forward pass, which is linear in w and in h
    loss = lambda hh, ww: (torch.where(there[..., None], hh[slots.clamp(min=0).long()], 0.0) * ww[..., None]  # noqa: E731
                           * dy.double()[:, None]).sum()
    d = torch.zeros_like(w, dtype=torch.float64)
    d[T // 2, k // 2] = 0.5
    num = loss(h.double(), w.double() + d) - loss(h.double(), w.double() - d)
    assert abs(float(dw[T // 2, k // 2]) - float(num)) <= 1e-4 * H ** 0.5


def test_offsets_past_32_bits():
    """Rows, tokens and logits whose elements are more than 2^32: the last of each."""
    g = rng(11)
    T, k, H = 40000, 8, 14336
    h = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    h[-64:] = randn(g, 64, H).bfloat16()
    slots = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k)
    w = randn(g, T, k)
    y = fq.moe_combine(h, slots, w)
    ref = (w[-8:, :, None].double() * h[-64:].view(8, k, H).double()).sum(1)
    mag = (w[-8:, :, None].double() * h[-64:].view(8, k, H).double()).abs().sum(1)
    assert not bool(y[:-8].any())
    lo, hi = (ref - 16 * U * mag).bfloat16(), (ref + 16 * U * mag).bfloat16()
    assert bool(((y[-8:] >= lo) & (y[-8:] <= hi)).all())
    dy = randn(g, T, H).bfloat16()
    dh, dw = fq.moe_combine_backward(dy, h, slots, w)
    assert torch.equal(dh[-k:], (w[-1][:, None] * dy[-1].float()).bfloat16())
    ref = (h[-64:].view(8, k, H).double() * dy[-8:, None].double()).sum(-1)
    mag = (h[-64:].view(8, k, H).double() * dy[-8:, None].double()).abs().sum(-1)
    assert bool(((dw[-8:] - ref).abs() <= H * U * mag).all()) and not bool(dw[:-8].any())
    del h, dh, dy, y
    T, E = 4200000, 1024
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    logits[-5:] = randn(g, 5, E).bfloat16()
    for n in (E, 250):   # (a wave to a token, and 16 lanes)
        part = logits if n == E else logits.view(-1)[:T * E // n * n].view(-1, n)[-(1 << 24) + 1:]
        wp, ep = fq.moe_route(part, 4)
        wl, el = fq.moe_route(part[-9:].contiguous(), 4)
        assert torch.equal(ep[-9:], el) and torch.equal(wp[-9:], wl)
        assert bool((ep[:100] == torch.arange(4, device="cuda", dtype=torch.int32)).all())
    dx = fq.moe_route_backward(wp, part, ep)
    assert torch.equal(dx[-9:], fq.moe_route_backward(wl, part[-9:].contiguous(), el))


def test_gather_gradient_is_combine_without_weights():
    """x[rows]'s gradient: each token's rows of it, added up."""
    g = rng(9)
    T, k, H, E = 50, 4, 264, 16
    _, rows, slots = placed(g, T, k, E)
    d = randn(g, T * k, H)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, rows.long(), d.double())
    assert torch.allclose(fq.moe_combine(d, slots).double(), ref, rtol=0, atol=5 * U * 20)


def test_unaligned_rows_and_other_streams():
    """Views that start off a 16-byte boundary take the element-wise variant and give the same
    values; calls on another stream run there."""
    g = rng(11)
    T, k, H = 20, 3, 64
    _, _, slots = placed(g, T, k, 8)
    w = torch.rand((T, k), generator=g, device="cuda")
    buf = randn(g, T * k * H + 1).to(torch.bfloat16)
    h = buf[1:].view(T * k, H)
    assert torch.equal(fq.moe_combine(h, slots, w), fq.moe_combine(h.clone(), slots, w))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = fq.moe_combine(h, slots, w)
        ww, ee = fq.moe_route(randn(rng(1), 9, 33).to(torch.bfloat16).view(-1)[:9 * 33].view(9, 33), 2)
    st.synchronize()
    assert torch.equal(y, fq.moe_combine(h, slots, w)) and int(ee.max()) < 33


def test_repeated_calls_give_the_same_bits():
    g = rng(12)
    logits = randn(g, 3000, 256)
    a = fq.moe_route(logits, 8, groups=8, topk_groups=4)
    b = fq.moe_route(logits, 8, groups=8, topk_groups=4)
    pa, pb = fq.moe_place(a[1], 256), fq.moe_place(b[1], 256)
    h = randn(g, 24000, 128)
    dy = randn(g, 3000, 128)
    ca, cb = (fq.moe_combine_backward(dy, h, p[2], r[0]) for p, r in ((pa, a), (pb, b)))
    for x, y in zip((*a, *pa, *ca), (*b, *pb, *cb)):
        assert torch.equal(x, y)


def test_empty_calls():
    z = torch.empty((0, 16), device="cuda")
    w, e = fq.moe_route(z, 2)
    assert w.shape == e.shape == (0, 2)
    assert fq.moe_route_backward(w, z, e).shape == (0, 16)
    slots = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    y = fq.moe_combine(torch.empty((0, 16), device="cuda"), slots, torch.ones((3, 2), device="cuda"))
    assert (y == 0).all()
    dh, dw = fq.moe_combine_backward(torch.ones((3, 16), device="cuda"), torch.empty((0, 16), device="cuda"), slots,
                                     torch.ones((3, 2), device="cuda"))
    assert dh.shape == (0, 16) and (dw == 0).all()
    assert fq.moe_combine(torch.empty((6, 0), device="cuda"), slots).shape == (3, 0)


def test_refusals():
    x = torch.zeros((4, 16), device="cuda")
    i = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    for bad in (dict(top_k=0), dict(top_k=17), dict(top_k=2, groups=3), dict(top_k=2, groups=4, topk_groups=5),
                dict(top_k=5, groups=4, topk_groups=1), dict(top_k=2, score="relu"), dict(top_k=2, group_score="sum"),
                dict(top_k=2, bias=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            fq.moe_route(x, **bad)
    with pytest.raises(TypeError):
        fq.moe_route(x.half(), 2)
    with pytest.raises(TypeError):
        fq.moe_route(x, 2, bias=torch.zeros(16, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        fq.moe_route(x.cpu(), 2)
    with pytest.raises(ValueError):
        fq.moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        fq.moe_route(torch.zeros((1, 1025), device="cuda"), 2)
    with pytest.raises(TypeError):
        fq.moe_route_backward(w, x, i.long())
    with pytest.raises(ValueError):
        fq.moe_route_backward(w[:3], x, i)
    with pytest.raises(TypeError):
        fq.moe_place(i.long(), 8)
    with pytest.raises(ValueError):
        fq.moe_place(i, 0)
    with pytest.raises(ValueError):
        fq.moe_place(i, 8, first=-1)
    with pytest.raises(fq.Fp8qError):   # refused by the library itself
        fq.moe_place(i, 8, first=2 ** 31)
    with pytest.raises(ValueError):
        fq.moe_place(i, 8, first=2 ** 70)
    with pytest.raises(TypeError):
        fq.moe_route(x, 2.5)
    with pytest.raises(TypeError):
        fq.moe_combine([1.0], i, w)
    h = torch.zeros((8, 32), device="cuda")
    with pytest.raises(ValueError):
        fq.moe_combine(h, i, w[:3])
    with pytest.raises(TypeError):
        fq.moe_combine(h.half(), i, w)
    with pytest.raises(ValueError):
        fq.moe_combine(h, i, w, out=torch.zeros((4, 31), device="cuda"))
    with pytest.raises(ValueError):
        fq.moe_combine_backward(torch.zeros((3, 32), device="cuda"), h, i, w)
    with pytest.raises(TypeError):
        fq.moe_combine_backward(torch.zeros((4, 32), device="cuda").bfloat16(), h, i, w)


def overlapped(H, dtype):
    """The columns that the last 16-byte piece of a row of H elements shares with the piece before, the first and the last."""
    n = 4 if dtype == "f32" else 8
    return [*range(H - n, H // n * n), 0, H - 1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(5, 1447), (300, 515), (1100, 515), (3, 10), (7, 1448)])
def test_combine_backward_of_infinities(T, H, dtype):
    """An infinity in a row of h, or in dy, gives the dot product that the definition has: an infinity
    of its sign wherever it stands (each element counts once), and numbers elsewhere."""
    g = rng(T + H)
    k = 3
    _, _, slots = placed(g, T, k, 8)
    w = torch.rand((T, k), generator=g, device="cuda")
    at = slots.long()
    for col in overlapped(H, dtype):
        for sign in (1.0, -1.0):
            h, dy = randn(g, T * k, H).to(DT[dtype]), randn(g, T, H).to(DT[dtype])
            h[at[T // 2, 1], col] = sign * torch.inf
            dh, dw = fq.moe_combine_backward(dy, h, slots, w)
            terms = h.double()[at] * dy.double()[:, None]
            ref, mag = terms.sum(-1), terms.abs().sum(-1)
            there = torch.isfinite(ref)
            assert int((~there).sum()) == 1 and torch.equal(dw[~there].double(), ref[~there]), (col, sign)
            assert ((dw.double() - ref).abs()[there] <= (H + 1) * U * mag[there]).all()
            assert torch.isfinite(dh).all()
            h[at[T // 2, 1], col] = 1.0
            dy[0, col] = sign * torch.inf
            dw = fq.moe_combine_backward(dy, h, slots, w)[1]
            assert torch.equal(dw[0].double(), (h.double()[at[0]] * dy[0].double()).sum(-1)), (col, sign)
            assert torch.isfinite(dw[1:]).all()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(9, 24, 5), (4100, 24, 5), (4100, 256, 8), (5, 1024, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward_of_small_scores(T, E, k, score, renormalize):
    """Selected scores near fp32's smallest numbers, whose sum has no reciprocal there: the gradient of the
    renormalised weights is an ordinary number (each score over the sum is).

    Bound: such a score, down to 2^-127.4, is off by expf's 2 ulp (2^-148) and a rounding (2^-150): within
    2^-20.2 = 14 u of its value; score over sum within 3 * 14 u + 8 u, the difference from the mean within
    2 * 50 u, their product and its sum within 160 u of the magnitudes."""
    g = rng(T + E + k)
    logits = -88.3 + 1.5 * torch.rand((T, E), generator=g, device="cuda")
    idx = torch.rand((T, E - 1), generator=g, device="cuda").topk(k, dim=-1).indices.to(torch.int32)
    if score == "softmax":
        logits[:, -1] = 0.0
    dw = 8.0 * randn(g, T, k)
    dx = fq.moe_route_backward(dw, logits, idx, score=score, renormalize=renormalize, scale=2.5)
    ref, mag = grad64(logits, idx, dw, score, renormalize, 2.5)
    assert torch.isfinite(dx).all()
    assert ((dx.double() - ref).abs() <= 160 * U * mag + 1e-37).all()
    if renormalize:
        assert float(ref.abs().max()) > 0.1


@pytest.mark.parametrize("dtype,H", [("bf16", 7161), ("f32", 7161), ("f32", 7168), ("bf16", 7168)])
def test_combine_of_more_rows_than_the_caches_hold(H, dtype):
    """Over 256 MB of rows, whose lengths are whole 16-byte pieces or not."""
    g = rng(H)
    T, k, E = 2401, 8, 64
    _, _, slots = placed(g, T, k, E, 60)
    h, dy = randn(g, T * k, H).to(DT[dtype]), randn(g, T, H).to(DT[dtype])
    w = torch.rand((T, k), generator=g, device="cuda")
    y = fq.moe_combine(h, slots, w)
    dh, dw = fq.moe_combine_backward(dy, h, slots, w)
    ref, mag = torch.zeros((2, T, H), dtype=torch.float64, device="cuda")
    for j in range(k):
        there = slots[:, j] >= 0
        hj = torch.where(there[:, None], h[slots[:, j].clamp(min=0).long()].double(), 0.0)
        term = w[:, j, None].double() * hj
        ref += term
        mag += term.abs()
        dot = hj * dy.double()
        assert ((dw[:, j].double() - dot.sum(-1)).abs() <= (H + 1) * U * dot.abs().sum(-1) + 1e-37).all()
        ref_h = (w[:, j, None].double() * dy.double())[there]
        assert within(dh[slots[there, j].long()], ref_h, U * ref_h.abs())
    assert within(y, ref, (k + 1) * U * mag)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(33, 256), (4097, 64), (8195, 256), (6, 1024)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_of_views_off_a_16_byte_boundary(T, E, score, dtype):
    """Logits and biases one element past an aligned start: bit for bit what aligned copies give, forward and
    backward, with a wave or 16 lanes to a token."""
    g = rng(T + E)
    logits = randn(g, T * E + 1).to(DT[dtype])[1:].view(T, E)
    bias = (0.1 * randn(g, E + 1))[1:]
    kw = dict(score=score, groups=4, topk_groups=2)
    w, e = fq.moe_route(logits, 8, bias=bias, **kw)
    for x, b in ((logits.clone(), bias), (logits, bias.clone()), (logits.clone(), bias.clone())):
        wa, ea = fq.moe_route(x, 8, bias=b, **kw)
        assert torch.equal(w, wa) and torch.equal(e, ea)
    dw = randn(g, T, 8)
    dx = fq.moe_route_backward(dw, logits, e, score=score)
    assert torch.equal(dx, fq.moe_route_backward(dw, logits.clone(), e, score=score))
    # and an output that starts off the boundary, which only the C interface can ask for
    out = torch.full((T * E + 2,), 7.0, dtype=DT[dtype], device="cuda")
    status = fq.lib.moe_route_backward(dw.data_ptr(), logits.data_ptr(), int(dtype == "bf16"), e.data_ptr(),
                                       out[1:].data_ptr(), T, E, 8, 1.0, int(score == "softmax"),
                                       torch.cuda.current_stream().cuda_stream)
    assert status == 0 and torch.equal(out[1:-1].view(T, E), dx) and out[0] == 7 and out[-1] == 7


@pytest.mark.parametrize("n", [2000, 1 << 22])
def test_sigmoid_scores_are_the_divided_form(n):
    """One expert's score is its sigmoid, bit for bit 1 / (1 + exp(-x)) with the addition and the quotient rounded
    to nearest (by numpy): dense logits from where the score is 1 to where it is the smallest number and 0, and
    logits that give every binade of the quotient's divisor. (A few tokens and many: both kernels.)"""
    logits = torch.cat([torch.linspace(-89.5, 20.0, n, device="cuda"), torch.linspace(-88.8, -86.9, n, device="cuda"),
                        10.0 * randn(rng(n), n), -torch.linspace(0.0, 88.0, 129, device="cuda")])
    with np.errstate(over="ignore"):
        ref = np.float32(1) / (np.float32(1) + torch.exp(-logits).cpu().numpy())
    for t0 in range(0, logits.numel(), 1000 if n == 2000 else n):
        part = logits[t0:t0 + (1000 if n == 2000 else n)]
        w, e = fq.moe_route(part[:, None].contiguous(), 1, renormalize=False)
        assert not bool(e.any())
        assert np.array_equal(w[:, 0].cpu().numpy().view(np.uint32), ref[t0:t0 + part.numel()].view(np.uint32))


@pytest.mark.parametrize("T", [9, 4100])
@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward_steps(score, k, T):
    """Ordinary scores: the formula's steps, each rounded to nearest in fp32, bit for bit. (With one or two
    experts sums have one order. One renormalised weight does not depend on the logits: what is left of its
    gradient is those steps' rounding.)"""
    E = 24
    g = rng(T + k)
    logits, dw = randn(g, T, E), randn(g, T, k)
    w, e = fq.moe_route(logits, E, score=score, renormalize=False)
    s = torch.empty_like(w).scatter_(1, e.long(), w).cpu().numpy()
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=-1).indices
    at = idx.cpu().numpy()
    sel, d = np.take_along_axis(s, at, 1), dw.cpu().numpy() * np.float32(2.5)
    total, dot = sel.sum(1, keepdims=True), (d * sel).sum(1, keepdims=True)
    d = (d - dot / total) / total
    dx = np.zeros_like(s)
    if score == "sigmoid":
        np.put_along_axis(dx, at, d * (sel * (1 - sel)), 1)
    else:
        np.put_along_axis(dx, at, d, 1)
        dx = s * (dx - (d * sel).sum(1, keepdims=True))
    got = fq.moe_route_backward(dw, logits, idx.to(torch.int32), score=score, scale=2.5).cpu().numpy()
    assert got.dtype == dx.dtype == np.float32 and np.array_equal(got, dx)
