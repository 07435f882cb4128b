"""GPU parity of the 8-bit integer products against plain implementations in 64 bits.

The integer sums are exact in float64 (below 2^53), so the reference knows them; the outputs'
only errors are the rounding of the sum to fp32, two products and, with a bias, one sum, each
within u = 2^-24: |y - ref| <= 4 u (|v| + |bias|), v the scaled sum; bf16 outputs lie between
the bf16 roundings of those bounds. Those steps are stated, so fp32 outputs are also compared bit for bit with the same
steps taken by numpy on the exact sum, and bf16 outputs with their rounding: whatever kernel
variant a shape takes, it gives the same bits.
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


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.1 + 1e-3


def check(y, a, sa, w, sw, bias, out):
    exact = a.double() @ w.double().t()
    v = exact * sa.double()[:, None] * sw.double()
    ref = v if bias is None else v + bias.double()
    mag = v.abs() if bias is None else v.abs() + bias.double().abs()
    lo, hi = ref - 4 * U * mag - 1e-37, ref + 4 * U * mag + 1e-37
    if out == "bf16":
        lo, hi = lo.bfloat16().double(), hi.bfloat16().double()
    assert ((y.double() >= lo) & (y.double() <= hi)).all(), float(((y.double() - ref).abs() / (mag + 1e-37)).max())
    e32 = exact.cpu().numpy().astype(np.float32)
    s = e32 * sa.cpu().numpy()[:, None] * sw.cpu().numpy()
    if bias is not None:
        s = s + bias.cpu().numpy()
    assert torch.equal(y.cpu(), torch.from_numpy(s).to(DT[out]))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,biased", [
    (1, 1, 16, True), (1, 16, 64, False), (1, 7168, 7168, False), (2, 100, 48, True), (15, 17, 144, False),
    (16, 130, 1040, True), (17, 33, 128, False), (31, 1000, 656, True), (33, 15, 64, True), (64, 300, 2064, False),
    (65, 129, 176, True), (128, 128, 128, False), (129, 257, 16, True), (200, 100, 1040, False),
    (300, 1001, 304, True), (1000, 576, 1536, False), (4096, 4100, 272, True), (4097, 4096, 144, False),
    (9, 7168, 1536, True), (100, 5000, 2048, False), (700, 1536, 3088, True), (513, 7168, 1024, False),
    (1030, 7168, 528, True), (2050, 7100, 1040, False),
])
def test_gemm(M, N, K, biased, out):
    g = rng(M + N + K)
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    bias = torch.randn(N, generator=g, device="cuda") if biased else None
    y = fq.int8_gemm(a, sa, w, sw, bias, out_dtype=DT[out])
    assert y.dtype == DT[out] and y.shape == (M, N)
    check(y, a, sa, w, sw, bias, out)


@pytest.mark.parametrize("M", [3, 100, 300])
def test_gemm_largest_sums(M):
    """Every code at the end of its range over the longest K: the sum nearly fills 32 bits."""
    K, N = (1 << 17) - 16, 20
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    g = rng(M)
    sa, sw = scales(g, M), scales(g, N)
    check(fq.int8_gemm(a, sa, w, sw, out_dtype=torch.float32), a, sa, w, sw, None, "f32")


@pytest.mark.parametrize("M,N", [(5, 33), (40, 70), (200, 130)])
def test_gemm_writes_only_its_output(M, N):
    """The output a view into a larger buffer, 4 bytes past a 16-byte boundary; operands that
    end where their allocation does are read no further (their neighbours hold other codes)."""
    g = rng(M)
    K = 208
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    for out, per in (("f32", 1), ("bf16", 2)):
        buf = torch.full((M * N + 64,), 7.0, dtype=DT[out], device="cuda")
        y = buf[per:per + M * N].view(M, N)
        fq.int8_gemm(a, sa, w, sw, out_dtype=DT[out], out=y)
        check(y, a, sa, w, sw, None, out)
        assert (buf[:per] == 7).all() and (buf[per + M * N:] == 7).all()


def test_gemm_empty():
    a = torch.empty((3, 0), dtype=torch.int8, device="cuda")
    w = torch.empty((5, 0), dtype=torch.int8, device="cuda")
    bias = torch.randn(5, device="cuda")
    y = fq.int8_gemm(a, torch.ones(3, device="cuda"), w, torch.ones(5, device="cuda"), bias, out_dtype=torch.float32)
    assert torch.equal(y, bias.expand(3, 5))
    z = fq.int8_linear(torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), w, torch.ones(5, device="cuda"), bias,
                       out_dtype=torch.float32)
    assert torch.equal(z, y)
    big = fq.int8_gemm(torch.empty((300, 0), dtype=torch.int8, device="cuda"), torch.ones(300, device="cuda"), w,
                       torch.ones(5, device="cuda"), out_dtype=torch.float32)
    assert (big == 0).all() and big.shape == (300, 5)
    assert fq.int8_gemm(torch.empty((0, 16), dtype=torch.int8, device="cuda"), torch.ones(0, device="cuda"),
                        torch.ones((5, 16), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda")).shape == (0, 5)


def quant_ref(x):
    x = x.float().cpu().numpy()
    top = np.abs(x).max(-1, initial=0)
    s = top * (np.float32(1) / np.float32(127))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, np.rint(x / s[..., None]), 0)
    return np.clip(q, -127, 127).astype(np.int8), s


@pytest.mark.parametrize("M,K", [(1, 16), (5, 48), (3, 512), (7, 528), (4, 2048), (9, 2064), (2, 7168), (3, 8192),
                                 (2, 8208), (3, 32768), (2, 32784), (2, 70000)])
def test_quant(M, K):
    g = rng(M + K)
    x = (torch.randn((M, K), generator=g, device="cuda") * torch.logspace(-3, 3, M, device="cuda")[:, None]).bfloat16()
    x[0, : K // 2] = 0
    q, s = fq.int8_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quant_every_pair():
    """Every (x, amax) pair of bf16 significands at every distance of exponents that can give a
    code other than 0 (x down to amax / 512), with both signs, and amax from the smallest
    subnormal to the largest number: the scale and the quotient round as the format says."""
    frac = torch.arange(128, dtype=torch.int32)
    rows = []
    for top_exp in (0, 1, 2, 3, 7, 8, 9, 64, 120, 127, 128, 134, 200, 254):
        for f in range(128):
            top = (top_exp << 7) | f
            if top == 0:
                continue
            body = [(max(top_exp - d, 0) << 7) | frac for d in range(10)]
            body = torch.cat(body)
            body = torch.where(body <= top, body, 0)
            rows.append(torch.cat([torch.tensor([top], dtype=torch.int32), body, body | 0x8000,
                                   torch.zeros(15, dtype=torch.int32)]))
    bits = torch.stack(rows)
    bits = torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16)
    x = bits.view(torch.bfloat16).cuda()
    q, s = fq.int8_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quant_zero_rows_and_empty():
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    x[1, 5] = -2.0
    q, s = fq.int8_quant(x)
    assert (s[[0, 2]] == 0).all() and (q[[0, 2]] == 0).all() and q[1, 5] == -127 and int(q[1].abs().sum()) == 127
    q, s = fq.int8_quant(torch.empty((4, 0), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (4, 0) and (s == 0).all()
    q, s = fq.int8_quant(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)


@pytest.mark.parametrize("M,K", [(512, 1040), (513, 1040), (600, 2048), (515, 512), (514, 2064), (130, 20000)])
def test_quant_many_rows(M, K):
    g = rng(M + K)
    x = (torch.randn((M, K), generator=g, device="cuda") * torch.logspace(-3, 3, M, device="cuda")[:, None]).bfloat16()
    x[M // 2] = 0
    q, s = fq.int8_quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape,N", [((1, 256), 96), ((2, 3, 1536), 200), ((300, 512), 576), ((1, 16), 1),
                                     ((2, 1040), 33), ((3, 7168), 130), ((4, 8192), 100), ((4, 8208), 100),
                                     ((5, 7168), 64), ((2, 2, 64), 7168), ((0, 64), 16)])
def test_linear(shape, N, out):
    """Quantisation and product against the 64-bit product of what the codes stand for."""
    g = rng(N)
    x = torch.randn(shape, generator=g, device="cuda").bfloat16()
    wq, ws = fq.int8_quant((torch.randn((N, shape[-1]), generator=g, device="cuda") * 0.02).bfloat16())
    bias = torch.randn(N, generator=g, device="cuda")
    y = fq.int8_linear(x, wq, ws, bias, out_dtype=DT[out])
    assert y.shape == (*shape[:-1], N)
    rq, rs = quant_ref(x.view(-1, shape[-1]))
    check(y.view(-1, N), torch.from_numpy(rq).cuda(), torch.from_numpy(rs).cuda(), wq, ws, bias, out)


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9])
@pytest.mark.parametrize("K,N", [(16, 40), (1040, 130), (2048, 16400), (2064, 100), (4096, 8200), (4112, 77),
                                 (8192, 50), (8208, 50)])
def test_linear_is_quant_and_gemm(M, K, N):
    """However many launches the layer takes, the outputs are those of its two halves, bit for bit;
    a row of zeros and one of subnormal numbers among them."""
    g = rng(M + K + N)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    if M > 2:
        x[0], x[1] = 0.0, 1e-40
    wq, ws = codes(g, N, K), scales(g, N)
    q, s = fq.int8_quant(x)
    for out in DT.values():
        y = fq.int8_linear(x, wq, ws, out_dtype=out)
        assert torch.equal(y, fq.int8_gemm(q, s, wq, ws, out_dtype=out))


def grouped_check(y, a, sa, w, sw, offsets, rows, out):
    bounds = offsets.tolist()
    for e in range(w.shape[0]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            t = torch.arange(lo, hi, device="cuda") if rows is None else rows[lo:hi].long()
            there = (t >= 0) & (t < a.shape[0])
            aa = torch.where(there[:, None], a[t.clamp(0, a.shape[0] - 1)], 0)
            ss = torch.where(there, sa[t.clamp(0, a.shape[0] - 1)], 0.0)
            check(y[lo:hi], aa, ss, w[e], sw[e], None, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,N,K", [
    ([0, 1, 127, 128, 129, 0, 300, 5], 256, 256), ([37, 0, 0, 200], 200, 400), ([3, 250, 1], 1100, 144),
    ([0, 0, 64], 64, 1024), ([1, 0, 2, 0, 0, 3, 16, 17, 0, 4], 100, 1040), ([0] * 63 + [1] + [0] * 10 + [2], 33, 48),
    ([1], 7, 16), ([0, 0], 16, 64), ([20] * 70, 48, 128), ([40, 0, 33, 64, 65], 500, 656),
])
def test_grouped(sizes, N, K, gather, out):
    E, R = len(sizes), sum(sizes)
    g = rng(E + R + N)
    tokens = max(1, R // 3) if gather else R
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int64, device="cuda")
    rows = torch.randint(0, tokens, (R,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    a, sa = codes(g, tokens, K), scales(g, tokens)
    w, sw = codes(g, E, N, K), scales(g, E, N)
    y = fq.int8_grouped_gemm(a, sa, w, sw, offsets, rows=rows, out_dtype=DT[out])
    assert y.shape == (R, N) and y.dtype == DT[out]
    grouped_check(y, a, sa, w, sw, offsets, rows, out)


def uneven(E, mean, seed):
    """Rows of E experts, some of them without any, `mean` on average."""
    r = np.random.default_rng(seed).gamma(1.5, mean / 1.5, E).astype(int)
    r[E // 2] = 0
    r[0] += max(0, E * mean - int(r.sum()))
    return r.tolist()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("E,N,K,mean", [
    (40, 1024, 7168, 3), (40, 1024, 7168, 20), (64, 1024, 7168, 60), (40, 1024, 7168, 360), (16, 256, 70000, 10),
    (16, 256, 70000, 100),
])
def test_grouped_weights_larger_than_the_caches(E, N, K, mean, out):
    """Over 256 MB of weights, at each size of block."""
    sizes = uneven(E, mean, E + mean)
    R = sum(sizes)
    g = rng(R)
    tokens = max(1, R // 2)
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int64, device="cuda")
    rows = torch.randint(0, tokens, (R,), generator=g, device="cuda", dtype=torch.int32)
    a, sa, w, sw = codes(g, tokens, K), scales(g, tokens), codes(g, E, N, K), scales(g, E, N)
    y = fq.int8_grouped_gemm(a, sa, w, sw, offsets, rows=rows, out_dtype=DT[out])
    grouped_check(y, a, sa, w, sw, offsets, rows, out)


@pytest.mark.parametrize("E,N,K,mean", [
    (40, 169, 1040, 38), (60, 106, 528, 72), (50, 300, 400, 52), (30, 1408, 272, 250), (8, 2000, 144, 128),
    (70, 1000, 656, 9), (64, 512, 1024, 200), (200, 600, 256, 5), (12, 1300, 3216, 700),
])
def test_grouped_sizes_of_blocks(E, N, K, mean):
    """Numbers of tiles on both sides of where the size of the blocks changes."""
    sizes = uneven(E, mean, E + mean)
    R = sum(sizes)
    g = rng(R)
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int64, device="cuda")
    a, sa, w, sw = codes(g, R, K), scales(g, R), codes(g, E, N, K), scales(g, E, N)
    for out in ("f32", "bf16"):
        y = fq.int8_grouped_gemm(a, sa, w, sw, offsets, out_dtype=DT[out])
        grouped_check(y, a, sa, w, sw, offsets, None, out)


@pytest.mark.parametrize("N", [512, 500, 504, 511])
def test_large_outputs_of_any_row_length(N):
    """Rows that are whole 64-byte blocks or not, in an output that begins anywhere that 4 bytes allow."""
    M, K = 5000, 272
    g = rng(N)
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    for out in ("f32", "bf16"):
        check(fq.int8_gemm(a, sa, w, sw, out_dtype=DT[out]), a, sa, w, sw, None, out)
        buf = torch.full((M * N + 64,), 7.0, dtype=DT[out], device="cuda")
        at = 4 // buf.element_size()
        y = buf[at:at + M * N].view(M, N)
        fq.int8_gemm(a, sa, w, sw, out_dtype=DT[out], out=y)
        check(y, a, sa, w, sw, None, out)
        assert (buf[:at] == 7).all() and (buf[at + M * N:] == 7).all()


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements, experts' weights and rows of more than 2^32 bytes: the
    ends of each."""
    g = rng(9)
    M, N, K = 70000, 32768, 16
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    y = fq.int8_gemm(a, sa, w, sw, out_dtype=torch.bfloat16)
    for part in (slice(0, 5), slice(M // 2, M // 2 + 5), slice(M - 5, M)):
        check(y[part], a[part], sa[part], w, sw, None, "bf16")
    del y
    E, N, K = 70, 8192, 8192
    w, sw = codes(g, E, N, K), scales(g, E, N)
    sizes = [0] * E
    sizes[0], sizes[40], sizes[E - 1] = 3, 40, 5
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int64, device="cuda")
    a, sa = codes(g, 48, K), scales(g, 48)
    grouped_check(fq.int8_grouped_gemm(a, sa, w, sw, offsets, out_dtype=torch.float32), a, sa, w, sw, offsets, None, "f32")
    del w
    M, K = 300000, 8192
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, K), generator=g, device="cuda").bfloat16()
    q, s = fq.int8_quant(x)
    rq, rs = quant_ref(x[-3:])
    assert np.array_equal(q[-3:].cpu().numpy(), rq) and np.array_equal(s[-3:].cpu().numpy(), rs)
    assert not bool(s[:-3].any())


@pytest.mark.parametrize("sizes", [[2, 0, 3], [150, 30, 0, 90]])
def test_grouped_rows_no_expert_owns(sizes):
    """Rows past the last offset are not written; rows of no token (-1, past the end) are rows
    of zeros; offsets that point outside are clamped."""
    E, R, N, K = len(sizes), sum(sizes) + 9, 64, 160
    g = rng(R)
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int64, device="cuda")
    a, sa, w, sw = codes(g, 11, K), scales(g, 11), codes(g, E, N, K), scales(g, E, N)
    rows = torch.randint(0, 11, (R,), generator=g, device="cuda", dtype=torch.int32)
    rows[1], rows[3] = -1, 11
    out = torch.full((R, N), 7.0, device="cuda")
    fq.int8_grouped_gemm(a, sa, w, sw, offsets, rows=rows, out_dtype=torch.float32, out=out)
    grouped_check(out, a, sa, w, sw, offsets, rows, "f32")
    assert (out[1] == 0).all() and (out[3] == 0).all() and (out[-9:] == 7).all()
    wild = offsets.clone()
    wild[-1] = 1 << 40
    wild[0] = -5
    out2 = fq.int8_grouped_gemm(a, sa, w, sw, wild, rows=rows, out_dtype=torch.float32)
    assert torch.equal(out2[:-9], out[:-9])


def test_grouped_with_placement():
    """moe_place's offsets and rows as the product takes them, against each token's own product."""
    T, k, E, N, K = 70, 4, 16, 96, 256
    g = rng(2)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    wq, ws = fq.int8_quant(torch.randn((E, N, K), generator=g, device="cuda").bfloat16())
    _, experts = fq.moe_route(torch.randn((T, E), generator=g, device="cuda"), k)
    offsets, rows, slots = fq.moe_place(experts, E)
    q, s = fq.int8_quant(x)
    y = fq.int8_grouped_gemm(q, s, wq, ws, offsets, rows=rows, out_dtype=torch.float32)
    for t in (0, 33, T - 1):
        for j in range(k):
            e = int(experts[t, j])
            check(y[slots[t, j]][None], q[t:t + 1], s[t:t + 1], wq[e], ws[e], None, "f32")


def test_other_stream_and_repeats():
    g = rng(3)
    a, w, sa, sw = codes(g, 200, 512), codes(g, 300, 512), scales(g, 200), scales(g, 300)
    y = fq.int8_gemm(a, sa, w, sw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        z = [fq.int8_gemm(a, sa, w, sw) for _ in range(3)]
    st.synchronize()
    assert all(torch.equal(y, v) for v in z)


def test_captured_in_a_graph():
    """A whole routed layer's calls captured once and replayed on new inputs, with eager work
    between the replays: every replay gives the eager result."""
    T, k, E, N, K = 24, 3, 8, 80, 128
    g = rng(4)
    wq, ws = fq.int8_quant(torch.randn((E, N, K), generator=g, device="cuda").bfloat16())
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=g, device="cuda")

    def layer():
        weights, experts = fq.moe_route(logits, k)
        offsets, rows, slots = fq.moe_place(experts, E)
        q, s = fq.int8_quant(x)
        return fq.moe_combine(fq.int8_grouped_gemm(q, s, wq, ws, offsets, rows=rows), slots, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for _ in range(4):
        x.copy_(torch.randn((T, K), generator=g, device="cuda"))
        logits.copy_(torch.randn((T, E), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer())


def test_refusals():
    a = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    w = torch.zeros((8, 32), dtype=torch.int8, device="cuda")
    sa, sw = torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(TypeError):
        fq.int8_gemm(a.float(), sa, w, sw)
    with pytest.raises(TypeError):
        fq.int8_gemm(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fq.int8_gemm(a[:, :16].contiguous(), sa, w, sw)
    with pytest.raises(ValueError):
        fq.int8_gemm(a[:, :24].contiguous(), sa, w[:, :24].contiguous(), sw)
    with pytest.raises(ValueError):
        fq.int8_gemm(a, sa[:3], w, sw)
    with pytest.raises(ValueError):
        fq.int8_gemm(a, sa, w.t().contiguous().t(), sw)
    with pytest.raises(ValueError):
        fq.int8_gemm(a, sa, w, sw, bias=torch.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        fq.int8_gemm(a, sa, w.cpu(), sw)
    with pytest.raises(ValueError):
        fq.int8_gemm(torch.zeros(4 * 32 + 1, dtype=torch.int8, device="cuda")[1:].view(4, 32), sa, w, sw)
    with pytest.raises(TypeError):
        fq.int8_linear(a, w, sw)
    with pytest.raises(ValueError):
        fq.int8_linear(a.bfloat16(), w[:, :16].contiguous(), sw)
    with pytest.raises(ValueError):
        fq.int8_linear(a.bfloat16(), w, sw[:7])
    with pytest.raises(TypeError):
        fq.int8_quant(torch.zeros((2, 16), device="cuda"))
    with pytest.raises(ValueError):
        fq.int8_quant(torch.zeros((2, 24), dtype=torch.bfloat16, device="cuda"))
    off = torch.tensor([0, 4], device="cuda")
    w3 = w[None]
    with pytest.raises(TypeError):
        fq.int8_grouped_gemm(a, sa, w3, sw[None], off.int())
    with pytest.raises(ValueError):
        fq.int8_grouped_gemm(a, sa, w3, sw[None], off[:1])
    with pytest.raises(ValueError):
        fq.int8_grouped_gemm(a, sa, w, sw, off)
    with pytest.raises(TypeError):
        fq.int8_grouped_gemm(a, sa, w3, sw[None], off, rows=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        fq.int8_grouped_gemm(a, sa, w3, sw[None], off, rows=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("M", [1, 2, 3, 9])
def test_linear_of_no_depth(M):
    """K = 0: the bias, or zeros, whatever the scales hold, at channel counts of every kernel; from the C
    interface also without x, weight and scales."""
    for N in (40, 16400):
        bias = torch.randn(N, generator=rng(N), device="cuda")
        x = torch.empty((M, 0), dtype=torch.bfloat16, device="cuda")
        w = torch.empty((N, 0), dtype=torch.int8, device="cuda")
        for bad in (torch.nan, torch.inf):
            for b in (None, bias):
                for out in DT.values():
                    y = fq.int8_linear(x, w, torch.full((N,), bad, device="cuda"), b, out_dtype=out)
                    assert torch.equal(y, (torch.zeros_like(bias) if b is None else b).to(out).expand(M, N))
        y = torch.full((M, N), 7.0, device="cuda")
        size = fq.lib.int8_linear_workspace_bytes(M, N, 0)
        ws = torch.empty(size + 16, dtype=torch.uint8, device="cuda")
        assert fq.lib.int8_linear(None, None, None, bias.data_ptr(), y.data_ptr(), 0, M, N, 0, ws.data_ptr(), size,
                                  torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(y, bias.expand(M, N))


def test_quant_of_more_rows_than_one_grid():
    """2^22 and some rows of more than 8192 elements: 1024 threads each, of which a grid counts 2^32 - 1."""
    M, K = (1 << 22) + 5, 8208
    g = rng(7)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    parts = [slice(0, 3), slice(M // 2, M // 2 + 3), slice((1 << 22) - 4, M)]
    for p in parts:
        x[p] = torch.randn(x[p].shape, generator=g, device="cuda").bfloat16()
    q, s = fq.int8_quant(x)
    assert int((s != 0).sum()) == 15
    for p in parts:
        rq, rs = quant_ref(x[p])
        assert np.array_equal(s[p].cpu().numpy().view(np.uint32), rs.view(np.uint32))
        assert np.array_equal(q[p].cpu().numpy(), rq)
    del x, q, s
    torch.cuda.empty_cache()


def test_gemm_of_more_rows_than_a_grid_of_small_tiles():
    """2^30 and some rows: more tiles of 64 rows than a grid's 2^32 - 1 threads hold."""
    M, N, K = (1 << 30) + 70, 16, 16
    g = rng(8)
    a = torch.empty((M, K), dtype=torch.int8, device="cuda").random_(-128, 128, generator=g)
    sa, w, sw = scales(g, M), codes(g, N, K), scales(g, N)
    y = fq.int8_gemm(a, sa, w, sw, out_dtype=torch.bfloat16)
    for p in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        check(y[p], a[p], sa[p], w, sw, None, "bf16")
    del a, sa, y
    torch.cuda.empty_cache()


def test_linear_of_more_channels_than_one_launch():
    """2^29 and some channels for one row: the ends and the middle."""
    N, K = (1 << 29) + 50, 16
    g = rng(12)
    w = torch.empty((N, K), dtype=torch.int8, device="cuda").random_(-128, 128, generator=g)
    ws, x = scales(g, N), torch.randn((1, K), generator=g, device="cuda").bfloat16()
    y = fq.int8_linear(x, w, ws, out_dtype=torch.float32)
    q, s = (torch.from_numpy(v).cuda() for v in quant_ref(x))
    for p in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        check(y[:, p], q, s, w[p], ws[p], None, "f32")
    del w, ws, y
    torch.cuda.empty_cache()


def test_outputs_are_filled_in_deterministic_mode():
    """Where torch fills uninitialised memory with NaN (deterministic algorithms), what no expert owns
    is filled too."""
    g = rng(10)
    a, sa, w, sw = codes(g, 9, 64), scales(g, 9), codes(g, 2, 32, 64), scales(g, 2, 32)
    offsets = torch.tensor([0, 2, 5], device="cuda")
    slots = torch.tensor([[0, -1], [3, 1]], dtype=torch.int32, device="cuda")
    h, dy, weights = torch.ones((9, 32), device="cuda"), torch.ones((2, 32), device="cuda"), torch.ones((2, 2), device="cuda")
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        y = fq.int8_grouped_gemm(a, sa, w, sw, offsets, out_dtype=torch.float32)
        dh, _ = fq.moe_combine_backward(dy, h, slots, weights)
    finally:
        torch.use_deterministic_algorithms(before)
    assert torch.isnan(y[5:]).all() and not torch.isnan(y[:5]).any()
    assert torch.isnan(dh[[2, 4, 5, 6, 7, 8]]).all() and (dh[[0, 1, 3]] == 1).all()


def test_quant_exponents_around_the_quotients_limit():
    """Every (x, amax) pair of bf16 significands where the scale passes 2^-92, from where the quotient takes
    another way."""
    frac = torch.arange(128, dtype=torch.int32)
    rows = []
    for top_exp in range(38, 47):
        for f in range(128):
            top = (top_exp << 7) | f
            body = torch.cat([((top_exp - d) << 7) | frac for d in range(10)])
            body = torch.where(body <= top, body, 0)
            rows.append(torch.cat([torch.tensor([top], dtype=torch.int32), body, body | 0x8000,
                                   torch.zeros(15, dtype=torch.int32)]))
    bits = torch.stack(rows)
    x = torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16).view(torch.bfloat16).cuda()
    q, s = fq.int8_quant(x)
    rq, rs = quant_ref(x)
    assert rs.min() < 2.0 ** -92 < rs.max()
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)
