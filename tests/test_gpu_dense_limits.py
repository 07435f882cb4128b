"""The dense block's operators at the ends of their documented range and where single elements are not finite,
against 64 bits.

Tolerances: half(t) is half a step of t relative to the value; U = 2^-24 is fp32's. The matrix unit adds
32 products at a time, with every product and addition off by at most 2 U: a sum over K is off by at most
2 (K / 32 + 32) U of the sum of its terms' magnitudes. The activations of the kernels are some 35 fp32
operations on the hardware's exponential and reciprocal, each within one unit in the last place (2 U), and a
polynomial within 5.1e-8 (0.9 U): 16 U relative covers the few of them that carry the result's full size.
"""
import pytest
import torch

import fp8_act_quant_amd as fq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACT = 16


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def act64(a, act):
    """The activation, its slope, and the sum of the slope's two terms' magnitudes."""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s)), s + (a * s * (1 - s)).abs()
    p = 0.5 * torch.erfc(-a * 0.5 ** 0.5)
    q = a * torch.exp(-a * a / 2) * (0.5 / torch.pi) ** 0.5
    return a * p, p + q, p + q.abs()


def product64(x, w):
    """x w^T and how far its fp32 sum may be off."""
    x, w = x.double(), w.double()
    return x @ w.t(), 2 * (x.shape[1] / 32 + 32) * U * (x.abs() @ w.abs().t())


def slopes64(dh, gu, off, act, lost):
    """The projections' gradient [dg du] from gu, each off by at most `off`, and how far it may be off itself after
    losing `lost` of each value in its rounding. (Slopes stay below 1.13, their derivatives below 0.8.)"""
    F = dh.shape[1]
    a, b, off_a, off_b, e = gu[:, :F], gu[:, F:], off[:, :F], off[:, F:], dh.double()
    p, s, mag = act64(a, act)
    d = torch.cat([e * b * s, e * p], -1)
    e = e.abs()
    err = torch.cat([e * ((b.abs() + off_b) * 0.8 * off_a + 1.13 * off_b) + ACT * U * e * b.abs() * mag,
                     e * 1.13 * off_a + ACT * U * e * p.abs()], -1)
    return d, err + lost * (d.abs() + err)


def product_of(d, off, w, terms):
    """d w, w [terms, N], and how far its fp32 form may be off where d is off by `off`."""
    w = w.double()
    return d @ w, off @ w.abs() + 2 * (terms / 32 + 32) * U * ((d.abs() + off) @ w.abs())


def near(got, ref, off, name=""):
    """Every element within its type's rounding and `off` of ref."""
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    limit = off + half(got.dtype) * (ref.abs() + off) + 1e-37
    assert ((got.double() - ref).abs() <= limit).all(), (name, float(((got.double() - ref).abs() / limit).max()))


def test_gradient_of_very_many_rows():
    """2^25 tokens, whose dx is 2^19 of the smallest tiles."""
    M, F, K = 1 << 25, 8, 8
    g = rng(1)
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=0.5), randn(g, M, F)
    dx, dw = fq.gated_linear_backward(dh, x, w, dx_dtype=torch.float32)
    at = torch.tensor([0, 63, 64, 127, 1 << 24, (1 << 24) + 1, M - 65, M - 1], device="cuda")
    d, off = slopes64(dh[at], *product64(x[at], w), "silu", half(torch.bfloat16))
    near(dx[at], *product_of(d, off, w, 2 * F), "dx")
    # a channel of dw over all rows; 2^25 roundings of either sign, each at most 2^-9 of a term, are far below 2^-9 in all
    ref = torch.zeros(K, dtype=torch.float64, device="cuda")
    for lo in range(0, M, 1 << 22):
        xs = x[lo:lo + (1 << 22)].double()
        ref += (dh[lo:lo + (1 << 22), F - 1].double() * act64(xs @ w[F - 1].double(), "silu")[0]) @ xs
    assert float((dw[2 * F - 1].double() - ref).norm() / ref.norm()) < half(torch.bfloat16)


def test_adapters_of_the_most_channels():
    """2^28 channels of an output that adapters are added to, for more than 32 rows: 2^24 of the smallest tiles."""
    M, N, K, r = 33, 1 << 28, 8, 8
    g = rng(2)
    x, a = randn(g, M, K), randn(g, 2, r, K, std=0.5)
    b = torch.empty((2, N, r), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = torch.tensor([0, 31, 32, 1 << 27, N - 33, N - 1], device="cuda")
    base = y[:, at].double()
    got = fq.adapter_add(y, x, a, b, ids, out=y)[:, at]
    ref, off = base.clone(), 2 * U * base.abs()
    for e in range(2):
        rows = (ids == e).nonzero()[:, 0]
        u, off_u = product64(x[rows], a[e])
        add, lost = product_of(u, off_u, b[e, at].t(), r)
        ref[rows] += add
        off[rows] += lost
    near(got, ref, off + 4 * U * ref.abs())
    assert torch.equal(got[ids < 0].double(), base[ids < 0])


WIDE = [(1, 8, 8), (1, 2048, 1536), (17, 72, 520), (31, 2056, 264), (64, 200, 64), (333, 1000, 1096), (1021, 512, 1544),
        (1500, 2048, 1032), (2050, 96, 4104)]


@pytest.mark.parametrize("M,F,K", WIDE)
def test_wide_gradient(M, F, K):
    """With `wide` the projections' gradient keeps 16 bits: two roundings to bf16, the second of what the first lost."""
    g = rng(M + F + K)
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=1.5 * K ** -0.5), randn(g, M, F)
    gu = fq.gated_linear(x, w, keep=True)[1]
    for act, kept in (("silu", True), ("gelu", False), ("gelu", True), ("silu", False)):
        at = (gu.double(), torch.zeros_like(gu, dtype=torch.float64)) if kept else product64(x, w)
        d, off = slopes64(dh, *at, act, half(torch.bfloat16) ** 2)
        want = product_of(d, off, w, 2 * F), product_of(d.t(), off.t(), x, M)
        args = (dh, x, w, gu if kept else None, act)
        got = fq.gated_linear_backward(*args, dx_dtype=torch.float32, wide=True)
        # (two sums, of the first and of the second numbers, whose magnitudes are 1 + 2^-8 of one's)
        for y, (ref, slack) in zip(got, want):
            near(y, ref, slack * (1 + 2 * half(torch.bfloat16)), (act, kept))
        rough = fq.gated_linear_backward(*args, dx_dtype=torch.float32)
        if M * F > 4096:
            for y, z, (ref, _) in zip(got, rough, want):
                assert float((z.double() - ref).norm()) > 20 * float((y.double() - ref).norm()), (act, kept)
        short = fq.gated_linear_backward(*args, dw_dtype=torch.bfloat16, wide=True)
        assert all(torch.equal(y.bfloat16(), z) for y, z in zip(got, short))


def test_wide_gradient_of_infinite_weights():
    """An infinite weight makes the gradient infinite, also where nothing was lost in the first rounding."""
    M, F, K = 40, 16, 24
    x, w = torch.zeros((M, K), device="cuda").bfloat16(), torch.zeros((2 * F, K), device="cuda").bfloat16()
    x[:, 0], x[:, 1] = 1.0, 1.0
    w[:F, 0], w[F:, 1] = 1.0, 1.0
    dh = torch.ones((M, F), device="cuda").bfloat16()
    gu = torch.ones((M, 2 * F), device="cuda").bfloat16()
    w[F + 3, 7] = float("inf")        # du = act(1) > 0 meets it; its rest may be of either sign
    w[F + 4, 8] = float("inf")
    gu[:, 4] = 0.0                    # act(0) = 0 meets it: NaN, as 0 * inf is
    for act in ("silu", "gelu"):
        dx, _ = fq.gated_linear_backward(dh, x, w, gu, act, dx_dtype=torch.float32, wide=True)
        assert (dx[:, 7] == float("inf")).all() and torch.isnan(dx[:, 8]).all()
        assert torch.isfinite(dx[:, [0, 1, 2, 6, 9]]).all()


def test_wide_gradient_empty_captured_and_on_a_stream():
    def e(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    dx, dw = fq.gated_linear_backward(e(0, 16), e(0, 64), e(32, 64), wide=True)
    assert dx.shape == (0, 64) and dw.shape == (32, 64) and (dw == 0).all()
    dx, dw = fq.gated_linear_backward(e(5, 0), e(5, 64), e(0, 64), wide=True)
    assert (dx == 0).all() and dw.shape == (0, 64)
    g = rng(8)
    M, F, K = 300, 264, 520
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=K ** -0.5), randn(g, M, F)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fq.gated_linear_backward(dh, x, w, wide=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.gated_linear_backward(dh, x, w, wide=True)
    for k in range(3):
        x.copy_(randn(g, M, K))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        with torch.cuda.stream(side):
            eager = fq.gated_linear_backward(dh, x, w, wide=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), k


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("M,F,K", [(5, 16, 64), (465, 616, 24), (759, 1168, 1600), (2909, 456, 976)])
def test_one_gradient_alone(M, F, K, wide):
    """The C call without dx, or without dw, whose launches are one or two: the other has the same bits, and a
    workspace of the stated size is not written past."""
    g = rng(M)
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=K ** -0.5), randn(g, M, F)
    want = fq.gated_linear_backward(dh, x, w, dw_dtype=torch.bfloat16, wide=wide)
    need = (fq.lib.gated_linear_backward_wide_workspace_bytes if wide else fq.lib.gated_linear_backward_workspace_bytes)(M, F, K)
    for k in range(2):
        ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        got = [torch.full_like(v, 7.0) for v in want]
        at = [v.data_ptr() if i == k else None for i, v in enumerate(got)]
        assert fq.lib.gated_linear_backward(dh.data_ptr(), x.data_ptr(), w.data_ptr(), None, 256 if wide else 0, at[0], 1, at[1],
                                            1, M, F, K, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(got[k], want[k]) and (got[1 - k] == 7).all() and (ws[need:] == 0xA5).all()


@pytest.mark.parametrize("H", [8, 515, 4100, 9001])
def test_norm_without_the_stream(H):
    """The C call with y and weight whose t is not wanted: z alone."""
    g = rng(H)
    for dtype, code in ((torch.bfloat16, 1), (torch.float32, 0)):
        x, y = randn(g, 37, H, dtype=dtype), randn(g, 37, H, dtype=dtype)
        w, post = torch.rand(H, device="cuda"), torch.rand(H, device="cuda")
        want = fq.residual_norm(x, y, w, post=post, gate=w, scale=0.5)[1]
        z = torch.empty_like(want)
        assert fq.lib.residual_norm(x.data_ptr(), y.data_ptr(), code, w.data_ptr(), post.data_ptr(), w.data_ptr(), 0, 0.5, 1e-6,
                                    None, z.data_ptr(), 37, H, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(z, want)


@pytest.mark.parametrize("M", [3, 60, 100, 300, 2305])
def test_adapter_infinities_by_every_way(M):
    """A row's own adapter with an infinity in B: u B is infinite where u is not 0, however few bits u has, and NaN
    where it is 0, whatever the way the rows are taken; infinite u too. Other columns and rows stay finite."""
    N, K, r = {300: 1500, 2305: 7408}.get(M, 200), 64, 40
    x = torch.zeros((M, K), device="cuda").bfloat16()
    x[:, 0] = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, -2.5)     # few bits: nothing is left below bf16
    x[:, 1] = torch.randn(M, device="cuda").abs() + 0.5
    x[:, 2] = 1.0
    a = torch.zeros((2, r, K), device="cuda").bfloat16()
    a[:, 0, 0] = a[:, 33, 1] = 1.0                         # u = x0 at rank 0, x1 at rank 33, 0 elsewhere
    a[:, 34, 1] = 1.0 + 2.0 ** -7
    a[:, 35, 2] = float("inf")
    b = torch.zeros((2, N, r), device="cuda").bfloat16()
    b[:, :, 35] = 1.0
    a[0, 35, 2] = 0.0
    b[0, 5, 0] = b[0, 9, 33] = float("inf")
    b[0, 6, 0] = b[0, 12, 34] = float("-inf")
    b[0, 7, 1] = float("inf")
    b[0, 8, 0] = float("nan")
    b[0, 10, 0], b[0, 10, 33] = float("inf"), 2.0
    ids = torch.where(torch.arange(M, device="cuda") % 16 == 7, 1, 0).to(torch.int32)
    ids[2::16] = -1
    mine, other = ids == 0, ids == 1
    sign = torch.sign(x[:, 0].float())
    base = torch.ones((M, N), device="cuda").bfloat16()
    w = torch.zeros((N, K), device="cuda").bfloat16()
    for y in (fq.adapter_linear(x, w, a, b, ids), fq.adapter_linear(x, w, a, b, ids, out_dtype=torch.float32),
              fq.adapter_add(base, x, a, b, ids)):
        y = y.float()
        inf = torch.full((M,), float("inf"), device="cuda")
        for column, want in ((5, inf * sign), (6, -inf * sign), (9, inf), (12, -inf), (10, inf * sign)):
            assert torch.equal(y[mine, column], want[mine]), column
        assert torch.isnan(y[mine][:, [7, 8]]).all()
        rest = [c for c in range(N) if c not in (5, 6, 7, 8, 9, 10, 12)]
        assert torch.isfinite(y[mine][:, rest]).all() and torch.isfinite(y[ids < 0]).all()
        assert (y[other] == float("inf")).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(3, 200), (60, 201), (300, 1500), (2305, 4100)])
def test_rows_without_an_adapter_keep_every_bit(M, N, dtype):
    """Added to another projection's output: where a row has no adapter, every bit of it stays, of negative zeros,
    subnormal numbers and infinities too; NaN stays NaN."""
    g = rng(M)
    K, r = 64, 40
    x, a, b = randn(g, M, K), randn(g, 3, r, K), randn(g, 3, N, r)
    ids = (torch.arange(M, device="cuda") % 5 - 2).to(torch.int32)
    y = randn(g, M, N, dtype=dtype)
    y[:, 1::7] = -0.0
    y[:, 2::7] = -1e-39 if dtype == torch.float32 else -2.0 ** -130
    y[:, 3::7] = float("-inf")
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    no = ids < 0
    before = y.clone()
    got = fq.adapter_add(y, x, a, b, ids)
    assert torch.equal(got[no].view(bits), before[no].view(bits)) and not torch.equal(got[~no], before[~no])
    y[no, 4] = float("nan")
    again = fq.adapter_add(y, x, a, b, ids, out=y)
    assert again is y or again.data_ptr() == y.data_ptr()
    keep = torch.arange(N, device="cuda") != 4
    assert torch.equal(y[no][:, keep].view(bits), before[no][:, keep].view(bits)) and torch.isnan(y[no, 4]).all()
    assert torch.equal(y[~no], got[~no])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_down_to_the_smallest_numbers(act):
    """Every bf16 number from -200 to 200 as the gate's projection: value and slope within ACT U wherever they are
    normal fp32 numbers, and nothing but less than the smallest of those otherwise."""
    a = torch.arange(0, 1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    a = a[(a.abs() <= 200) & (a.abs() >= 1e-30) | (a == 0)]
    x = torch.zeros((a.numel(), 8), device="cuda").bfloat16()
    x[:, 0], x[:, 1] = a, 1.0
    w = torch.zeros((16, 8), device="cuda").bfloat16()
    w[:8, 0] = w[8:, 1] = 1.0
    tiny = 2.0 ** -126
    value, slope, mag = act64(a.double(), act)
    for rows in (slice(0, a.numel()), slice(0, 16)):      # by tiles, and few rows
        h, gu = fq.gated_linear(x[rows].contiguous(), w, act=act, keep=True, out_dtype=torch.float32)
        assert ((h[:, 0].double() - value[rows]).abs() <= ACT * U * value[rows].abs() + tiny).all()
    h, gu = fq.gated_linear(x, w, act=act, keep=True, out_dtype=torch.float32)
    far = (value.abs() > 2 * tiny) & (a < -80 if act == "silu" else a < -12.5)
    assert far.any() and (h[far] != 0).all()
    one = torch.zeros((a.numel(), 8), device="cuda").bfloat16()
    one[:, 3] = 1.0
    for kept in (gu, None):
        dx, _ = fq.gated_linear_backward(one, x, w, kept, act=act, dx_dtype=torch.float32)
        assert ((dx[:, 0].double() - slope).abs() <= half(torch.bfloat16) * slope.abs() + 2 * ACT * U * mag + tiny).all()
        assert ((dx[:, 1].double() - value).abs() <= half(torch.bfloat16) * value.abs() * (1 + ACT * U) + ACT * U * value.abs() + tiny).all()
    # beyond all of that, the limits
    x[:, 0] = 1e30
    x[::2, 0] = -1e30
    h = fq.gated_linear(x, w, act=act, out_dtype=torch.float32)
    assert (h[::2] == 0).all() and (h[1::2] == x[1::2, :1].float()).all()


def test_keep_raises_its_own_error():
    """keep is taken for its truth, and an object that has none raises its own error."""
    x, w = torch.ones((2, 8), device="cuda").bfloat16(), torch.ones((16, 8), device="cuda").bfloat16()

    class Neither:
        def __bool__(self):
            raise KeyError("neither")
    with pytest.raises(KeyError, match="neither"):
        fq.gated_linear(x, w, keep=Neither())
    assert len(fq.gated_linear(x, w, keep=1)) == 2 and torch.is_tensor(fq.gated_linear(x, w, keep=[]))


def test_output_over_an_argument_is_refused():
    """y may be what it is added to; over anything else that is read while it is written there is no result."""
    g = rng(4)
    M, K, r = 70, 64, 8
    x, w, a, b = randn(g, M, K), randn(g, K, K), randn(g, 2, r, K), randn(g, 2, K, r)
    ids = torch.zeros(M, device="cuda", dtype=torch.int32)
    buffer = torch.zeros(4 * M * K, device="cuda").bfloat16()
    y, shifted = buffer[:M * K].view(M, K), buffer[8:8 + M * K].view(M, K)
    for bad in (lambda: fq.adapter_linear(x, w, a, b, ids, out=x), lambda: fq.adapter_linear(y, w, a, b, ids, out=shifted),
                lambda: fq.adapter_linear(x, y[:K], a, b, ids, out=y), lambda: fq.adapter_add(y, x, a, b, ids, out=shifted),
                lambda: fq.adapter_add(x, x, a, y[:16].view(2, K, r), ids, out=y),
                lambda: fq.adapter_add(x, x, a, b, y.view(-1)[:2 * M].view(torch.int32), out=y)):
        with pytest.raises(ValueError, match="overlap"):
            bad()
    want = fq.adapter_add(x, x, a, b, ids)
    assert torch.equal(fq.adapter_add(x.clone(), x, a, b, ids, out=y), want)
    assert torch.equal(fq.adapter_add(y.copy_(x), x, a, b, ids, out=y), want)
    z = x.clone()
    assert torch.equal(fq.adapter_add(x, z, a, b, ids, out=z), want)      # (x is read before)
    assert fq.adapter_linear(x[:0], w, a, b, ids[:0], out=x[:0]).shape == (0, K)


def test_one_row_without_a_leading_dimension_and_none():
    """x [K] is one row, with ids of no dimension; a leading dimension of 0 is no row."""
    g = rng(6)
    x, y, w, a, b = randn(g, 64), randn(g, 64), randn(g, 128, 64), randn(g, 2, 8, 64), randn(g, 2, 64, 8)
    ids = torch.tensor(1, device="cuda", dtype=torch.int32)
    v = torch.rand(64, device="cuda")
    row = lambda t: t.view(1, -1)    # noqa: E731
    pairs = [(fq.rms_norm(x, v), fq.rms_norm(row(x), v)),
             (fq.residual_norm(x, y, v, gate=y), fq.residual_norm(row(x), row(y), v, gate=row(y))),
             (fq.residual_norm(x.float(), y.float(), v, gate=v), fq.residual_norm(row(x.float()), row(y.float()), v, gate=v)),
             (fq.residual_norm_backward(x, y, x, y, v, gate=v, post=v), fq.residual_norm_backward(row(x), row(y), row(x), row(y), v, gate=v, post=v)),
             (fq.gated_linear(x, w), fq.gated_linear(row(x), w)),
             (fq.gated_linear_backward(y, x, w, wide=True), fq.gated_linear_backward(row(y), row(x), w, wide=True)),
             (fq.adapter_linear(x, w, a, torch.cat([b, b], 1), ids), fq.adapter_linear(row(x), w, a, torch.cat([b, b], 1), row(ids)[0])),
             (fq.adapter_add(y, x, a, b, ids), fq.adapter_add(row(y), row(x), a, b, row(ids)[0]))]
    for one, many in pairs:
        for p, q in zip(one if isinstance(one, tuple) else (one,), many if isinstance(many, tuple) else (many,)):
            assert p.numel() == q.numel() and torch.equal(p.view(-1), q.view(-1))
    none = torch.empty((3, 0, 64), device="cuda").bfloat16()
    assert fq.rms_norm(none, v).shape == fq.adapter_linear(none, w[:64], a, b, ids.expand(3, 0).contiguous()).shape == none.shape
    dx, dw = fq.gated_linear_backward(none, none, w, wide=True)
    assert dx.shape == none.shape and dw.shape == w.shape and (dw == 0).all()
