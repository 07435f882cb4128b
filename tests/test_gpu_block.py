"""GPU parity of the dense block's operators against plain implementations in 64 bits.

Tolerances count roundings. u = 2^-24 is fp32's half step, half(t) the output type's
(finfo.eps / 2), each relative to the value; sums add at most one u a term and level to the sum of
the terms' magnitudes:

* rows: a row's sum is 8 to 32 terms a thread, 6 steps within a wave and 8 across waves, so fewer than
  48 u of its magnitudes, of which a square root halves the effect; each output has some 10 steps
  more. ROW = 64 covers both. Sums over T rows add one u a row of a workgroup (T / 256 of them, or 32)
  and 32 for the partial sums.
* products: the matrix unit adds 32 products to a sum at a time; with every product and every such
  addition off by 2 u (a unit that cuts off instead of rounding) the sum is off by 2 (K / 32 + 32) u of
  sum |x w|.
* activations: expf and erfcf within 4 units in the last place, 4 more steps: ACT = 16. Slopes of
  SiLU and GELU stay below 1.13, their second derivatives below 0.8 (2 / sqrt(2 pi), GELU at 0).
* the gradient's products take the projections' gradient rounded to bf16.
"""
import math

import pytest
import torch

import fp8_act_quant_amd as fq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROW, ACT = 64, 16
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def near(got, ref, slack, name=""):
    """Every element within its output's rounding and `slack` (an fp32 rounding error) of ref."""
    assert got.shape == ref.shape
    off = (got.double() - ref).abs()
    limit = half(got.dtype) * (ref.abs() + slack) + slack + 1e-37
    assert torch.isfinite(got).all(), name
    assert (off <= limit).all(), (name, float((off / limit).max()))


# ---- norms ---------------------------------------------------------------------------------

def norm64(v, mag, w):
    """norm(v) * w, and how far it is off (in units of ROW u) where v is off by as much of `mag`."""
    r = 1.0 / (v.square().mean(-1, keepdim=True) + EPS).sqrt()
    spread = mag.norm(dim=-1, keepdim=True) / v.norm(dim=-1, keepdim=True).clamp(min=1e-300)
    return v * r * w, w.abs() * r * (mag + v.abs() * (1 + spread))


def forward64(x, y, weight, post, gate, scale):
    x, y = x.double(), y.double()
    n, mag = (y, y.abs()) if post is None else norm64(y, y.abs(), post.double())
    c = 1.0 if gate is None else gate.double()
    t = scale * x + c * n
    mag_t = abs(scale) * x.abs() + (c if gate is None else c.abs()) * mag
    z = None if weight is None else norm64(t, mag_t, weight.double())
    return t, mag_t, z


def norm_inputs(T, H, dtype, post, gate, seed):
    g = rng(seed)
    s = dict(x=randn(g, T, H, std=3.0, dtype=dtype), y=randn(g, T, H, std=0.5, dtype=dtype),
             weight=1 + 0.1 * randn(g, H, dtype=torch.float32), post=None, gate=None)
    if post:
        s["post"] = 1 + 0.1 * randn(g, H, dtype=torch.float32)
    if gate == "channel":
        s["gate"] = 0.5 + 0.2 * randn(g, H, dtype=torch.float32)
    elif gate == "element":
        s["gate"] = (0.5 + 0.2 * randn(g, T, H, dtype=torch.float32)).to(dtype)
    return s


SHAPES = [(1, 8), (3, 9), (5, 64), (2, 511), (7, 512), (9, 513), (4, 1023), (130, 1024), (6, 1091), (33, 2048),
          (5, 2055), (300, 4096), (3, 4100), (1, 7168), (600, 7168), (17, 8191), (2, 8193), (4, 16383), (259, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_residual_norm(T, H, dtype):
    for k, (post, gate) in enumerate([(True, "channel"), (False, None), (True, "element"), (False, "channel")]):
        s = norm_inputs(T, H, DT[dtype], post, gate, 10 * H + k)
        scale = (1.0, 0.75, -0.3, 1.0)[k]
        t, z = fq.residual_norm(s["x"], s["y"], s["weight"], post=s["post"], gate=s["gate"], scale=scale, eps=EPS)
        rt, mag, (rz, mag_z) = forward64(scale=scale, **s)
        near(t, rt, ROW * U * mag, "t")
        near(z, rz, ROW * U * mag_z, "z")
        t2, none = fq.residual_norm(s["x"], s["y"], post=s["post"], gate=s["gate"], scale=scale, eps=EPS)
        assert none is None and torch.equal(t, t2)
    z = fq.rms_norm(s["x"], s["weight"], eps=EPS)
    rz, mag_z = norm64(s["x"].double(), s["x"].double().abs(), s["weight"].double())
    near(z, rz, ROW * U * mag_z, "rms_norm")


def backward64(dt, dz, t, y, weight, post, gate, scale):
    """The gradients and their magnitudes: each sum's terms by their absolute values."""
    t, y = t.double(), y.double()
    d = mag = torch.zeros_like(t)
    if dt is not None:
        d, mag = dt.double(), dt.double().abs()
    out = {}
    if weight is not None:
        r = 1.0 / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
        th, a = t * r, dz.double() * weight.double()
        d = d + r * (a - th * (a * th).mean(-1, keepdim=True))
        mag = mag + r * (a.abs() + th.abs() * (a * th).abs().mean(-1, keepdim=True) * 2)
        out["dweight"] = (dz.double() * th).sum(0), (dz.double() * th).abs().sum(0)
    out["dx"] = scale * d, abs(scale) * mag
    q = 1.0 / (y.square().mean(-1, keepdim=True) + EPS).sqrt() if post is not None else 1.0
    yh = y * q
    n = yh if post is None else yh * post.double()
    dn, mag_n = d, mag
    if gate is not None:
        c = gate.double()
        dn, mag_n = d * c, mag * c.abs()
        dg, mag_g = d * n, mag * n.abs()
        out["dgate"] = (dg, mag_g) if gate.dim() == 2 else (dg.sum(0), mag_g.sum(0))
    if post is None:
        out["dy"] = dn, mag_n
    else:
        out["dpost"] = (dn * yh).sum(0), (mag_n * yh.abs()).sum(0)
        b, mag_b = dn * post.double(), mag_n * post.double().abs()
        out["dy"] = (q * (b - yh * (b * yh).mean(-1, keepdim=True)),
                     q * (mag_b + yh.abs() * (mag_b * yh.abs()).mean(-1, keepdim=True) * 2))
    return out


NAMES = ("dx", "dy", "dweight", "dpost", "dgate")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES + [(1500, 300), (9000, 200), (2047, 1091)])
def test_residual_norm_backward(T, H, dtype):
    rows = max(32, T // 256 + 1) + 32
    for k, (post, gate, with_dt, with_z) in enumerate([(True, "channel", True, True), (False, None, True, True),
                                                       (True, "element", False, True), (False, "channel", True, False),
                                                       (True, None, True, False)]):
        s = norm_inputs(T, H, DT[dtype], post, gate, 10 * H + k)
        g = rng(H + k)
        t = s.pop("x")
        if not with_z:
            s["weight"] = None
        dt = randn(g, T, H, dtype=DT[dtype]) if with_dt else None
        dz = randn(g, T, H, dtype=DT[dtype]) if with_z else None
        scale = (1.0, 0.75, -0.3, 1.0, 1.0)[k]
        got = dict(zip(NAMES, fq.residual_norm_backward(dt, dz, t, s["y"], s["weight"], post=s["post"], gate=s["gate"],
                                                        scale=scale, eps=EPS)))
        ref = backward64(dt, dz, t, scale=scale, **s)
        for name in NAMES:
            assert (got[name] is None) == (name not in ref), name
            if name in ref:
                v, mag = ref[name]
                near(got[name], v, (ROW + (rows if v.dim() == 1 else 0)) * U * mag, name)
    dx, dweight = fq.rms_norm_backward(dz := randn(g, T, H, dtype=DT[dtype]), t, w := torch.rand(H, device="cuda"), eps=EPS)
    ref = backward64(None, dz, t, t, w, None, None, 1.0)
    near(dx, ref["dx"][0], ROW * U * ref["dx"][1], "dx")
    near(dweight, ref["dweight"][0], (ROW + rows) * U * ref["dweight"][1], "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 9000), (129, 10240), (600, 9001)])
def test_gradient_of_long_rows(T, H, dtype):
    test_residual_norm_backward(T, H, dtype)


def test_gradient_of_long_rows_is_its_own():
    """A NaN in one row stays in its row and in the sums; the same call gives the same bits."""
    g = rng(7)
    T, H = 300, 8200
    t, y, dz = (randn(g, T, H) for _ in range(3))
    w, post = torch.rand(H, device="cuda"), torch.rand(H, device="cuda")
    one, two = (fq.residual_norm_backward(None, dz, t, y, w, post=post) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one[:4], two[:4]))
    bad = y.clone()
    bad[77] = float("nan")
    dx, dy, dw, dp, _ = fq.residual_norm_backward(None, dz, t, bad, w, post=post)
    keep = torch.arange(T, device="cuda") != 77
    assert torch.equal(dx, one[0]) and torch.equal(dw, one[2]) and torch.equal(dy[keep], one[1][keep])
    assert torch.isnan(dy[77]).all() and torch.isnan(dp).all()


def test_norm_gradient_by_differences():
    """The formulas above, against differences of the forward formula in 64 bits."""
    g = rng(5)
    T, H = 3, 40
    x, y, weight, post, gate, dt, dz = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float64) for shape in
                                        ((T, H), (T, H), (H,), (H,), (H,), (T, H), (T, H)))

    def loss(x, y, weight, post, gate):
        t, _, (z, _) = forward64(x, y, weight, post, gate, 0.7)
        return float((t * dt).sum() + (z * dz).sum())
    t = forward64(x, y, weight, post, gate, 0.7)[0]
    got = backward64(dt, dz, t, y, weight, post, gate, 0.7)
    at = [x, y, weight, post, gate]
    for i, name in enumerate(NAMES):
        d = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = ([v + s * d if k == i else v for k, v in enumerate(at)] for s in (h, -h))
        want = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(want - float((got[name][0] * d).sum())) < 1e-6 * (1 + abs(want)), name


def test_norm_rows_of_zeros_and_large_values():
    x = torch.zeros((3, 100), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(100, device="cuda")
    assert (fq.rms_norm(x, w) == 0).all()
    t, z = fq.residual_norm(x, x, w, post=w)
    assert (t == 0).all() and (z == 0).all()
    # a row's infinities and NaN stay in the row
    x[1, 5] = float("inf")
    x[0] = 1.0
    z = fq.rms_norm(x, w)
    assert torch.isnan(z[1, 5]) and (z[2] == 0).all() and (z[0] == 1.0).all()


def test_norm_in_place_and_any_alignment():
    """t may be x; rows that start off a 16-byte boundary; nothing outside the outputs is written."""
    g = rng(11)
    for dtype, per in ((torch.bfloat16, 1), (torch.float32, 1)):
        T, H = 37, 515
        buf = randn(g, T * H + 16, dtype=dtype)
        x, y = buf[per:per + T * H].view(T, H), randn(g, T, H, dtype=dtype)
        w = torch.rand(H, device="cuda")
        want, z = fq.residual_norm(x, y, w, scale=0.5)
        first, last = buf[:per].clone(), buf[per + T * H:].clone()
        z2 = torch.empty_like(z)
        code = 1 if dtype == torch.bfloat16 else 0
        assert fq.lib.residual_norm(x.data_ptr(), y.data_ptr(), code, w.data_ptr(), None, None, 0, 0.5, EPS,
                                    x.data_ptr(), z2.data_ptr(), T, H, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(x, want) and torch.equal(z, z2)
        assert torch.equal(buf[:per], first) and torch.equal(buf[per + T * H:], last)


def test_norm_empty():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    t, z = fq.residual_norm(x, x, w, post=w, gate=w)
    assert t.shape == z.shape == (0, 64)
    dx, dy, dw, dp, dg = fq.residual_norm_backward(x, x, x, x, w, post=w, gate=w)
    assert dx.shape == dy.shape == (0, 64) and (dw == 0).all() and (dp == 0).all() and (dg == 0).all()


# ---- gated projections ---------------------------------------------------------------------

def act64(a, kind):
    if kind == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    p = 0.5 * torch.erfc(-a / math.sqrt(2))
    return a * p, p + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)


def product64(x, w):
    """x w^T and how far its fp32 sum may be off."""
    x, w = x.double(), w.double()
    return x @ w.t(), 2 * (x.shape[1] / 32 + 32) * U * (x.abs() @ w.abs().t())


def projections64(x, w):
    gu, off = product64(x, w)
    F = w.shape[0] // 2
    return gu[:, :F], gu[:, F:], off[:, :F], off[:, F:]


GATED = [(1, 8, 8), (1, 128, 64), (1, 2048, 7168), (2, 40, 72), (3, 1000, 1096), (15, 24, 520), (16, 136, 136), (17, 8, 64),
         (31, 264, 1032), (48, 2048, 1536), (64, 200, 64), (65, 1032, 264), (129, 512, 8), (200, 96, 1536),
         (257, 2048, 1096), (333, 1000, 1096), (1000, 584, 200), (1021, 4096, 136), (2050, 2048, 264), (4099, 1544, 136)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_linear(M, F, K, out):
    g = rng(M + F + K)
    x, w = randn(g, M, K), randn(g, 2 * F, K, std=1.5 * K ** -0.5)
    a, b, off_a, off_b = projections64(x, w)
    for act in ("silu", "gelu"):
        h, gu = fq.gated_linear(x, w, act=act, keep=True, out_dtype=DT[out])
        assert h.dtype == DT[out] and gu.dtype == torch.bfloat16
        p, _ = act64(a, act)
        near(h, p * b, 1.13 * off_a * b.abs() + (p.abs() + 1.13 * off_a) * off_b + ACT * U * (p * b).abs(), act)
        near(gu, torch.cat([a, b], -1), torch.cat([off_a, off_b], -1), "gu")
        assert torch.equal(h, fq.gated_linear(x, w, act=act, out_dtype=DT[out]))


@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_linear_backward(M, F, K):
    g = rng(M + F + K + 1)
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=1.5 * K ** -0.5), randn(g, M, F)
    gu = fq.gated_linear(x, w, keep=True)[1]
    for k, (act, kept, dt) in enumerate([("silu", True, torch.bfloat16), ("gelu", False, torch.float32),
                                         ("gelu", True, torch.float32), ("silu", False, torch.bfloat16)]):
        dx, dw = fq.gated_linear_backward(dh, x, w, gu if kept else None, act=act, dx_dtype=dt, dw_dtype=dt)
        assert dx.dtype == dw.dtype == dt
        if kept:
            a, b = gu.double()[:, :F], gu.double()[:, F:]
            off_a = off_b = torch.zeros_like(a)
        else:
            a, b, off_a, off_b = projections64(x, w)
        p, s = act64(a, act)
        e = dh.double().abs()
        d = torch.cat([dh.double() * b * s, dh.double() * p], -1)
        # (the slope's terms p and a p' are of either sign: their magnitudes bound the slope's error)
        mags = torch.cat([e * b.abs() * (1.13 + a.abs().clamp(max=1.13)), e * p.abs()], -1)
        off = torch.cat([e * ((b.abs() + off_b) * 0.8 * off_a + 1.13 * off_b), e * 1.13 * off_a], -1) + ACT * U * mags
        off = off + half(torch.bfloat16) * (d.abs() + off)
        for got, ref, terms, slack in (
                (dx, d @ w.double(), 2 * F, off @ w.double().abs()),
                (dw, d.t() @ x.double(), M, off.t() @ x.double().abs())):
            sums = (d.abs() + off) @ w.double().abs() if got is dx else (d.abs() + off).t() @ x.double().abs()
            near(got, ref, slack + 2 * (terms / 32 + 32) * U * sums, (act, kept))
            if M * F > 4096:   # roundings of either sign: in the mean far less than their bound
                assert float((got.double() - ref).norm() / ref.norm()) < half(torch.bfloat16)


def test_gated_gradient_by_differences():
    """The slopes above, against differences of the activations in 64 bits."""
    a = torch.linspace(-12, 12, 4001, dtype=torch.float64, device="cuda")
    for act in ("silu", "gelu"):
        want = (act64(a + 1e-5, act)[0] - act64(a - 1e-5, act)[0]) / 2e-5
        slope = act64(a, act)[1]
        assert float((want - slope).abs().max()) < 1e-8 and float(slope.abs().max()) < 1.13


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_large_projections(act):
    """Far on either side of zero the activation is 0 or its argument, and the gradient finite."""
    x = torch.tensor([[300.0], [-300.0], [30.0], [-30.0], [1e4], [-1e4], [0.0]], device="cuda").bfloat16() @ \
        torch.ones((1, 8), device="cuda").bfloat16()
    w = torch.full((16, 8), 0.125, device="cuda").bfloat16()
    h = fq.gated_linear(x, w, act=act, out_dtype=torch.float32)
    a = x.double()
    near(h, act64(a, act)[0] * a, ACT * U * (act64(a, act)[0] * a).abs() + 300 * 2 * 33 * U)
    dx, dw = fq.gated_linear_backward(torch.ones((7, 8), device="cuda").bfloat16(), x, w, act=act)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations(act):
    """Every bf16 number from -90 to 90 as the gate's projection, the other one 1: the activation itself in fp32,
    and its slope. Below fp32's normal range results may be 0."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32, device="cuda").to(torch.int16)
    a = bits.view(torch.bfloat16)
    a = a[(a.abs() <= 90) & (a.abs() >= 1e-30) | (a == 0)]
    x = torch.zeros((a.numel(), 8), device="cuda").bfloat16()
    x[:, 0], x[:, 1] = a, 1.0
    w = torch.zeros((16, 8), device="cuda").bfloat16()
    w[:8, 0] = w[8:, 1] = 1.0
    h, gu = fq.gated_linear(x, w, act=act, keep=True, out_dtype=torch.float32)
    assert torch.equal(gu[:, 0], a) and (gu[:, 8:] == 1).all()
    value, slope = act64(a.double(), act)
    tiny = 100 * 2.0 ** -126
    assert ((h[:, 0].double() - value).abs() <= ACT * U * value.abs() + tiny).all()
    # dg = slope, du = act of one row at a time come back as dx = [dg du] w
    one = torch.zeros((a.numel(), 8), device="cuda").bfloat16()
    one[:, 3] = 1.0
    dx, _ = fq.gated_linear_backward(one, x, w, gu, act=act, dx_dtype=torch.float32)
    again, _ = fq.gated_linear_backward(one, x, w, None, act=act, dx_dtype=torch.float32)
    assert torch.equal(dx, again)
    mag = torch.sigmoid(a.double()) if act == "silu" else 0.5 * torch.erfc(-a.double() / math.sqrt(2))
    mag = mag + (slope - mag).abs()
    assert ((dx[:, 0].double() - slope).abs() <= half(torch.bfloat16) * slope.abs() + ACT * U * mag * 2 + tiny).all()
    assert ((dx[:, 1].double() - value).abs() <= half(torch.bfloat16) * value.abs() * (1 + ACT * U) + ACT * U * value.abs() + tiny).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_specials(act):
    """+inf is itself, NaN stays NaN in its row, and neither reaches another row."""
    x = torch.zeros((3, 8), device="cuda").bfloat16()
    x[0, 0], x[1, 0], x[2, 0] = float("inf"), float("nan"), 2.0
    w = torch.zeros((16, 8), device="cuda").bfloat16()
    w[:8, 0], w[8:, 1] = 1.0, 1.0
    x[:, 1] = 1.0
    h, gu = fq.gated_linear(x[:, :].clone(), w, act=act, keep=True)
    # (inf * 0 in the up projection: w's zeros meet x's infinities)
    dx, dw = fq.gated_linear_backward(torch.ones((1, 8), device="cuda").bfloat16(), x[2:].clone(), w, gu[2:].clone(), act=act)
    assert torch.isnan(h[1]).all() and torch.isfinite(h[2]).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    w[8:, 0] = 1.0   # both projections infinite
    h = fq.gated_linear(x, w, act=act)
    assert (h[0] == float("inf")).all() and torch.isnan(h[1]).all() and torch.isfinite(h[2]).all()


def test_gated_empty():
    def e(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    assert fq.gated_linear(e(0, 64), e(32, 64)).shape == (0, 16)
    assert fq.gated_linear(e(3, 64), e(0, 64)).shape == (3, 0)
    for M in (3, 200):
        h, gu = fq.gated_linear(e(M, 0), e(32, 0), keep=True)
        assert (h == 0).all() and (gu == 0).all() and h.shape == (M, 16)
    dx, dw = fq.gated_linear_backward(e(0, 16), e(0, 64), e(32, 64))
    assert dx.shape == (0, 64) and dw.shape == (32, 64) and (dw == 0).all()
    dx, dw = fq.gated_linear_backward(e(5, 0), e(5, 64), e(0, 64))
    assert (dx == 0).all() and dw.shape == (0, 64)


@pytest.mark.parametrize("M", [5, 40, 300])
def test_gated_reads_and_writes_only_its_own(M):
    """Operands that end where their allocation does, whose neighbours are NaN; outputs between guards."""
    g = rng(M)
    F, K = 72, 200
    nan = torch.full((M * K + 2 * F * K + 512,), float("nan"), device="cuda").bfloat16()
    x, w = nan[64:64 + M * K].view(M, K), nan[128 + M * K:128 + M * K + 2 * F * K].view(2 * F, K)
    x.copy_(randn(g, M, K))
    w.copy_(randn(g, 2 * F, K, std=0.1))
    assert x.data_ptr() % 16 == 0 and w.data_ptr() % 16 == 0
    a, b, off_a, off_b = projections64(x, w)
    h = torch.full((M * F + 64,), 7.0, device="cuda").bfloat16()
    gu = torch.full((M * 2 * F + 64,), 7.0, device="cuda").bfloat16()
    assert fq.lib.gated_linear(x.data_ptr(), w.data_ptr(), h[2:].data_ptr(), 1, gu[2:].data_ptr(), 0, M, F, K,
                               torch.cuda.current_stream().cuda_stream) == 0
    p, _ = act64(a, "silu")
    near(h[2:2 + M * F].view(M, F), p * b, 1.13 * off_a * b.abs() + (p.abs() + off_a) * off_b + ACT * U * (p * b).abs())
    near(gu[2:2 + M * 2 * F].view(M, 2 * F), torch.cat([a, b], -1), torch.cat([off_a, off_b], -1))
    for t, n in ((h, M * F), (gu, M * 2 * F)):
        assert (t[:2] == 7).all() and (t[2 + n:] == 7).all()
    dh = randn(g, M, F)
    want = fq.gated_linear_backward(dh, x.clone(), w.clone())
    got = fq.gated_linear_backward(dh, x, w)
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and torch.isfinite(got[1]).all()


# ---- adapters ------------------------------------------------------------------------------

def adapters64(x, w, a, b, ids, scales, bias, base):
    """y and how far its fp32 form may be off."""
    if base is None:
        y, off = product64(x, w)
    else:
        y, off = base.double(), U * base.double().abs()
    if bias is not None:
        y = y + bias.double()
        off = off + U * bias.double().abs()
    for e in range(a.shape[0]):
        at = (ids == e).nonzero()[:, 0]
        if at.numel():
            u, off_u = product64(x[at], a[e])
            s = 1.0 if scales is None else float(scales[e])
            u, off_u = s * u, abs(s) * (off_u + 2 * U * u.abs())
            bd = b[e].double()
            y[at] += u @ bd.t()
            off[at] += off_u @ bd.abs().t() + 2 * (3 * a.shape[1] / 32 + 32) * U * (u.abs() @ bd.abs().t())
    return y, off + 4 * U * y.abs()


def adapter_inputs(M, N, K, L, r, order, seed):
    g = rng(seed)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    if order == "runs":
        ids = ids[(torch.arange(M, device="cuda") // 23)]
    elif order == "one":
        ids = torch.full_like(ids, L - 1)
    elif order == "none":
        ids = torch.where(ids > 0, 2 ** 31 - 1, -2 ** 31).to(torch.int32)
    return dict(x=randn(g, M, K), a=randn(g, L, r, K, std=max(K, 1) ** -0.5), b=randn(g, L, N, r, std=0.3), ids=ids,
                scales=0.5 + torch.rand(L, generator=g, device="cuda"), w=randn(g, N, K, std=max(K, 1) ** -0.5),
                bias=torch.randn(N, generator=g, device="cuda"))


ADAPTERS = [(1, 1, 8, 1, 8, "one"), (1, 7168, 1536, 4, 16, "one"), (2, 33, 72, 3, 24, "mixed"), (7, 100, 520, 40, 64, "mixed"),
            (16, 1000, 264, 16, 16, "mixed"), (16, 64, 1536, 5, 256, "mixed"), (17, 65, 136, 7, 8, "mixed"),
            (48, 1533, 1096, 32, 16, "mixed"), (64, 300, 64, 2, 40, "none"), (100, 5000, 264, 9, 32, "mixed"),
            (130, 129, 136, 30, 64, "mixed"), (200, 1000, 1032, 1, 128, "one"), (257, 257, 200, 12, 24, "runs"),
            (300, 2001, 328, 60, 16, "mixed"), (513, 1536, 520, 8, 64, "runs"), (1021, 1533, 136, 12, 24, "runs"),
            (1030, 7168, 136, 300, 8, "mixed"), (2050, 4100, 264, 8, 72, "runs"), (4100, 2048, 72, 64, 136, "mixed")]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,L,r,order", ADAPTERS)
def test_adapter_linear(M, N, K, L, r, order, out):
    s = adapter_inputs(M, N, K, L, r, order, M + N + K)
    y = fq.adapter_linear(**s, out_dtype=DT[out])
    assert y.dtype == DT[out]
    near(y, *adapters64(**s, base=None), "linear")
    s["bias"] = s["scales"] = None
    near(fq.adapter_linear(**s, out_dtype=DT[out]), *adapters64(**s, base=None), "without scales and bias")
    s["w"] = None
    base = randn(rng(M), M, N, dtype=DT[out])
    args = [s[k] for k in ("x", "a", "b", "ids", "scales")]
    got = fq.adapter_add(base, *args)
    near(got, *adapters64(**s, base=base), "add")
    assert got.data_ptr() != base.data_ptr()
    if order == "none":
        assert torch.equal(got, base)
    inside = base.clone()
    assert fq.adapter_add(inside, *args, out=inside) is not None and torch.equal(inside, got)


def test_adapter_rows_are_their_own():
    """What one adapter, or one row, holds (infinities, NaN) does not reach the rows of others."""
    for M in (5, 40, 700):
        s = adapter_inputs(M, 200, 136, 6, 24, "mixed", M)
        y = fq.adapter_linear(**s)
        bad = {k: s[k].clone() for k in ("a", "b", "scales")}
        bad["a"][2], bad["b"][3], bad["scales"][4] = float("nan"), float("inf"), float("nan")
        z = fq.adapter_linear(**{**s, **bad})
        touched = (s["ids"] >= 2) & (s["ids"] <= 4)
        assert torch.equal(y[~touched], z[~touched])
        assert not torch.isfinite(z[touched]).all(dim=-1).any()
        x = s["x"].clone()
        x[0] = float("inf")
        z = fq.adapter_linear(**{**s, "x": x})
        assert torch.equal(y[1:], z[1:])


@pytest.mark.parametrize("M,N", [(40, 200), (130, 200), (513, 1536), (1030, 7168)])
def test_adapters_added_are_their_own(M, N):
    """The same beside another projection; rows without an adapter, and calls without any, keep their bits."""
    s = adapter_inputs(M, N, 136, 6, 64, "mixed", M)
    base = randn(rng(M), M, N)
    args = [s[k] for k in ("x", "a", "b", "ids", "scales")]
    y = fq.adapter_add(base, *args)
    a, b, scales = (s[k].clone() for k in ("a", "b", "scales"))
    a[2], b[3], scales[4] = float("nan"), float("inf"), float("nan")
    z = fq.adapter_add(base, s["x"], a, b, s["ids"], scales)
    touched = (s["ids"] >= 2) & (s["ids"] <= 4)
    assert torch.equal(y[~touched], z[~touched])
    assert not torch.isfinite(z[touched]).all(dim=-1).any()
    no = (s["ids"] < 0) | (s["ids"] >= 6)
    assert no.any() and torch.equal(y[no], base[no])
    assert torch.equal(fq.adapter_add(base, s["x"], a[:0], b[:0], s["ids"], scales[:0]), base)


def test_adapter_sums_keep_fp32():
    """x a^T of 24 bits: with W zero and b one, fp32 output holds it to the last bit but one."""
    g = rng(3)
    for M in (3, 300):
        K, r = 264, 8
        x, a = randn(g, M, K), torch.zeros((1, r, K), device="cuda").bfloat16()
        a[0, 0] = randn(g, K)
        b = torch.zeros((1, 130, r), device="cuda").bfloat16()
        b[0, :, 0] = 1.0
        y = fq.adapter_linear(x, torch.zeros((130, K), device="cuda").bfloat16(), a, b,
                              torch.zeros(M, device="cuda", dtype=torch.int32), out_dtype=torch.float32)
        ref, off = product64(x, a[0, :1])
        assert (y == y[:, :1]).all()
        assert ((y[:, :1].double() - ref).abs() <= off).all()


def test_adapter_infinite_sums():
    """An infinite x a^T gives infinities, not NaN, where b is finite."""
    for M in (3, 300):
        x = torch.full((M, 64), 3e38, device="cuda").bfloat16()
        a, b = torch.ones((1, 8, 64), device="cuda").bfloat16(), torch.ones((1, 40, 8), device="cuda").bfloat16()
        ids = torch.zeros(M, device="cuda", dtype=torch.int32)
        y = fq.adapter_linear(x, torch.zeros((40, 64), device="cuda").bfloat16(), a, b, ids)
        assert (y == float("inf")).all()


def test_adapter_empty():
    s = adapter_inputs(5, 40, 64, 3, 8, "mixed", 1)
    plain = fq.adapter_linear(s["x"], s["w"], s["a"][:0], s["b"][:0], s["ids"], bias=s["bias"])
    none = fq.adapter_linear(**{**s, "ids": torch.full_like(s["ids"], -1)})
    assert torch.equal(plain, none)
    assert fq.adapter_linear(s["x"][:0], s["w"], s["a"], s["b"], s["ids"][:0]).shape == (0, 40)
    for M in (5, 300):
        t = adapter_inputs(M, 40, 0, 3, 8, "mixed", 1)
        assert torch.equal(fq.adapter_linear(**t, out_dtype=torch.float32), t["bias"].expand(M, 40))
    assert fq.adapter_linear(s["x"], s["w"][:0], s["a"], s["b"][:, :0], s["ids"]).shape == (5, 0)


def test_leading_dimensions():
    g = rng(9)
    x = randn(g, 2, 3, 64)
    w, wn = randn(g, 32, 64), torch.rand(64, device="cuda")
    h = fq.gated_linear(x, w)
    assert torch.equal(h.view(6, 16), fq.gated_linear(x.view(6, 64), w)) and h.shape == (2, 3, 16)
    dx, _ = fq.gated_linear_backward(h, x, w)
    assert dx.shape == x.shape
    assert torch.equal(fq.rms_norm(x, wn).view(6, 64), fq.rms_norm(x.view(6, 64), wn))
    a, b = randn(g, 2, 8, 64), randn(g, 2, 16, 8)
    ids = torch.tensor([[0, 1, -1], [1, 1, 0]], device="cuda", dtype=torch.int32)
    y = fq.adapter_linear(x, w[:16], a, b, ids)
    assert torch.equal(y.view(6, 16), fq.adapter_linear(x.view(6, 64), w[:16], a, b, ids.view(6)))
