"""The dense block's operators at the ends of their documented range and where single elements are not finite,
against 64 bits.

Tolerances: half(t) is half a step of t relative to the value; U = 2^-24 is fp32's. The matrix unit adds
32 products at a time, with every product and addition off by at most 2 U: a sum over K is off by at most
2 (K / 32 + 32) U of the sum of its terms' magnitudes. The activations of the kernels are some 35 fp32
operations on the hardware's exponential and reciprocal, each within one unit in the last place (2 U), and a
polynomial fitted to 7e-8 (1.2 U): 16 U relative covers the few of them that carry the result's full size.
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
