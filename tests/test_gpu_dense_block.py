"""The dense block's operators together, as examples/dense_block.py runs them: forward with and without adapters,
gradient, captured in a graph, on other streams; and the operators at offsets past 32 bits.

Forward, against float64: n, h, y and t are each rounded to bf16 (at most 2^-8 of a value, some 0.42 times
that in rms): four roundings in a row are below 2^-8 in rms. With FP8 weights and activations of the
down-projection each product's two operands are off by 2.6% rms, 8-bit integers by 1%, of the block's
part of t: 5% and 2.5% bound them. A gradient passes up to six such roundings, 2^-7 bounds it.
"""
import importlib.util
import os

import pytest
import torch

import fp8_act_quant_amd as fq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("dense_block", os.path.join(ROOT, "examples", "dense_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(T, H, L, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    return x, torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("weights,limit", [("bf16", 2.0 ** -8), ("fp8", 0.05), ("int8", 0.025)])
@pytest.mark.parametrize("T", [1, 40, 333])
def test_forward(example, T, weights, limit, act):
    args, lora = example.example_weights(256, 384, adapters=5, seed=T)
    block = example.DenseBlock(*args, adapters=lora, scale=0.75, act=act, down_weights=weights)
    x, ids = inputs(T, 256, 5, T)
    for rows in (None, ids):
        got, ref = block(x, rows), example.plain(block, x, rows)
        for y, r in zip(got, ref):
            assert float((y.double() - r).norm()) <= limit * float(r.norm())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient(example, act):
    """Against torch's autograd of the plain block in float64."""
    T, H = 100, 256
    args, _ = example.example_weights(H, 384, seed=3)
    block = example.DenseBlock(*args, scale=0.75, act=act)
    x, _ = inputs(T, H, 1, 4)
    dt, dz = inputs(T, H, 1, 5)[0], inputs(T, H, 1, 6)[0]
    block(x, keep=True)
    got = block.gradient(dt, dz)
    wide = example.DenseBlock(*(v.double().requires_grad_() for v in args), scale=0.75, act=act)
    leaf = x.double().requires_grad_()
    t, z = example.plain(wide, leaf)
    ((t * dt.double()).sum() + (z * dz.double()).sum()).backward()
    want = dict(x=leaf.grad, up=wide.up.grad, down=wide.down.grad, before=wide.before.grad, after=wide.after.grad,
                next=wide.next.grad, gate=wide.gate.grad)
    for name, ref in want.items():
        assert float((got[name].double() - ref).norm() / ref.norm()) < 2.0 ** -7, name


def test_captured(example):
    """Forward and gradient captured once and replayed with other inputs, between eager work."""
    T, H, L = 70, 256, 5
    args, lora = example.example_weights(H, 384, adapters=L, seed=1)
    block = example.DenseBlock(*args, adapters=lora)
    x, ids = inputs(T, H, L, 0)
    dt, dz = inputs(T, H, 1, 1)[0], inputs(T, H, 1, 2)[0]

    def step():
        t, z = block(x, ids)
        n = fq.rms_norm(x, block.before)
        h, gu = fq.gated_linear(n, block.up, keep=True)
        back = fq.residual_norm_backward(dt, dz, t, t, block.next, post=block.after, gate=block.gate)
        grads = fq.gated_linear_backward(h, n, block.up, gu) + fq.gated_linear_backward(h, n, block.up)
        return (t, z, h) + tuple(back) + tuple(grads)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        nx, nids = inputs(T, H, L, 10 + k)
        x.copy_(nx)
        ids.copy_(nids)
        graph.replay()
        torch.cuda.synchronize()
        again = [v.clone() for v in out]
        eager = step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(again, eager)):
            assert torch.equal(a, b), (k, i)


def test_streams(example):
    """Calls that overlap on two streams of one device, each with its own outputs and workspaces."""
    args, lora = example.example_weights(1024, 1024, adapters=8, seed=2)
    block = example.DenseBlock(*args, adapters=lora)
    sets = [inputs(T, 1024, 8, T) for T in (30, 700)]
    dh = [torch.randn((T, 1024), device="cuda").bfloat16() for T in (30, 700)]

    def work(k):
        x, ids = sets[k]
        t, z = block(x, ids)
        return (t, z) + tuple(fq.gated_linear_backward(dh[k], x, block.up)) + \
            tuple(v for v in fq.residual_norm_backward(t, z, t, t, block.next, post=block.after) if v is not None)
    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(work(k))
        torch.cuda.synchronize()
        for k in (0, 1):
            for a, b in zip(want[k], got[k]):
                assert torch.equal(a, b)


def test_same_bits_twice(example):
    """No result depends on the order in which workgroups run."""
    args, lora = example.example_weights(1536, 1000, adapters=8, seed=7)
    block = example.DenseBlock(*args, adapters=lora)
    x, ids = inputs(1021, 1536, 8, 3)
    first = None
    for _ in range(3):
        t, z = block(x, ids, keep=False)
        h, gu = fq.gated_linear(x, block.up, keep=True)
        got = (t, z, h) + tuple(fq.gated_linear_backward(h, x, block.up, gu)) + \
            tuple(fq.residual_norm_backward(z, t, t, x, block.next, post=block.after, gate=block.gate))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_largest_tiles_last_round():
    """More of the largest tiles than the GPU takes at once, the last of them cut into halves, whose second half may
    have no rows (2305 of them): forward, gradient, adapters."""
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

    def close(y, ref, limit=2.0 ** -8):
        assert torch.isfinite(y).all() and float((y.double() - ref).norm()) <= limit * float(ref.norm())
        # and no element far off: 16 times the rms rounding of a sum of random terms
        assert float((y.double() - ref).abs().max()) <= 16 * limit * float(ref.abs().max())
    M, F, K = 2305, 3704, 1032
    x, w = randn(M, K), randn(2 * F, K, std=K ** -0.5)
    gu = x.double() @ w.double().t()
    h, kept = fq.gated_linear(x, w, keep=True)
    close(h, torch.nn.functional.silu(gu[:, :F]) * gu[:, F:])
    close(kept, gu)
    y = fq.adapter_linear(x, w, randn(2, 16, K, std=K ** -0.5), b := randn(2, 2 * F, 16), torch.full((M,), -1, device="cuda", dtype=torch.int32))
    close(y, gu)
    assert b.shape[1] == 2 * F
    del gu, h, kept, y
    M, F, K = 4099, 2056, 2304
    x, w, dh = randn(M, K), randn(2 * F, K, std=K ** -0.5), randn(M, F)
    gu = fq.gated_linear(x, w, keep=True)[1]
    a, u = gu.double()[:, :F], gu.double()[:, F:]
    s = torch.sigmoid(a)
    d = torch.cat([dh.double() * u * s * (1 + a * (1 - s)), dh.double() * a * s], -1)
    for got in (fq.gated_linear_backward(dh, x, w, gu, dw_dtype=torch.bfloat16), fq.gated_linear_backward(dh, x, w)):
        close(got[0], d @ w.double(), 2.0 ** -7)
        close(got[1], d.t() @ x.double(), 2.0 ** -7)


# ---- offsets past 32 bits ------------------------------------------------------------------

ROWS = (1 << 20) + 5


def sample():
    return torch.tensor([0, 1, 300_001, (1 << 19) + 3, ROWS - 6, ROWS - 1], device="cuda")


def test_norm_of_many_rows():
    H = 4104                                           # rows x H is past 2^32
    x = torch.empty((ROWS, H), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand(H, device="cuda")
    t, z = fq.residual_norm(x, x, w, scale=0.5)
    at = sample()
    small = fq.residual_norm(x[at], x[at], w, scale=0.5)
    assert torch.equal(t[at], small[0]) and torch.equal(z[at], small[1])
    del t, z
    dx, dy, dw, _, _ = fq.residual_norm_backward(x, x, x, x, w, scale=0.5)
    small = fq.residual_norm_backward(x[at], x[at], x[at], x[at], w, scale=0.5)
    assert torch.equal(dx[at], small[0]) and torch.equal(dy[at], small[1])
    # dweight = sum x^2 r is the sum over rows of x^2 over their rms: near the number of rows, all alike
    assert float((dw / ROWS - dw.mean() / ROWS).abs().max()) < 0.01 and abs(float(dw.mean()) / ROWS - 1) < 0.01


def test_gated_of_many_rows():
    F, K = 4104, 8
    x = torch.empty((ROWS, K), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn((2 * F, K), device="cuda").bfloat16()
    at = sample()
    h = fq.gated_linear(x, w)
    assert torch.equal(h[at], fq.gated_linear(x[at], w))
    dx, dw = fq.gated_linear_backward(h, x, w)
    gu = x[at].double() @ w.double().t()
    a, u = gu[:, :F], gu[:, F:]
    s = torch.sigmoid(a)
    dh = h[at].double()
    ref = torch.cat([dh * u * s * (1 + a * (1 - s)), dh * a * s], -1) @ w.double()
    assert float((dx[at].double() - ref).norm() / ref.norm()) < 2.0 ** -7
    # dw of the last hidden channel, over all rows
    g, v = (x.double() @ w[[F - 1, 2 * F - 1]].double().t()).unbind(-1)
    du = h[:, F - 1].double() * g * torch.sigmoid(g)
    want = du @ x.double()
    assert float((dw[2 * F - 1].double() - want).norm() / want.norm()) < 2.0 ** -7


def test_adapters_past_32_bits():
    """Rows of y, and adapters, that lie past 2^32 bytes and elements."""
    N, K, r = 4104, 8, 8
    x = torch.empty((ROWS, K), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn((N, K), device="cuda").bfloat16()
    a, b = torch.randn((3, r, K), device="cuda").bfloat16(), torch.randn((3, N, r), device="cuda").bfloat16()
    ids = (torch.arange(ROWS, device="cuda") // 1000 % 4 - 1).to(torch.int32)
    at = sample()
    y = fq.adapter_linear(x, w, a, b, ids)
    ref = x[at].double() @ w.double().t()
    for k, e in enumerate(ids[at].tolist()):
        if e >= 0:
            ref[k] += x[at[k]].double() @ a[e].double().t() @ b[e].double().t()
    assert float((y[at].double() - ref).norm() / ref.norm()) < 2.0 ** -8
    ref = y[at].double()
    for k, e in enumerate(ids[at].tolist()):
        if e >= 0:
            ref[k] += x[at[k]].double() @ a[e].double().t() @ b[e].double().t()
    z = fq.adapter_add(y, x, a, b, ids, out=y)
    assert float((z[at].double() - ref).norm() / ref.norm()) < 2.0 ** -8
    del z, y, ref
    L, N, r = 1200, 7168, 256                          # b: 4.4 GB
    b = torch.empty((L, N, r), dtype=torch.bfloat16, device="cuda").normal_()
    a = torch.empty((L, r, 64), dtype=torch.bfloat16, device="cuda").normal_()
    for T in (3, 600):
        x = torch.randn((T, 64), device="cuda").bfloat16()
        ids = torch.full((T,), L - 1, device="cuda", dtype=torch.int32)
        y = fq.adapter_linear(x, torch.zeros((N, 64), device="cuda").bfloat16(), a, b, ids)
        ref = x.double() @ a[-1].double().t() @ b[-1].double().t()
        assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -8


# ---- refusals on GPU tensors ---------------------------------------------------------------

def test_refusals():
    def bf(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    def f32(*shape):
        return torch.zeros(shape, device="cuda")
    x, ids = bf(4, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    w64 = f32(64)
    for bad in (lambda: fq.rms_norm(bf(4, 64).t(), f32(4)), lambda: fq.rms_norm(x, f32(63)), lambda: fq.rms_norm(bf(4, 7), f32(7)),
                lambda: fq.rms_norm(x, w64, eps=-1.0), lambda: fq.rms_norm(x, w64, eps=float("nan")),
                lambda: fq.rms_norm(x, w64.cpu()), lambda: fq.rms_norm(bf(2, 16392), f32(16392)),
                lambda: fq.residual_norm(x, bf(5, 64)), lambda: fq.residual_norm(x, x, w64, gate=bf(4, 32)),
                lambda: fq.residual_norm_backward(x, None, x, x, w64), lambda: fq.residual_norm_backward(None, None, x, x),
                lambda: fq.residual_norm_backward(x, x, x, x), lambda: fq.gated_linear(x, bf(31, 64)),
                lambda: fq.gated_linear(x, bf(32, 56)), lambda: fq.gated_linear(bf(4, 60), bf(32, 60)),
                lambda: fq.gated_linear(x, bf(24, 64)), lambda: fq.gated_linear_backward(bf(4, 8), x, bf(32, 64)),
                lambda: fq.gated_linear_backward(bf(4, 16), x, bf(32, 64), bf(4, 16)),
                lambda: fq.gated_linear(bf(300)[1:257].view(4, 64), bf(32, 64)),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 12, 64), bf(2, 10, 12), ids),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 264, 64), bf(2, 10, 264), ids),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(3, 10, 8), ids),
                lambda: fq.adapter_linear(x, bf(11, 64), bf(2, 8, 64), bf(2, 10, 8), ids),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(2, 10, 8), ids[:3]),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(2, 10, 8), ids, f32(3)),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(2, 10, 8), ids, bias=f32(9)),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(2, 10, 8), ids, out=bf(4, 11)),
                lambda: fq.adapter_add(bf(4, 11), x, bf(2, 8, 64), bf(2, 10, 8), ids)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fq.rms_norm(x.half(), w64), lambda: fq.rms_norm(x, bf(64)), lambda: fq.residual_norm(x, f32(4, 64)),
                lambda: fq.residual_norm(x, x, w64, gate=bf(64).float().half()), lambda: fq.gated_linear(f32(4, 64), bf(32, 64)),
                lambda: fq.gated_linear(x, f32(32, 64)), lambda: fq.gated_linear(x, bf(32, 64), out_dtype=torch.float16),
                lambda: fq.adapter_linear(x, bf(10, 64), bf(2, 8, 64), bf(2, 10, 8), ids.long()),
                lambda: fq.adapter_linear(x, None, bf(2, 8, 64), bf(2, 10, 8), ids),
                lambda: fq.adapter_add(bf(4, 10).half(), x, bf(2, 8, 64), bf(2, 10, 8), ids)):
        with pytest.raises(TypeError):
            bad()
