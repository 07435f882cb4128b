"""The dense block's products at one shape at least for every kind of launch that their cost models choose (which
test_dense_plans.py checks), against 64 bits with the bounds of test_gpu_block.py and test_gpu_dense_limits.py.
"""
import pytest
import torch

import fp8_act_quant_amd as fq
from test_gpu_block import DT, adapter_inputs, adapters64
from test_gpu_dense_limits import ACT, U, act64, half, near, product64, product_of, randn, rng, slopes64

pytestmark = pytest.mark.gpu

# (tokens, hidden, channels); by the gradient's launches: each product its own tiles or both one launch, K whole or in parts
PROJECTIONS = [(465, 616, 24), (660, 296, 168), (982, 1224, 224), (3259, 344, 176), (4171, 232, 336), (4167, 1064, 240),
               (5233, 2640, 232), (5676, 5392, 224), (998, 13912, 176), (2188, 416, 1520), (1247, 664, 2200), (759, 1168, 1600),
               (2909, 456, 976), (973, 3352, 912), (2935, 408, 2160), (5351, 24, 3624), (5943, 24, 5312), (10, 2040, 6896),
               (1, 12616, 1192), (323, 168, 3760), (749, 344, 6048)]
# one and nine tokens of a layer whose rows of W are many and long, whose stages' loop runs on
STEPS = [(1, 18432, 7168), (9, 10248, 4104), (16, 2056, 7176)]
# (rows, channels out, channels in, adapters, rank)
ADAPTERS = [(29, 8341, 520, 5, 40), (47, 8999, 1032, 11, 24), (63, 7247, 368, 9, 16), (98, 2956, 2848, 20, 16),
            (729, 1356, 2056, 33, 8), (2052, 1758, 568, 7, 16),
            (2305, 7408, 1032, 2, 64), (4099, 4609, 264, 40, 24)]


def check_forward(x, w, act, dtype):
    h, gu = fq.gated_linear(x, w, act=act, keep=True, out_dtype=dtype)
    ref, off = product64(x, w)
    near(gu, ref, off, "gu")
    F = w.shape[0] // 2
    (p, _, _), b, off_a, off_b = act64(ref[:, :F], act), ref[:, F:], off[:, :F], off[:, F:]
    near(h, p * b, 1.13 * off_a * b.abs() + (p.abs() + 1.13 * off_a) * off_b + ACT * U * (p * b).abs(), act)
    return gu


@pytest.mark.parametrize("M,F,K", PROJECTIONS)
def test_projections(M, F, K):
    g = rng(M + F + K)
    x, w, dh = randn(g, M, K), randn(g, 2 * F, K, std=1.5 * K ** -0.5), randn(g, M, F)
    gu = check_forward(x, w, "silu", torch.bfloat16)
    check_forward(x, w, "gelu", torch.float32)
    for act, kept, dtype, wide in (("silu", True, torch.bfloat16, False), ("gelu", False, torch.float32, False),
                                   ("gelu", True, torch.float32, True)):
        at = (gu.double(), torch.zeros_like(gu, dtype=torch.float64)) if kept else product64(x, w)
        d, off = slopes64(dh, *at, act, half(torch.bfloat16) ** (2 if wide else 1))
        got = fq.gated_linear_backward(dh, x, w, gu if kept else None, act, dx_dtype=dtype, dw_dtype=dtype, wide=wide)
        more = 1 + 2 * half(torch.bfloat16) * wide
        for name, y, (ref, slack) in zip(("dx", "dw"), got, (product_of(d, off, w, 2 * F), product_of(d.t(), off.t(), x, M))):
            near(y, ref, slack * more, (name, act, kept, wide))


@pytest.mark.parametrize("M,F,K", STEPS)
def test_steps_of_wide_layers(M, F, K):
    g = rng(M + F + K)
    x, w = randn(g, M, K), randn(g, 2 * F, K, std=K ** -0.5)
    for dtype in (torch.bfloat16, torch.float32):
        check_forward(x, w, "silu", dtype)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("M,N,K,L,r", ADAPTERS)
def test_adapters(M, N, K, L, r, order, out):
    s = adapter_inputs(M, N, K, L, r, order, M + N + K)
    ref, off = adapters64(**s, base=None)
    near(fq.adapter_linear(**s, out_dtype=DT[out]), ref, off, "linear")
    s["w"] = s["bias"] = None
    base = randn(rng(M), M, N, dtype=DT[out])
    ref, off = adapters64(**s, base=base)
    near(fq.adapter_add(base, *(s[k] for k in ("x", "a", "b", "ids", "scales"))), ref, off, "add")
