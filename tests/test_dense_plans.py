"""Which kernels the dense block's products choose (host only): every choice within the documented sizes, as far as
their operands fit a GPU's memory, is one that a grid holds, and every kind of choice is one that a GPU test runs."""
import ctypes
import itertools
import math
import random

import test_gpu_block
import test_gpu_dense_limits
import test_gpu_dense_shapes
from fp8_act_quant_amd import _lib as L

MEMORY = 288 << 30
GRID = 2 ** 32 - 1           # threads


def plan(call, M, N, K, rank=8):
    out = (ctypes.c_int64 * 12)()
    assert L.lib.fp8q_dense_plan(call, M, N, K, rank, out) == L.FP8Q_OK
    return tuple(out[:6]), tuple(out[6:])


def tiles(M, N, launch):
    return -(-M // launch[0]) * -(-N // launch[1])


def sizes(least, most, step=8):
    """Numbers over a whole range, on both sides of its powers of two."""
    n = least
    while n < most:
        yield from (v for v in (n - step, n, n + step) if least <= v <= most)
        n *= 2
    yield most


def test_gated_plans_fit_a_grid():
    seen = 0
    for M, F, K in itertools.product(sizes(1, 1 << 26, 1), sizes(8, (1 << 22) - 8), sizes(8, (1 << 23) - 8)):
        held = 2 * M * K + 4 * F * K + 2 * M * F
        if held > MEMORY:
            continue
        r, _ = plan(L.FP8Q_PLAN_GATED, M, F, K)
        wanted = -(-M // r[0]) * -(-F // (r[1] // 2))
        assert wanted <= r[4] <= wanted + 144 and r[4] * r[5] <= GRID, (M, F, K, r)
        if held + 2 * M * K + 4 * F * K + 4 * M * F > MEMORY:      # dx, dw and dg, du beside them
            continue
        seen += 1
        for call, pieces, need in ((L.FP8Q_PLAN_GATED_BACKWARD, 1, L.lib.gated_linear_backward_workspace_bytes(M, F, K)),
                                   (L.FP8Q_PLAN_GATED_BACKWARD_WIDE, 2, L.lib.gated_linear_backward_wide_workspace_bytes(M, F, K))):
            if pieces == 2 and held + 10 * M * K + 20 * F * K + 8 * M * F > MEMORY:   # (and both pieces' sums)
                continue
            w, x = plan(call, M, F, K)
            n = [pieces * tiles(2 * F, K, w) * w[2], pieces * tiles(M, K, x) * x[2]]
            assert w[3] == x[3] and (not w[3] or w[4:] == x[4:])
            for mine, r in zip(n if not w[3] else [sum(n)], (w, x)):
                assert mine <= r[4] <= 2 * mine + 144 and r[4] * r[5] <= GRID, (call, M, F, K, r)
            # and the call itself has nothing against the size
            assert need >= 4 * M * F * pieces
            assert L.lib.gated_linear_backward(65536, 65536, 65536, None, L.FP8Q_GATED_WIDE * (pieces - 1), 65536, 1, 65536,
                                               1, M, F, K, 65536, need - 1, None) == L.FP8Q_ERR_WORKSPACE
    assert seen > 5000


def test_gradients_past_a_grid_are_refused():
    """dw alone would be 2^29 tiles."""
    F = K = (1 << 22) - 8
    assert L.lib.gated_linear_backward_workspace_bytes(8, F, K) == 0
    assert L.lib.gated_linear_backward(65536, 65536, 65536, None, 0, 65536, 1, 65536, 1, 8, F, K, 65536, 1 << 60,
                                       None) == L.FP8Q_ERR_SHAPE
    assert plan(L.FP8Q_PLAN_GATED_BACKWARD, 8, F, K)[0][4] == -1


def test_adapter_plans_fit_a_grid():
    """y, x and W or base within memory, and u, of adapters of the least and the most ranks."""
    seen = 0
    for M, N, K in itertools.product(sizes(1, 1 << 26, 1), sizes(1, 1 << 28, 1), sizes(8, (1 << 23) - 8)):
        if 2 * M * K + 2 * M * N + 2 * N * K > MEMORY:
            continue
        for rank in (8, 256):
            if 4 * M * rank + 2 * rank * (K + N) > MEMORY:
                continue
            seen += 1
            for call in (L.FP8Q_PLAN_ADAPTER, L.FP8Q_PLAN_ADAPTER_ADD):
                r, u = plan(call, M, N, K, rank)
                assert tiles(M, N, r) <= r[4] <= tiles(M, N, r) + 144 and r[4] * r[5] <= GRID, (call, M, N, K, rank, r)
                assert 0 < u[4] * u[5] <= GRID and u[1] * u[2] >= 16, (M, N, K, rank, u)
    assert seen > 5000


def test_wide_flag_is_the_gradients():
    def back(act):
        return L.lib.gated_linear_backward(65536, 65536, 65536, None, act, 65536, 1, 65536, 1, 4, 16, 64, None, 0, None)
    assert back(L.FP8Q_GATED_WIDE) == back(L.FP8Q_GATED_WIDE | L.FP8Q_ACT_GELU) == L.FP8Q_ERR_WORKSPACE
    for act in (L.FP8Q_GATED_WIDE | 2, L.FP8Q_GATED_WIDE * 2, L.FP8Q_GATED_WIDE * 3, -L.FP8Q_GATED_WIDE, -1):
        assert back(act) == L.FP8Q_ERR_DTYPE, act
    assert L.lib.gated_linear(65536, 65536, 65536, 1, None, L.FP8Q_GATED_WIDE, 4, 16, 64, None) == L.FP8Q_ERR_DTYPE
    assert L.lib.gated_linear_backward_wide_workspace_bytes(4, 12, 64) == 0


def test_plan_arguments():
    out = (ctypes.c_int64 * 12)()
    for args, status in (((5, 8, 8, 8, 8, out), L.FP8Q_ERR_DTYPE), ((-1, 8, 8, 8, 8, out), L.FP8Q_ERR_DTYPE),
                         ((0, 0, 8, 8, 8, out), L.FP8Q_ERR_SHAPE), ((0, 8, 12, 8, 8, out), L.FP8Q_ERR_SHAPE),
                         ((1, 8, 8, 12, 8, out), L.FP8Q_ERR_SHAPE), ((2, 8, 0, 8, 8, out), L.FP8Q_ERR_SHAPE),
                         ((3, 8, 8, 8, 12, out), L.FP8Q_ERR_SHAPE), ((0, 8, 8, 8, 8, None), L.FP8Q_ERR_NULL)):
        assert L.lib.fp8q_dense_plan(*args) == status, args
    assert list(out) == [0] * 12


def kinds(call, M, N, K, rank=8):
    """What kinds of launches a call makes: tiles, marks, and whether K is in parts."""
    a, b = plan(call, M, N, K, rank)
    if call == L.FP8Q_PLAN_GATED:
        return {(call, *a[:2])}
    if call in (L.FP8Q_PLAN_ADAPTER, L.FP8Q_PLAN_ADAPTER_ADD):
        return {(call, *a[:2], a[3]), ("u", *b[:2], b[3], b[2] > 1)}
    if a[3]:
        return {(call, "joint", *a[:2], a[2] > 1, b[2] > 1)}
    return {(call, "dw", *a[:2], a[2] > 1), (call, "dx", *b[:2], b[2] > 1)}


def test_every_kind_of_launch_is_tested():
    """Sizes drawn over the whole range, beside the shapes that the GPU tests run."""
    tested = set()
    for M, F, K in test_gpu_block.GATED + test_gpu_dense_shapes.PROJECTIONS:
        tested |= kinds(L.FP8Q_PLAN_GATED, M, F, K) | kinds(L.FP8Q_PLAN_GATED_BACKWARD, M, F, K)
    for M, F, K in test_gpu_dense_limits.WIDE + test_gpu_dense_shapes.PROJECTIONS:
        tested |= kinds(L.FP8Q_PLAN_GATED_BACKWARD_WIDE, M, F, K)
    for M, N, K, _, r, *_ in test_gpu_block.ADAPTERS + test_gpu_dense_shapes.ADAPTERS:
        tested |= kinds(L.FP8Q_PLAN_ADAPTER, M, N, K, r) | kinds(L.FP8Q_PLAN_ADAPTER_ADD, M, N, K, r)
    rng = random.Random(1)

    def log(least, most):
        return int(round(math.exp(rng.uniform(math.log(least), math.log(most + 0.49)))))
    met = set()
    for _ in range(20000):
        M, N, K, r = log(1, 16384), 8 * log(1, 2304), 8 * log(1, 896), 8 * log(1, 32)
        for call in (L.FP8Q_PLAN_GATED, L.FP8Q_PLAN_GATED_BACKWARD, L.FP8Q_PLAN_GATED_BACKWARD_WIDE):
            met |= kinds(call, M, N, K)
        N = log(1, 18432)
        for call in (L.FP8Q_PLAN_ADAPTER, L.FP8Q_PLAN_ADAPTER_ADD):
            met |= kinds(call, M, N, K, r)
    assert len(met) > 70 and not met - tested, met - tested
