"""Host-side validation of the routed-expert and 8-bit integer entry points (no GPU needed):
every call below is refused, or is an empty call, before a device is touched."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from fp8_act_quant_amd import _lib
    return _lib


def route(L, logits=FAKE, dtype=0, bias=None, w=FAKE, e=FAKE, T=4, E=16, k=2, groups=1, kept=1, flags=0):
    return L.lib.moe_route(logits, dtype, bias, w, e, T, E, k, groups, kept, 1.0, flags, None)


def test_route_validation(L):
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64), dict(k=17), dict(groups=3),
                dict(groups=0), dict(groups=128, E=256), dict(groups=4, kept=5), dict(groups=4, kept=0),
                dict(groups=4, kept=1, k=5), dict(T=1 << 24)):
        assert route(L, **bad) == L.FP8Q_ERR_SHAPE, bad
    assert route(L, dtype=2) == L.FP8Q_ERR_DTYPE
    assert route(L, flags=8) == L.FP8Q_ERR_DTYPE
    for bad in (dict(logits=None), dict(w=None), dict(e=None)):
        assert route(L, **bad) == L.FP8Q_ERR_NULL
    for bad in (dict(logits=FAKE + 2), dict(bias=FAKE + 1), dict(w=FAKE + 2), dict(e=FAKE + 2),
                dict(logits=FAKE + 1, dtype=1)):
        assert route(L, **bad) == L.FP8Q_ERR_ALIGN
    assert route(L, logits=None, w=None, e=None, T=0) == L.FP8Q_OK


def test_route_backward_validation(L):
    def call(dw=FAKE, x=FAKE, dtype=0, e=FAKE, dx=FAKE, T=4, E=16, k=2, flags=0):
        return L.lib.moe_route_backward(dw, x, dtype, e, dx, T, E, k, 1.0, flags, None)
    for bad in (dict(T=-1), dict(E=1025), dict(k=0), dict(k=33), dict(T=1 << 24)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE
    assert call(dtype=3) == L.FP8Q_ERR_DTYPE
    assert call(flags=L.FP8Q_MOE_GROUP_MAX) == L.FP8Q_ERR_DTYPE
    for bad in (dict(dw=None), dict(x=None), dict(e=None), dict(dx=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL
    assert call(dx=FAKE + 2) == L.FP8Q_ERR_ALIGN
    assert call(T=0, x=None) == L.FP8Q_OK


def test_place_validation(L):
    def call(a=FAKE, off=FAKE, rows=FAKE, slots=FAKE, T=4, k=2, n=8, first=0, ws=None, size=0):
        return L.lib.moe_place(a, off, rows, slots, T, k, n, first, ws, size, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(n=0), dict(n=1025), dict(first=-1), dict(first=2 ** 31),
                dict(T=1 << 23, k=32, n=1 << 20)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE
    for bad in (dict(a=None), dict(off=None), dict(rows=None), dict(slots=None), dict(T=0, off=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL
    for bad in (dict(off=FAKE + 4), dict(rows=FAKE + 2), dict(ws=FAKE + 2, size=1 << 20)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN
    need = L.lib.moe_place_workspace_bytes(16384, 8, 256)
    assert need > 0 and L.lib.moe_place_workspace_bytes(8, 8, 256) == 0
    assert L.lib.moe_place_workspace_bytes(-1, 8, 256) == L.lib.moe_place_workspace_bytes(16384, 0, 256) == 0
    assert call(T=16384, k=8, n=256) == L.FP8Q_ERR_WORKSPACE
    assert call(T=16384, k=8, n=256, ws=FAKE, size=need - 1) == L.FP8Q_ERR_WORKSPACE


def test_combine_validation(L):
    def call(h=FAKE, dtype=1, slots=FAKE, w=FAKE, y=FAKE, T=4, k=2, rows=8, H=64):
        return L.lib.moe_combine(h, dtype, slots, w, y, T, k, rows, H, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(rows=-1), dict(rows=2 ** 31), dict(H=-1), dict(H=1 << 25),
                dict(T=1 << 24)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE
    assert call(dtype=2) == L.FP8Q_ERR_DTYPE
    for bad in (dict(h=None), dict(slots=None), dict(y=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL
    for bad in (dict(h=FAKE + 1), dict(y=FAKE + 2, dtype=0), dict(slots=FAKE + 2), dict(w=FAKE + 2)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN
    assert call(T=0, y=None) == call(H=0, y=None) == L.FP8Q_OK

    def back(dy=FAKE, h=FAKE, dtype=1, slots=FAKE, w=FAKE, dh=FAKE, dw=FAKE, T=4, k=2, rows=8, H=64):
        return L.lib.moe_combine_backward(dy, h, dtype, slots, w, dh, dw, T, k, rows, H, None)
    for bad in (dict(T=-1), dict(k=33), dict(H=-1)):
        assert back(**bad) == L.FP8Q_ERR_SHAPE
    for bad in (dict(dy=None), dict(h=None), dict(w=None), dict(dh=None), dict(dw=None)):
        assert back(**bad) == L.FP8Q_ERR_NULL
    assert back(dw=FAKE + 2) == back(dh=FAKE + 1) == L.FP8Q_ERR_ALIGN
    assert back(T=0, dy=None) == L.FP8Q_OK


def test_int8_validation(L):
    lib = L.lib
    assert lib.int8_quant(FAKE, FAKE, FAKE, 4, 24, None) == L.FP8Q_ERR_SHAPE
    assert lib.int8_quant(FAKE, FAKE, FAKE, -1, 16, None) == L.FP8Q_ERR_SHAPE
    assert lib.int8_quant(None, FAKE, FAKE, 4, 16, None) == L.FP8Q_ERR_NULL
    assert lib.int8_quant(FAKE + 8, FAKE, FAKE, 4, 16, None) == L.FP8Q_ERR_ALIGN
    assert lib.int8_quant(None, None, None, 0, 16, None) == lib.int8_quant(None, None, None, 4, 0, None) == L.FP8Q_OK

    def gemm(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, bias=None, y=FAKE, dtype=0, M=4, N=8, K=32):
        return lib.int8_gemm(a, sa, w, sw, bias, y, dtype, M, N, K, None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-16), dict(K=24), dict(K=1 << 17), dict(M=1 << 37)):
        assert gemm(**bad) == L.FP8Q_ERR_SHAPE, bad
    assert gemm(dtype=2) == L.FP8Q_ERR_DTYPE
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None)):
        assert gemm(**bad) == L.FP8Q_ERR_NULL
    for bad in (dict(a=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 2), dict(sa=FAKE + 2), dict(bias=FAKE + 2)):
        assert gemm(**bad) == L.FP8Q_ERR_ALIGN
    assert gemm(M=0, a=None, y=None) == gemm(N=0, w=None) == L.FP8Q_OK

    def linear(x=FAKE, w=FAKE, sw=FAKE, bias=None, y=FAKE, dtype=1, M=100, N=8, K=32, ws=FAKE, size=1 << 20):
        return lib.int8_linear(x, w, sw, bias, y, dtype, M, N, K, ws, size, None)
    for bad in (dict(M=-1), dict(K=24), dict(M=1 << 24)):
        assert linear(**bad) == L.FP8Q_ERR_SHAPE
    assert linear(x=None) == linear(sw=None) == linear(y=None) == L.FP8Q_ERR_NULL
    assert linear(x=FAKE + 8) == linear(ws=FAKE + 8) == L.FP8Q_ERR_ALIGN
    need = lib.int8_linear_workspace_bytes(100, 8, 32)
    assert need >= 100 * 36 and lib.int8_linear_workspace_bytes(1, 8, 32) == 0
    assert lib.int8_linear_workspace_bytes(0, 8, 32) == lib.int8_linear_workspace_bytes(100, 8, 31) == 0
    assert linear(ws=None) == linear(size=need - 1) == L.FP8Q_ERR_WORKSPACE
    assert linear(M=0, x=None, ws=None) == L.FP8Q_OK

    def grouped(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, off=FAKE, rows=None, y=FAKE, dtype=0, E=2, M=4, tokens=4, N=8, K=32):
        return lib.int8_grouped_gemm(a, sa, w, sw, off, rows, y, dtype, E, M, tokens, N, K, None)
    for bad in (dict(E=0), dict(E=1025), dict(tokens=3), dict(tokens=-1, rows=FAKE), dict(K=8), dict(M=1 << 31),
                dict(rows=FAKE, tokens=1 << 20, K=8192)):
        assert grouped(**bad) == L.FP8Q_ERR_SHAPE, bad
    for bad in (dict(a=None), dict(off=None), dict(w=None), dict(y=None)):
        assert grouped(**bad) == L.FP8Q_ERR_NULL
    for bad in (dict(off=FAKE + 4), dict(rows=FAKE + 2), dict(w=FAKE + 8)):
        assert grouped(**bad) == L.FP8Q_ERR_ALIGN
    assert grouped(M=0, tokens=7) == L.FP8Q_OK


def test_linear_layers_wider_than_one_launch(L):
    """One or two rows of more channels than the one-launch kernel's grid holds take two launches, for which
    they need a workspace (and are refused without one)."""
    lib = L.lib
    most = (2 ** 32 - 1) // 256 * 32
    for M in (1, 2):
        assert lib.int8_linear_workspace_bytes(M, most, 2064) == 0
        assert lib.int8_linear_workspace_bytes(M, most + 1, 2064) >= M * 2068
        assert lib.int8_linear(FAKE, FAKE, FAKE, None, FAKE, 0, M, most + 1, 2064, None, 0, None) == L.FP8Q_ERR_WORKSPACE


def test_package_without_the_native_binding():
    """Where the binding cannot be loaded the calls that need it say so, and the others are there."""
    code = """
import sys
sys.modules["fp8_act_quant_amd._native"] = None      # its import fails
import fp8_act_quant_amd as fq
from fp8_act_quant_amd import *
assert callable(act_quant) and callable(fq.fp8_gemm) and fq.lib.fp8q_version() >> 16 == 1
for name in ("moe_route", "moe_route_backward", "moe_place", "moe_combine", "moe_combine_backward", "int8_quant",
             "int8_gemm", "int8_linear", "int8_grouped_gemm"):
    assert getattr(fq, name).__name__ == name
    try:
        getattr(fq, name)(None, 1)
    except ImportError as e:
        assert name in str(e) and "native binding" in str(e)
    else:
        raise SystemExit(name)
print("fine")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.stdout == "fine\n", out.stderr


def test_package_with_the_native_binding():
    import fp8_act_quant_amd as fq
    from fp8_act_quant_amd import int8, moe
    assert fq.moe_route is moe.moe_route and fq.int8_linear is int8.int8_linear
