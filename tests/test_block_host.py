"""Host-side validation of the dense block's entry points (no GPU needed): every call below is refused, or
is an empty call, before a device is touched."""
import inspect
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


def test_norm_validation(L):
    def call(x=FAKE, y=FAKE, dtype=1, weight=FAKE, post=FAKE, gate=FAKE, flags=0, t=FAKE, z=FAKE, T=4, H=64):
        return L.lib.residual_norm(x, y, dtype, weight, post, gate, flags, 1.0, 1e-6, t, z, T, H, None)
    for bad in (dict(T=-1), dict(H=7), dict(H=0), dict(H=-8), dict(H=16385), dict(T=1 << 45)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE, bad
    for bad in (dict(dtype=2), dict(dtype=-1), dict(flags=2), dict(flags=-1)):
        assert call(**bad) == L.FP8Q_ERR_DTYPE, bad
    for bad in (dict(x=None), dict(z=None), dict(weight=None, t=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL, bad
    for bad in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(t=FAKE + 1), dict(z=FAKE + 1), dict(weight=FAKE + 2),
                dict(post=FAKE + 2), dict(gate=FAKE + 2), dict(gate=FAKE + 1, flags=1), dict(x=FAKE + 2, dtype=0),
                dict(gate=FAKE + 2, flags=1, dtype=0)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN, bad
    assert call(T=0, x=None, t=None, z=None) == L.FP8Q_OK


def test_norm_backward_validation(L):
    lib = L.lib

    def call(dt=FAKE, dz=FAKE, t=FAKE, y=FAKE, dtype=1, weight=FAKE, post=FAKE, gate=FAKE, flags=0, dx=FAKE, dy=FAKE,
             dweight=FAKE, dpost=FAKE, dgate=FAKE, T=400, H=64, ws=FAKE, size=1 << 30):
        return lib.residual_norm_backward(dt, dz, t, y, dtype, weight, post, gate, flags, 1.0, 1e-6, dx, dy, dweight,
                                          dpost, dgate, T, H, ws, size, None)
    for bad in (dict(T=-1), dict(H=7), dict(H=16385), dict(T=1 << 45)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE, bad
    for bad in (dict(dtype=2), dict(flags=4)):
        assert call(**bad) == L.FP8Q_ERR_DTYPE, bad
    for bad in (dict(dz=None), dict(t=None), dict(dx=None), dict(dy=None), dict(dweight=None), dict(dpost=None),
                dict(dgate=None), dict(dgate=None, flags=1), dict(dt=None, weight=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL, bad
    for bad in (dict(dt=FAKE + 1), dict(dz=FAKE + 1), dict(t=FAKE + 1), dict(y=FAKE + 1), dict(dx=FAKE + 1),
                dict(dy=FAKE + 1), dict(dweight=FAKE + 2), dict(dpost=FAKE + 2), dict(dgate=FAKE + 2),
                dict(dgate=FAKE + 1, flags=1), dict(weight=FAKE + 2), dict(post=FAKE + 2), dict(gate=FAKE + 2),
                dict(ws=FAKE + 8)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN, bad
    need = lib.residual_norm_backward_workspace_bytes(400, 64)
    assert need > 0 and need % (3 * 64 * 4) == 0 and lib.residual_norm_backward_workspace_bytes(1, 64) == 0
    assert lib.residual_norm_backward_workspace_bytes(400, 7) == lib.residual_norm_backward_workspace_bytes(-1, 64) == 0
    assert call(size=need - 1) == call(ws=None) == L.FP8Q_ERR_WORKSPACE
    # as many partial rows at the most as there is sense in
    assert lib.residual_norm_backward_workspace_bytes(1 << 30, 7168) <= 1024 * 3 * 7168 * 4


def test_gated_validation(L):
    lib = L.lib

    def call(x=FAKE, w=FAKE, h=FAKE, dtype=1, gu=None, act=0, M=4, F=16, K=64):
        return lib.gated_linear(x, w, h, dtype, gu, act, M, F, K, None)
    for bad in (dict(M=-1), dict(F=-8), dict(K=-8), dict(F=12), dict(K=60), dict(K=1 << 23), dict(F=1 << 22),
                dict(M=(1 << 26) + 1)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE, bad
    for bad in (dict(dtype=2), dict(act=2), dict(act=-1)):
        assert call(**bad) == L.FP8Q_ERR_DTYPE, bad
    for bad in (dict(x=None), dict(w=None), dict(h=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL, bad
    for bad in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(h=FAKE + 2), dict(gu=FAKE + 2)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN, bad
    assert call(M=0, x=None, h=None) == call(F=0, w=None, h=None) == L.FP8Q_OK

    def back(dh=FAKE, x=FAKE, w=FAKE, gu=FAKE, act=0, dx=FAKE, dxt=1, dw=FAKE, dwt=0, M=4, F=16, K=64, ws=FAKE, size=1 << 20):
        return lib.gated_linear_backward(dh, x, w, gu, act, dx, dxt, dw, dwt, M, F, K, ws, size, None)
    for bad in (dict(M=-1), dict(F=12), dict(K=60), dict(K=1 << 23), dict(F=1 << 22), dict(M=(1 << 26) + 1)):
        assert back(**bad) == L.FP8Q_ERR_SHAPE, bad
    for bad in (dict(dxt=2), dict(dwt=2), dict(act=7)):
        assert back(**bad) == L.FP8Q_ERR_DTYPE, bad
    for bad in (dict(dh=None), dict(x=None), dict(w=None)):
        assert back(**bad) == L.FP8Q_ERR_NULL, bad
    for bad in (dict(dh=FAKE + 8), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(gu=FAKE + 8), dict(dx=FAKE + 2),
                dict(dw=FAKE + 2), dict(ws=FAKE + 8)):
        assert back(**bad) == L.FP8Q_ERR_ALIGN, bad
    need = lib.gated_linear_backward_workspace_bytes(4, 16, 64)
    assert need >= 4 * 2 * 16 * 2
    for bad in ((4, 12, 64), (4, 16, 60), (-1, 16, 64)):
        assert lib.gated_linear_backward_workspace_bytes(*bad) == 0
    assert back(size=need - 1) == back(ws=None) == L.FP8Q_ERR_WORKSPACE
    assert back(dx=None, dw=None) == back(K=0) == L.FP8Q_OK


def test_adapter_validation(L):
    lib = L.lib

    def call(x=FAKE, w=FAKE, bias=None, a=FAKE, b=FAKE, scales=None, ids=FAKE, base=None, y=FAKE, dtype=1, M=4, N=10, K=64,
             adapters=3, rank=16, ws=FAKE, size=1 << 20):
        return lib.adapter_linear(x, w, bias, a, b, scales, ids, base, y, dtype, M, N, K, adapters, rank, ws, size, None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-8), dict(K=60), dict(K=1 << 23), dict(adapters=-1), dict(adapters=1 << 31),
                dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=264), dict(M=(1 << 26) + 1), dict(N=(1 << 28) + 1)):
        assert call(**bad) == L.FP8Q_ERR_SHAPE, bad
    assert call(dtype=2) == L.FP8Q_ERR_DTYPE
    for bad in (dict(x=None), dict(w=None), dict(a=None), dict(b=None), dict(ids=None), dict(y=None)):
        assert call(**bad) == L.FP8Q_ERR_NULL, bad
    for bad in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(a=FAKE + 8), dict(b=FAKE + 8), dict(bias=FAKE + 2),
                dict(scales=FAKE + 2), dict(ids=FAKE + 2), dict(w=None, base=FAKE + 2), dict(y=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(**bad) == L.FP8Q_ERR_ALIGN, bad
    need = lib.adapter_linear_workspace_bytes(4, 64, 16)
    assert need >= 4 * 16 * 4
    for bad in ((4, 64, 12), (-1, 64, 8), (4, 60, 8)):
        assert lib.adapter_linear_workspace_bytes(*bad) == 0
    assert call(size=need - 1) == call(ws=None) == L.FP8Q_ERR_WORKSPACE
    assert call(M=0, x=None, ids=None, y=None) == call(N=0, w=None, y=None) == L.FP8Q_OK


def test_python_arguments():
    """What is refused before a tensor is looked at, and names and defaults as documented."""
    import fp8_act_quant_amd as fq
    from fp8_act_quant_amd import block
    for name in ("rms_norm", "rms_norm_backward", "residual_norm", "residual_norm_backward", "gated_linear",
                 "gated_linear_backward", "adapter_linear", "adapter_add"):
        assert getattr(fq, name) is getattr(block, name) and name in fq.__all__
        assert getattr(fq, name).__doc__
    with pytest.raises(ValueError):
        fq.gated_linear(None, None, act="relu")
    with pytest.raises(TypeError):
        fq.gated_linear(None, None)
    with pytest.raises(TypeError):
        fq.gated_linear(None, None, out_dtype=int)
    with pytest.raises(TypeError):
        fq.adapter_linear(None, None, None, None, None)
    with pytest.raises(TypeError):
        fq.residual_norm(None, None)
    assert inspect.signature(fq.rms_norm).parameters["eps"].default == 1e-6


def test_package_without_the_native_binding():
    code = """
import sys
sys.modules["fp8_act_quant_amd._native"] = None      # its import fails
import fp8_act_quant_amd as fq
for name in ("rms_norm", "rms_norm_backward", "residual_norm", "residual_norm_backward", "gated_linear",
             "gated_linear_backward", "adapter_linear", "adapter_add"):
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
