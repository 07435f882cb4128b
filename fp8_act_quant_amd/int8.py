"""Products in 8-bit integers with one scale per token and one per output channel.

``int8_quant`` quantises rows (an activation's tokens, or a weight's channels), ``int8_gemm``
multiplies, ``int8_linear`` does both for bf16 activations and ``int8_grouped_gemm`` multiplies
every expert's rows by its own weight. The integer sums are exact. Arguments are marshalled
only; every step runs in the kernels behind the C ABI.
"""
from __future__ import annotations

import math

import torch

from ._lib import lib
from ._tensor import CODE, launch, need

STEP = 16            # K is a multiple of this
MAX_K = 1 << 17      # and below this, so that 32-bit sums are exact


def _depth(K: int) -> None:
    if K % STEP or K >= MAX_K:
        raise ValueError(f"the last dimension must be a multiple of {STEP} below {MAX_K}")


def _out(out, shape, out_dtype, a) -> torch.Tensor:
    if out_dtype not in CODE:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    if out is None:
        return a.new_empty(shape, dtype=out_dtype)
    need(out, "out", out_dtype, shape, device=a.device)
    return out


def int8_quant(x: torch.Tensor):
    """One scale per row of a bf16 x [..., K] (K a multiple of 16): the tokens of an
    activation, or the output channels of a weight. Returns ``(q, s)``: q int8 [..., K] in
    -127 .. 127 and s float32 [...], s = max|x| * float32(1 / 127), q = x / s rounded to
    nearest even."""
    need(x, "x", torch.bfloat16, align=16)
    if x.dim() < 1 or x.shape[-1] % STEP:
        raise ValueError(f"the last dimension must be a multiple of {STEP}")
    q = torch.empty_like(x, dtype=torch.int8)
    K = x.shape[-1]
    # (rows of no elements have the scale of a zero row)
    s = (x.new_empty if K else x.new_zeros)(x.shape[:-1], dtype=torch.float32)
    launch("int8_quant", lib.int8_quant, x, x.data_ptr(), q.data_ptr(), s.data_ptr(), math.prod(x.shape[:-1]), K)
    return q, s


def int8_gemm(a: torch.Tensor, a_s: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor,
              bias: torch.Tensor | None = None, out_dtype=torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (a . w^T) * a_s * w_s (+ bias). a int8 [..., K] with scales a_s float32 [...], w int8
    [N, K] with w_s float32 [N] (K a multiple of 16 below 2^17), bias: optional float32 [N],
    added before the output's rounding. Returns [..., N] in out_dtype (bfloat16 or float32)."""
    need(a, "a", torch.int8, align=16)
    need(w, "w", torch.int8, align=16, device=a.device)
    if a.dim() < 1 or w.dim() != 2 or w.shape[1] != a.shape[-1]:
        raise ValueError("w must be [N, K] with the activation's K")
    N, K = w.shape
    _depth(K)
    need(a_s, "a_s", torch.float32, a.shape[:-1], device=a.device)
    need(w_s, "w_s", torch.float32, (N,), device=a.device)
    b_ptr = None
    if bias is not None:
        need(bias, "bias", torch.float32, (N,), device=a.device)
        b_ptr = bias.data_ptr()
    out = _out(out, (*a.shape[:-1], N), out_dtype, a)
    launch("int8_gemm", lib.int8_gemm, a, a.data_ptr(), a_s.data_ptr(), w.data_ptr(), w_s.data_ptr(), b_ptr,
           out.data_ptr(), CODE[out_dtype], math.prod(a.shape[:-1]), N, K)
    return out


def int8_linear(x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
                bias: torch.Tensor | None = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """y = x . weight^T (+ bias) for bf16 activations x [..., K] and an 8-bit weight [N, K] with
    one scale per channel [N] (as int8_quant gives them): int8_gemm of int8_quant(x), bit for
    bit, in one call (at most 4 tokens: in one launch)."""
    need(x, "x", torch.bfloat16, align=16)
    need(weight, "weight", torch.int8, align=16, device=x.device)
    if x.dim() < 1 or weight.dim() != 2 or weight.shape[1] != x.shape[-1]:
        raise ValueError("weight must be [N, K] with the activation's K")
    N, K = weight.shape
    _depth(K)
    need(weight_scale, "weight_scale", torch.float32, (N,), device=x.device)
    b_ptr = None
    if bias is not None:
        need(bias, "bias", torch.float32, (N,), device=x.device)
        b_ptr = bias.data_ptr()
    M = math.prod(x.shape[:-1])
    out = _out(None, (*x.shape[:-1], N), out_dtype, x)
    ws_bytes = lib.int8_linear_workspace_bytes(M, N, K)
    # from torch's allocator, which keeps it from calls on other streams until this one is done
    ws = x.new_empty(ws_bytes, dtype=torch.int8) if ws_bytes else None
    launch("int8_linear", lib.int8_linear, x, x.data_ptr(), weight.data_ptr(), weight_scale.data_ptr(), b_ptr,
           out.data_ptr(), CODE[out_dtype], M, N, K, ws.data_ptr() if ws_bytes else None, ws_bytes)
    return out


def int8_grouped_gemm(a: torch.Tensor, a_s: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor,
                      offsets: torch.Tensor, rows: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """Routed experts' products in one launch: row r, of the expert e with offsets[e] <= r <
    offsets[e + 1], is a[rows[r]] (or a[r] without rows) times w[e]. a int8 [tokens, K] with
    a_s float32 [tokens]; w int8 [E, N, K] with w_s float32 [E, N]; offsets int64 [E + 1] and
    rows int32 [R] as moe_place returns them, on the device. Returns [R, N] (R = tokens
    without rows) in out_dtype; rows that no expert owns are left as they were in `out`, or
    uninitialised."""
    need(a, "a", torch.int8, align=16)
    need(w, "w", torch.int8, align=16, device=a.device)
    if a.dim() != 2 or w.dim() != 3 or w.shape[2] != a.shape[1]:
        raise ValueError("a must be [tokens, K] and w [E, N, K]")
    tokens, K = a.shape
    E, N = w.shape[:2]
    _depth(K)
    need(a_s, "a_s", torch.float32, (tokens,), device=a.device)
    need(w_s, "w_s", torch.float32, (E, N), device=a.device)
    need(offsets, "offsets", torch.int64, (E + 1,), align=8, device=a.device)
    R, r_ptr = tokens, None
    if rows is not None:
        need(rows, "rows", torch.int32, device=a.device)
        if rows.dim() != 1:
            raise ValueError("rows must be [R]")
        R, r_ptr = rows.shape[0], rows.data_ptr()
    out = _out(out, (R, N), out_dtype, a)
    launch("int8_grouped_gemm", lib.int8_grouped_gemm, a, a.data_ptr(), a_s.data_ptr(), w.data_ptr(), w_s.data_ptr(),
           offsets.data_ptr(), r_ptr, out.data_ptr(), CODE[out_dtype], E, R, tokens, N, K)
    return out
