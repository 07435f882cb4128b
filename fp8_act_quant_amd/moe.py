"""Routing of tokens to experts, and rows into expert order and back.

Around a mixture-of-experts layer's grouped products (fp8_grouped_gemm, int8_grouped_gemm):
``moe_route`` gives each token its experts and their weights, ``moe_place`` the grouped
products' offsets and which token each row is, ``moe_combine`` the weighted sum of a token's
rows. Each has its gradient beside it. Arguments are marshalled only; every step runs in the
kernels behind the C ABI.
"""
from __future__ import annotations

import torch

from ._lib import FP8Q_MOE_GROUP_MAX, FP8Q_MOE_KEEP_SCORES, FP8Q_MOE_SOFTMAX, lib
from ._tensor import CODE, launch, need, need_float

_SCORES = {"sigmoid": 0, "softmax": FP8Q_MOE_SOFTMAX}
_GROUPS = {"top2": 0, "max": FP8Q_MOE_GROUP_MAX}
MAX_EXPERTS, MAX_TOP_K, MAX_GROUPS = 1024, 32, 64


def _score_flags(score: str, renormalize: bool) -> int:
    if score not in _SCORES:
        raise ValueError('score must be "sigmoid" or "softmax"')
    return _SCORES[score] | (0 if renormalize else FP8Q_MOE_KEEP_SCORES)


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "sigmoid", bias: torch.Tensor | None = None,
              groups: int = 1, topk_groups: int = 1, group_score: str = "top2", renormalize: bool = True,
              scale: float = 1.0):
    """Each token's experts. logits [..., E] (float32 or bfloat16) are the gate's.

    Scores are sigmoid(x) or softmax(x); bias [E] (float32) is added for the selection only.
    With groups > 1 the experts are that many equal runs, of which the topk_groups with the
    largest value (the sum of a run's two largest choices, or with group_score="max" its
    largest) take part. Returns ``(weights, experts)``, both [..., top_k]: float32 weights
    (the scores, divided by their sum if renormalize, times scale) and int32 experts, the
    largest choice first, equal ones by index."""
    need_float(logits, "logits")
    if logits.dim() < 1:
        raise ValueError("logits must be [..., E]")
    E = logits.shape[-1]
    flags = _score_flags(score, renormalize)
    if group_score not in _GROUPS:
        raise ValueError('group_score must be "top2" or "max"')
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts are supported, got {E}")
    if not 1 <= groups <= MAX_GROUPS or E % groups or not 1 <= topk_groups <= groups:
        raise ValueError(f"groups must divide the experts (at most {MAX_GROUPS}) and be at least topk_groups")
    if not 1 <= top_k <= min(MAX_TOP_K, topk_groups * (E // groups)):
        raise ValueError(f"top_k must be 1 to {MAX_TOP_K} and at most the experts of the topk_groups groups")
    b_ptr = None
    if bias is not None:
        need(bias, "bias", torch.float32, (E,), device=logits.device)
        b_ptr = bias.data_ptr()
    shape = (*logits.shape[:-1], top_k)
    weights = logits.new_empty(shape, dtype=torch.float32)
    experts = torch.empty_like(weights, dtype=torch.int32)
    launch("moe_route", lib.moe_route, logits, logits.data_ptr(), CODE[logits.dtype], b_ptr, weights.data_ptr(),
           experts.data_ptr(), logits.numel() // E, E, top_k, groups, topk_groups, scale,
           flags | _GROUPS[group_score])
    return weights, experts


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
                       score: str = "sigmoid", renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of moe_route's weights with respect to the logits (which it has the shape and
    dtype of). dweights [..., k] float32 and experts [..., k] int32 as moe_route returned
    them; score, renormalize and scale as in that call. The selection has no gradient."""
    need_float(logits, "logits")
    if logits.dim() < 1 or not 1 <= logits.shape[-1] <= MAX_EXPERTS:
        raise ValueError(f"logits must be [..., E] with 1 to {MAX_EXPERTS} experts")
    need(experts, "experts", torch.int32, device=logits.device)
    if experts.shape[:-1] != logits.shape[:-1] or not 1 <= experts.shape[-1] <= MAX_TOP_K:
        raise ValueError(f"experts must be [..., k] for the logits' tokens, k at most {MAX_TOP_K}")
    need(dweights, "dweights", torch.float32, experts.shape, device=logits.device)
    flags = _score_flags(score, renormalize)
    E = logits.shape[-1]
    dlogits = torch.empty_like(logits)
    launch("moe_route_backward", lib.moe_route_backward, logits, dweights.data_ptr(), logits.data_ptr(),
           CODE[logits.dtype], experts.data_ptr(), dlogits.data_ptr(), logits.numel() // E, E, experts.shape[-1],
           scale, flags)
    return dlogits


def moe_place(experts: torch.Tensor, n_experts: int, *, first: int = 0):
    """Rows in expert order. experts [T, k] int32 are each token's; those in
    [first, first + n_experts) get rows (one GPU's experts of an expert-parallel layer).

    Returns ``(offsets, rows, slots)``: offsets int64 [n_experts + 1], the grouped products'
    bounds; rows int32 [T * k], each row's token (ascending within an expert; -1 past the
    last row, offsets[-1]); slots int32 [T, k], each choice's row or -1."""
    need(experts, "experts", torch.int32)
    if experts.dim() != 2 or not 1 <= experts.shape[1] <= MAX_TOP_K:
        raise ValueError(f"experts must be [T, k], k at most {MAX_TOP_K}")
    if not 1 <= n_experts <= MAX_EXPERTS or first < 0:
        raise ValueError(f"n_experts must be 1 to {MAX_EXPERTS} and first not negative")
    T, k = experts.shape
    offsets = experts.new_empty(n_experts + 1, dtype=torch.int64)
    rows = experts.new_empty(T * k)
    slots = torch.empty_like(experts)
    need_bytes = lib.moe_place_workspace_bytes(T, k, n_experts)
    # from torch's allocator, which keeps it from calls on other streams until this one is done
    ws = experts.new_empty(need_bytes, dtype=torch.uint8) if need_bytes else None
    launch("moe_place", lib.moe_place, experts, experts.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
           slots.data_ptr(), T, k, n_experts, first, ws.data_ptr() if need_bytes else None, need_bytes)
    return offsets, rows, slots


def _rows_of(h: torch.Tensor, slots: torch.Tensor) -> None:
    need_float(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be [rows, H]")
    need(slots, "slots", torch.int32, device=h.device)
    if slots.dim() != 2 or not 1 <= slots.shape[1] <= MAX_TOP_K:
        raise ValueError(f"slots must be [T, k], k at most {MAX_TOP_K}")


def moe_combine(h: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum over j of weights[t, j] * h[slots[t, j]], [T, H] in h's dtype (float32 or
    bfloat16), summed in float32. Slots outside h's rows (-1) add nothing. weights float32
    [T, k], or None for all 1: with moe_place's slots that is the gradient of x[rows]."""
    _rows_of(h, slots)
    w_ptr = None
    if weights is not None:
        need(weights, "weights", torch.float32, slots.shape, device=h.device)
        w_ptr = weights.data_ptr()
    T, k = slots.shape
    shape = (T, h.shape[1])
    if out is None:
        out = h.new_empty(shape)
    else:
        need_float(out, "out", h.dtype, shape, h.device)
    launch("moe_combine", lib.moe_combine, h, h.data_ptr(), CODE[h.dtype], slots.data_ptr(), w_ptr, out.data_ptr(),
           T, k, h.shape[0], h.shape[1])
    return out


def moe_combine_backward(dy: torch.Tensor, h: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor):
    """Gradients of moe_combine: ``(dh, dweights)``, dh[slots[t, j]] = weights[t, j] * dy[t] in
    h's shape and dtype and dweights[t, j] = <dy[t], h[slots[t, j]]> in float32. Rows of dh
    that no slot names are uninitialised (no expert owns them)."""
    _rows_of(h, slots)
    need(weights, "weights", torch.float32, slots.shape, device=h.device)
    T, k = slots.shape
    need_float(dy, "dy", h.dtype, (T, h.shape[1]), h.device)
    dh, dweights = torch.empty_like(h), torch.empty_like(weights)
    launch("moe_combine_backward", lib.moe_combine_backward, h, dy.data_ptr(), h.data_ptr(), CODE[h.dtype],
           slots.data_ptr(), weights.data_ptr(), dh.data_ptr(), dweights.data_ptr(), T, k, h.shape[0], h.shape[1])
    return dh, dweights
