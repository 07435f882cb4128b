"""The native binding of the routed-expert, 8-bit integer and dense-block operators (csrc/binding.cpp): it
checks arguments, allocates outputs with torch and calls libfp8q.so. No fallback: if it is
missing the import fails."""
from __future__ import annotations

import torch

from . import _lib  # noqa: F401  (libfp8q.so, and the error that _native raises for its statuses)

try:
    from . import _native as native
except ImportError as e:
    raise ImportError(
        f"the native binding cannot be loaded ({e}): build it with "
        "`python -c 'import __graft_entry__ as g; g.build()'`; there is no fallback implementation") from e

OUT_TYPES = {torch.float32: _lib.FP8Q_OUT_F32, torch.bfloat16: _lib.FP8Q_OUT_BF16}


def out_code(out_dtype) -> int:
    code = OUT_TYPES.get(out_dtype)
    if code is None:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    return code
