"""torch front end of the linear products grouped by expert (forge_linear_grouped_* of
include/forge_linear.h).

Token matrices hold the experts' rows one after the other; offsets, an int32 CUDA tensor
[experts + 1], says where each expert's begin.  It is read on the GPU only.  The checks, the
allocation and the call are in csrc/front.cpp.
"""
from __future__ import annotations

import torch

from . import _lib


def _fp32(out_dtype, dtype):
    if out_dtype is None:
        return None
    if out_dtype not in (dtype, torch.float32):
        raise ValueError(f"out_dtype must be {dtype} or torch.float32")
    return out_dtype is torch.float32


def linear_grouped_fwd(x, w, offsets, out=None, out_dtype=None):
    """y[r] = x[r] w_e^T for the rows r of each expert e.  x: [rows, in] bf16 or fp16; w:
    [experts, out, in] of the same type; y: [rows, out] in that type or fp32 (out's, or
    out_dtype).  Rows of no expert are left as they were (undefined in a new tensor)."""
    return _lib.front().grouped_fwd(x, w, offsets, out,
                                    None if out_dtype is None else _fp32(out_dtype, x.dtype))


def linear_grouped_bwd_dx(dy, w, offsets, out=None, out_dtype=None):
    """dx[r] = dy[r] w_e for the rows r of each expert e.  dy: [rows, out]; w: [experts, out,
    in]; dx: [rows, in].  Types and rows of no expert as for linear_grouped_fwd."""
    return _lib.front().grouped_dx(dy, w, offsets, out,
                                   None if out_dtype is None else _fp32(out_dtype, dy.dtype))


def linear_grouped_bwd_dw(dy, x, offsets, out=None, accumulate=False):
    """dw_e = sum over expert e's rows r of dy[r]^T x[r], fp32 [experts, out, in]; accumulate
    adds to `out`.  An expert without rows gets zeros (accumulate: keeps its values)."""
    return _lib.front().grouped_dw(dy, x, offsets, out, accumulate)
