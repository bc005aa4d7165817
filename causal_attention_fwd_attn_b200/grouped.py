"""torch front end of the linear products grouped by expert (forge_linear_grouped_* of
include/forge_linear.h).

Token matrices hold the experts' rows one after the other; offsets, an int32 CUDA tensor
[experts + 1], says where each expert's begin.  It is read on the GPU only.
"""
from __future__ import annotations

import torch

from . import _lib
from ._front import DTYPES16, check, run

_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _rows(a, b, offsets, a_name, b_name, b_dims):
    """Checks the first operand (2-D), the second (`b_dims`-D) and the offsets; returns the
    device's index and the type's flag."""
    index = a.get_device() if isinstance(a, torch.Tensor) else -1
    check(a, a_name, DTYPES16, max(index, 0))
    check(b, b_name, (a.dtype,), index)
    if a.dim() != 2 or b.dim() != b_dims:
        raise ValueError(f"{a_name} must be 2-dimensional and {b_name} {b_dims}-dimensional")
    check(offsets, "offsets", _I32, index)
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be an int32 tensor [experts + 1]")
    return index, _lib.FP16 if a.dtype is torch.float16 else 0


def _experts(w, offsets):
    if w.shape[0] != offsets.numel() - 1:
        raise ValueError(f"w has {w.shape[0]} experts, offsets {offsets.numel() - 1}")


def _out(out, out_dtype, shape, dtype, index):
    if out is not None:
        return check(out, "out", (dtype, torch.float32), index, shape)
    out_dtype = dtype if out_dtype is None else out_dtype
    if out_dtype not in (dtype, torch.float32):
        raise ValueError(f"out_dtype must be {dtype} or torch.float32")
    return torch.empty(shape, dtype=out_dtype, device=torch.device("cuda", index))


def linear_grouped_fwd(x, w, offsets, out=None, out_dtype=None):
    """y[r] = x[r] w_e^T for the rows r of each expert e.  x: [rows, in] bf16 or fp16; w:
    [experts, out, in] of the same type; y: [rows, out] in that type or fp32 (out's, or
    out_dtype).  Rows of no expert are left as they were (undefined in a new tensor)."""
    index, flags = _rows(x, w, offsets, "x", "w", 3)
    _experts(w, offsets)
    E, fout, fin = w.shape
    rows = x.shape[0]
    if x.shape[1] != fin:
        raise ValueError(f"x has {x.shape[1]} features, w takes {fin}")
    y = _out(out, out_dtype, (rows, fout), x.dtype, index)
    run(index, "forge_linear_grouped_fwd", _lib.forge_linear_grouped_fwd, x.data_ptr(), w.data_ptr(),
        y.data_ptr(), offsets.data_ptr(), rows, E, fin, fout,
        flags | (_lib.OUT_F32 if y.dtype is torch.float32 else 0))
    return y


def linear_grouped_bwd_dx(dy, w, offsets, out=None, out_dtype=None):
    """dx[r] = dy[r] w_e for the rows r of each expert e.  dy: [rows, out]; w: [experts, out,
    in]; dx: [rows, in].  Types and rows of no expert as for linear_grouped_fwd."""
    index, flags = _rows(dy, w, offsets, "dy", "w", 3)
    _experts(w, offsets)
    E, fout, fin = w.shape
    rows = dy.shape[0]
    if dy.shape[1] != fout:
        raise ValueError(f"dy has {dy.shape[1]} features, w gives {fout}")
    dx = _out(out, out_dtype, (rows, fin), dy.dtype, index)
    run(index, "forge_linear_grouped_bwd_dx", _lib.forge_linear_grouped_bwd_dx, dy.data_ptr(),
        w.data_ptr(), dx.data_ptr(), offsets.data_ptr(), rows, E, fin, fout,
        flags | (_lib.OUT_F32 if dx.dtype is torch.float32 else 0))
    return dx


def linear_grouped_bwd_dw(dy, x, offsets, out=None, accumulate=False):
    """dw_e = sum over expert e's rows r of dy[r]^T x[r], fp32 [experts, out, in]; accumulate
    adds to `out`.  An expert without rows gets zeros (accumulate: keeps its values)."""
    index, flags = _rows(dy, x, offsets, "dy", "x", 2)
    rows, fout = dy.shape
    fin = x.shape[1]
    if x.shape[0] != rows:
        raise ValueError(f"x has {x.shape[0]} rows, dy {rows}")
    E = offsets.numel() - 1
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((E, fout, fin), dtype=torch.float32, device=dy.device)
    else:
        check(out, "out", _F32, index, (E, fout, fin))
    run(index, "forge_linear_grouped_bwd_dw", _lib.forge_linear_grouped_bwd_dw, dy.data_ptr(),
        x.data_ptr(), out.data_ptr(), offsets.data_ptr(), rows, E, fin, fout,
        int(bool(accumulate)), flags)
    return out
