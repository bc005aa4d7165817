"""What the torch front ends share: the call on the tensors' device and stream, and the
checks of the tensors handed to it.

A call on a few rows takes the GPU less time than the host spends on it, so the checks are
written to cost little where they pass: one expression, and the search for what is wrong only
after it has failed.
"""
from __future__ import annotations

import torch

from . import _lib

DTYPES16 = (torch.bfloat16, torch.float16)

_raw_stream = torch._C._cuda_getCurrentRawStream


def run(index: int, where: str, fn, *args) -> None:
    """fn(*args, stream) of the C ABI on CUDA device `index`'s current stream, with that device
    current (a kernel is launched on the current device); raises on any status but OK."""
    if torch.cuda.current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != _lib.OK:
        raise _lib.ForgeAttnError(st, where)


def check(t, name: str, dtypes, index, shape=None) -> torch.Tensor:
    """`t` must be a contiguous tensor of one of `dtypes` on CUDA device `index`, of `shape` if
    that is given."""
    if (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype in dtypes
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t
    refuse(t, name, dtypes, index, shape)
    raise ValueError(f"{name} must be contiguous")


def refuse(t, name, dtypes, index, shape) -> None:
    """Raises for the first thing wrong with `t` (its strides apart)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def address(t):
    return None if t is None else t.data_ptr()
