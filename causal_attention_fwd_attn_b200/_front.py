"""What the torch front ends share: the call on the tensors' device and stream, and the
checks of the tensors handed to it."""
from __future__ import annotations

import torch

from . import _lib

DTYPES16 = (torch.bfloat16, torch.float16)


def run(device: torch.device, where: str, fn, *args) -> None:
    """fn(*args, stream) of the C ABI on `device`'s current stream, with that device current
    (a kernel is launched on the current device); raises on any status but OK."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if st != _lib.OK:
        raise _lib.ForgeAttnError(st, where)


def check(t, name: str, dtypes, device, shape=None) -> torch.Tensor:
    """`t` must be a contiguous CUDA tensor of one of `dtypes` on `device` (None: any CUDA
    device), of `shape` if that is given."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def address(t):
    return None if t is None else t.data_ptr()
