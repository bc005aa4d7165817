"""torch front end of the global gradient norm and of clipping at it (forge_grad_norm /
forge_grad_clip of include/forge_adamw.h) over a list of fp32, bf16 and fp16 tensors."""
from __future__ import annotations

import torch

from . import _lib
from ._front import check, run

_CODE = {torch.float32: _lib.GRAD_F32, torch.bfloat16: _lib.GRAD_BF16,
         torch.float16: _lib.GRAD_F16}


def _table(grads, out):
    """The device, the number of tensors and the C ABI's table of them.  out None: the
    gradients are only read."""
    written = out is not None
    out = out if written else grads
    n = len(grads)
    if n < 1:
        raise ValueError("no gradients")
    if len(out) != n:
        raise ValueError(f"{n} gradients, {len(out)} outputs")
    if not isinstance(grads[0], torch.Tensor) or not grads[0].is_cuda:
        raise ValueError("gradients must be tensors on a CUDA device (there is no CPU path)")
    dev = grads[0].device
    index = dev.index
    fields = []
    for g, o in zip(grads, out):
        code = _CODE.get(getattr(g, "dtype", None))
        if code is None or g.get_device() != index or not g.is_contiguous():
            raise ValueError(f"gradients must be contiguous fp32, bf16 or fp16 tensors on {dev}")
        size = g.numel()
        if o is not g and (not isinstance(o, torch.Tensor) or o.dtype != g.dtype
                           or o.get_device() != index or o.shape != g.shape
                           or not o.is_contiguous()):
            raise ValueError("outputs must be contiguous and have their gradient's shape, type "
                             "and device")
        fields += (g.data_ptr(), o.data_ptr(), size, code)
    if written and len(set(fields[1::4])) < n:
        places = [p for p, size in zip(fields[1::4], fields[2::4]) if size]
        if len(set(places)) < len(places):
            raise ValueError("the same tensor is written twice")
    return dev, n, _lib.grad_table(fields, n)


def _workspace(n, workspace, dev):
    if workspace is None:
        return torch.empty(_lib.forge_grad_workspace_size(n), dtype=torch.uint8, device=dev)
    return check(workspace, "workspace", (torch.uint8,), dev)


def _norm(norm, dev):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device=dev)
    check(norm, "norm", (torch.float32,), dev)
    if norm.numel() != 1:
        raise ValueError("norm must have one element")
    return norm


def grad_norm(grads, norm=None, workspace=None):
    """The 2-norm of all values of `grads` (a sequence of contiguous fp32, bf16 or fp16 CUDA
    tensors) as a fp32 tensor; nothing is read back to the host."""
    dev, n, table = _table(list(grads), None)
    norm = _norm(norm, dev)
    ws = _workspace(n, workspace, dev)
    run(dev, "forge_grad_norm", _lib.forge_grad_norm, table, n, norm.data_ptr(), ws.data_ptr(),
        ws.numel())
    return norm


def grad_clip(grads, max_norm, out=None, norm=None, workspace=None):
    """Scales `grads` by max_norm / norm where their norm exceeds max_norm (> 0), in place or
    into the tensors `out`, and returns the norm (before clipping) as a fp32 tensor."""
    grads = list(grads)
    dev, n, table = _table(grads, grads if out is None else list(out))
    norm = _norm(norm, dev)
    ws = _workspace(n, workspace, dev)
    run(dev, "forge_grad_clip", _lib.forge_grad_clip, table, n, float(max_norm), norm.data_ptr(),
        ws.data_ptr(), ws.numel())
    return norm


def grad_workspace_bytes(n_tensors) -> int:
    return int(_lib.forge_grad_workspace_size(n_tensors))
