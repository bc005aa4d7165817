"""torch front end of the global gradient norm and of clipping at it (forge_grad_norm /
forge_grad_clip of include/forge_adamw.h) over a list of fp32, bf16 and fp16 tensors."""
from __future__ import annotations

import torch

from . import _lib
from ._front import check, run

_CODE = {torch.float32: _lib.GRAD_F32, torch.bfloat16: _lib.GRAD_BF16,
         torch.float16: _lib.GRAD_F16}


def _columns(tensors, index, what):
    """Addresses, sizes and type codes of contiguous tensors on CUDA device `index`."""
    try:
        codes = [_CODE[t.dtype] for t in tensors]
        if {t.get_device() for t in tensors} == {index} and all([t.is_contiguous() for t in tensors]):
            return [t.data_ptr() for t in tensors], [t.numel() for t in tensors], codes
    except (AttributeError, KeyError):
        pass
    raise ValueError(f"{what} must be contiguous fp32, bf16 or fp16 tensors on cuda:{index}")


def _table(grads, out):
    """The device's index, the number of tensors and the C ABI's table of them.  out None: the
    gradients are only read."""
    n = len(grads)
    if n < 1:
        raise ValueError("no gradients")
    if not isinstance(grads[0], torch.Tensor) or not grads[0].is_cuda:
        raise ValueError("gradients must be tensors on a CUDA device (there is no CPU path)")
    index = grads[0].get_device()
    places, sizes, codes = _columns(grads, index, "gradients")
    fields = [0] * (4 * n)
    fields[0::4], fields[2::4], fields[3::4] = places, sizes, codes
    if out is not None:
        if out is not grads:
            if len(out) != n:
                raise ValueError(f"{n} gradients, {len(out)} outputs")
            places, out_sizes, out_codes = _columns(out, index, "outputs")
            if out_sizes != sizes or out_codes != codes:
                raise ValueError("outputs must have their gradients' sizes and types")
        if len(set(places)) < n:
            written = [p for p, size in zip(places, sizes) if size]
            if len(set(written)) < len(written):
                raise ValueError("the same tensor is written twice")
    fields[1::4] = places
    return index, n, _lib.grad_table(fields, n)


def _workspace(n, workspace, index):
    if workspace is None:
        return torch.empty(_lib.forge_grad_workspace_size(n), dtype=torch.uint8,
                           device=torch.device("cuda", index))
    return check(workspace, "workspace", (torch.uint8,), index)


def _norm(norm, index):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device=torch.device("cuda", index))
    check(norm, "norm", (torch.float32,), index)
    if norm.numel() != 1:
        raise ValueError("norm must have one element")
    return norm


def grad_norm(grads, norm=None, workspace=None):
    """The 2-norm of all values of `grads` (a sequence of contiguous fp32, bf16 or fp16 CUDA
    tensors) as a fp32 tensor; nothing is read back to the host."""
    index, n, table = _table(list(grads), None)
    norm = _norm(norm, index)
    ws = _workspace(n, workspace, index)
    run(index, "forge_grad_norm", _lib.forge_grad_norm, table, n, norm.data_ptr(), ws.data_ptr(),
        ws.numel())
    return norm


def grad_clip(grads, max_norm, out=None, norm=None, workspace=None):
    """Scales `grads` by max_norm / norm where their norm exceeds max_norm (> 0), in place or
    into the tensors `out`, and returns the norm (before clipping) as a fp32 tensor."""
    grads = list(grads)
    index, n, table = _table(grads, grads if out is None else list(out))
    norm = _norm(norm, index)
    ws = _workspace(n, workspace, index)
    run(index, "forge_grad_clip", _lib.forge_grad_clip, table, n, float(max_norm), norm.data_ptr(),
        ws.data_ptr(), ws.numel())
    return norm


def grad_workspace_bytes(n_tensors) -> int:
    return int(_lib.forge_grad_workspace_size(n_tensors))
