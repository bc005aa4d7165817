"""torch front end of the global gradient norm and of clipping at it (forge_grad_norm /
forge_grad_clip of include/forge_adamw.h) over a list of fp32, bf16 and fp16 tensors.  The
checks, the allocation and the call are in csrc/front.cpp."""
from __future__ import annotations

from . import _lib


def grad_norm(grads, norm=None, workspace=None):
    """The 2-norm of all values of `grads` (a sequence of contiguous fp32, bf16 or fp16 CUDA
    tensors, each starting on 16 bytes: slices of a packed buffer have to be placed so) as a fp32
    tensor; nothing is read back to the host.  norm: a tensor of one
    element to write it into; workspace: uint8 of at least grad_workspace_bytes()."""
    return _lib.front().grad(grads, False, 0.0, None, norm, workspace)


def grad_clip(grads, max_norm, out=None, norm=None, workspace=None):
    """Scales `grads` by max_norm / norm where their norm exceeds max_norm (> 0), in place or
    into the tensors `out`, and returns the norm (before clipping) as a fp32 tensor.  For
    gradients that something else than forge_adamw_step reads, which clips its fp32 ones itself."""
    return _lib.front().grad(grads, True, max_norm, out, norm, workspace)


def grad_workspace_bytes(n_tensors) -> int:
    return _lib.forge_grad_workspace_size(n_tensors)
