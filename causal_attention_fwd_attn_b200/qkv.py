"""torch front end of the stage between the QKV projection and the attention
(forge_qkv_fwd / forge_qkv_bwd of include/forge_attn.h): per-head RMS norm of queries and
keys, rotary positions with one or several axes, and the attention's head layout.

The projection's tensors are [B, T, heads, d] views, usually slices of one packed
[B, T, H + 2 Hkv, d] tensor; only the last dimension has to be contiguous.  T may be 1 (a
decoding step's tokens at positions of their own); attn_fwd reads q, k and v of one length and no
cache, so that where such k and v go is the caller's.  The checks, the
allocation and the call are in csrc/front.cpp.
"""
from __future__ import annotations

from . import _lib


def qkv_fwd(q, k, v, q_weight=None, k_weight=None, *, eps=1e-6, inv_freq=None, positions=None,
            pair_axis=None, adjacent=False, out=None):
    """The attention's q, k, v [B, H, T, d] from the projection's q [B, T, H, d] and k, v
    [B, T, Hkv, d] (bf16 or fp16, d 64 or 128, H a multiple of Hkv; key / value heads are
    repeated H / Hkv times).

    q_weight, k_weight: fp32 [d] weights of an RMS norm of every head (None: no norm).
    inv_freq: float64 [rot / 2], the angle per position of each pair of the first rot
    elements (None: no rotation).  positions: int32 [B, T] or [axes, B, T] (None: 0 .. T - 1);
    pair_axis: int32 [rot / 2], the axis of each pair (None: axis 0).  Pairs are
    (j, j + rot / 2), or with `adjacent` (2j, 2j + 1).  out: (q, k, v) to write into, three
    tensors that do not overlap."""
    return _lib.front().qkv_fwd(q, k, v, q_weight, k_weight, eps, inv_freq, positions, pair_axis,
                                adjacent, out)


def qkv_bwd(dq, dk, dv, q, k, q_weight=None, k_weight=None, *, eps=1e-6, inv_freq=None,
            positions=None, pair_axis=None, adjacent=False, out=None, weight_out=None,
            accumulate=False, workspace=None):
    """Gradients of qkv_fwd: (q, k, v, q_weight, k_weight), the first three laid out like the
    projection's tensors, the last two fp32 [d] (None where there is no weight).

    dq, dk, dv: contiguous [B, H, T, d], in q's type or fp32 (as attn_bwd returns them); q, k
    and the other arguments as for qkv_fwd.  out: (q, k, v) views to write into (default:
    slices of one packed [B, T, H + 2 Hkv, d] tensor).  weight_out: (q_weight, k_weight) to
    write into, or to add to with `accumulate`; two tensors, also where q and k share one
    weight (whose gradient is their sum).  workspace: uint8 of at least
    qkv_workspace_bytes(d)."""
    return _lib.front().qkv_bwd(dq, dk, dv, q, k, q_weight, k_weight, eps, inv_freq, positions,
                                pair_axis, adjacent, out, weight_out, accumulate, workspace)


def qkv_workspace_bytes(d) -> int:
    """Bytes of qkv_bwd's workspace for head dimension d."""
    return _lib.forge_qkv_bwd_workspace_size(d)
