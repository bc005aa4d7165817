"""torch front end of the stage between the QKV projection and the attention
(forge_qkv_fwd / forge_qkv_bwd of include/forge_attn.h): per-head RMS norm of queries and
keys, rotary positions with one or several axes, and the attention's head layout.

The projection's tensors are [B, T, heads, d] views, usually slices of one packed
[B, T, H + 2 Hkv, d] tensor; only the last dimension has to be contiguous.
"""
from __future__ import annotations

import torch

from . import _lib
from ._front import DTYPES16, address, check, refuse, run

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_F64 = (torch.float64,)


def _view(t, name, shape, dtype, index):
    """A projection-side tensor as the C ABI's descriptor."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype is not dtype
            or t.shape != shape):
        refuse(t, name, (dtype,), index, shape)
    sb, st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _lib.qkv_tensor(t.data_ptr(), sb, st, sh)


def _sizes(q, k):
    """B, T, H, Hkv, d, the type and the device's index."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not isinstance(k, torch.Tensor) \
            or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d] tensors")
    B, T, H, d = q.shape
    if q.dtype not in DTYPES16:
        raise ValueError(f"q has dtype {q.dtype}, expected one of {DTYPES16}")
    index = q.get_device()
    if index < 0:
        raise ValueError("q must be on a CUDA device (there is no CPU path)")
    return B, T, H, k.shape[2], d, q.dtype, index


def _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, index):
    if q_weight is not None:
        check(q_weight, "q_weight", _F32, index, (d,))
    if k_weight is not None:
        check(k_weight, "k_weight", _F32, index, (d,))
    rot, axes = 0, 1
    if inv_freq is not None:
        check(inv_freq, "inv_freq", _F64, index)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be one-dimensional")
        pairs = inv_freq.numel()
        rot = 2 * pairs
        if positions is not None:
            check(positions, "positions", _I32, index)
            shape = positions.shape
            if len(shape) == 3:
                axes = shape[0]
            if axes < 1 or len(shape) not in (2, 3) or shape[-2] != B or shape[-1] != T:
                raise ValueError(f"positions has shape {tuple(shape)}, expected {(B, T)} or "
                                 f"(axes, {B}, {T})")
        if pair_axis is not None:
            check(pair_axis, "pair_axis", _I32, index, (pairs,))
            if positions is None:
                raise ValueError("pair_axis needs positions")
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    return _lib.qkv_config(B, T, H, Hkv, d, rot, axes, eps, address(inv_freq), address(positions),
                           address(pair_axis), address(q_weight), address(k_weight))


def qkv_fwd(q, k, v, q_weight=None, k_weight=None, *, eps=1e-6, inv_freq=None, positions=None,
            pair_axis=None, adjacent=False, out=None):
    """The attention's q, k, v [B, H, T, d] from the projection's q [B, T, H, d] and k, v
    [B, T, Hkv, d] (bf16 or fp16, d 64 or 128, H a multiple of Hkv; key / value heads are
    repeated H / Hkv times).

    q_weight, k_weight: fp32 [d] weights of an RMS norm of every head (None: no norm).
    inv_freq: float64 [rot / 2], the angle per position of each pair of the first rot
    elements (None: no rotation).  positions: int32 [B, T] or [axes, B, T] (None: 0 .. T - 1);
    pair_axis: int32 [rot / 2], the axis of each pair (None: axis 0).  Pairs are
    (j, j + rot / 2), or with `adjacent` (2j, 2j + 1).  out: (q, k, v) to write into."""
    B, T, H, Hkv, d, dt, index = _sizes(q, k)
    vq = _view(q, "q", (B, T, H, d), dt, index)
    vk = _view(k, "k", (B, T, Hkv, d), dt, index)
    vv = _view(v, "v", (B, T, Hkv, d), dt, index)
    cfg = _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, index)
    shape = (B, H, T, d)
    if out is None:
        out = tuple(torch.empty(shape, dtype=dt, device=q.device) for _ in range(3))
    elif len(out) != 3:
        raise ValueError("out must be (q, k, v)")
    oq, ok, ov = out
    kinds = (dt,)
    check(oq, "out q", kinds, index, shape)
    check(ok, "out k", kinds, index, shape)
    check(ov, "out v", kinds, index, shape)
    flags = (_lib.FP16 if dt is torch.float16 else 0) | (_lib.QKV_ADJACENT if adjacent else 0)
    run(index, "forge_qkv_fwd", _lib.forge_qkv_fwd, cfg, vq, vk, vv, oq.data_ptr(), ok.data_ptr(),
        ov.data_ptr(), flags)
    return oq, ok, ov


def qkv_bwd(dq, dk, dv, q, k, q_weight=None, k_weight=None, *, eps=1e-6, inv_freq=None,
            positions=None, pair_axis=None, adjacent=False, out=None, weight_out=None,
            accumulate=False, workspace=None):
    """Gradients of qkv_fwd: (q, k, v, q_weight, k_weight), the first three laid out like the
    projection's tensors, the last two fp32 [d] (None where there is no weight).

    dq, dk, dv: contiguous [B, H, T, d], in q's type or fp32 (as attn_bwd returns them); q, k
    and the other arguments as for qkv_fwd.  out: (q, k, v) views to write into (default:
    slices of one packed [B, T, H + 2 Hkv, d] tensor).  weight_out: (q_weight, k_weight) to
    write into, or to add to with `accumulate`.  workspace: uint8 of at least
    qkv_workspace_bytes(d)."""
    B, T, H, Hkv, d, dt, index = _sizes(q, k)
    vq = _view(q, "q", (B, T, H, d), dt, index)
    vk = _view(k, "k", (B, T, Hkv, d), dt, index)
    shape = (B, H, T, d)
    check(dq, "dq", (dt, torch.float32), index, shape)
    kinds = (dq.dtype,)
    check(dk, "dk", kinds, index, shape)
    check(dv, "dv", kinds, index, shape)
    cfg = _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, index)
    dev = q.device
    if out is None:
        packed = torch.empty((B, T, H + 2 * Hkv, d), dtype=dt, device=dev)
        out = (packed[:, :, :H], packed[:, :, H:H + Hkv], packed[:, :, H + Hkv:])
    elif len(out) != 3:
        raise ValueError("out must be (q, k, v)")
    gq, gk, gv = out
    oq = _view(gq, "out q", (B, T, H, d), dt, index)
    ok = _view(gk, "out k", (B, T, Hkv, d), dt, index)
    ov = _view(gv, "out v", (B, T, Hkv, d), dt, index)
    gwq = gwk = ws = None
    ws_bytes = 0
    if accumulate and weight_out is None:
        raise ValueError("accumulate needs weight_out")
    if q_weight is not None or k_weight is not None:
        given = (None, None) if weight_out is None else weight_out
        if len(given) != 2:
            raise ValueError("weight_out must be (q_weight, k_weight)")
        gwq, gwk = (_weight_out(w, g, d, accumulate, index, dev)
                    for w, g in zip((q_weight, k_weight), given))
        ws = workspace
        if ws is None:
            ws = torch.empty(qkv_workspace_bytes(d, index), dtype=torch.uint8, device=dev)
        check(ws, "workspace", (torch.uint8,), index)
        ws_bytes = ws.numel()
    flags = ((_lib.FP16 if dt is torch.float16 else 0) | (_lib.QKV_ADJACENT if adjacent else 0)
             | (_lib.QKV_GRAD_F32 if dq.dtype is torch.float32 else 0))
    run(index, "forge_qkv_bwd", _lib.forge_qkv_bwd, cfg, dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), vq, vk, oq, ok, ov, address(gwq), address(gwk), 1 if accumulate else 0,
        address(ws), ws_bytes, flags)
    return gq, gk, gv, gwq, gwk


def _weight_out(weight, given, d, accumulate, index, dev):
    if weight is None:
        return None
    if given is None:
        if accumulate:
            raise ValueError("accumulate needs weight_out")
        return torch.empty(d, dtype=torch.float32, device=dev)
    return check(given, "weight_out", _F32, index, (d,))


def qkv_workspace_bytes(d, index=None) -> int:
    """Bytes of qkv_bwd's workspace for head dimension d on CUDA device `index` (default: the
    current one)."""
    if index is None or torch.cuda.current_device() == index:
        return _lib.forge_qkv_bwd_workspace_size(d)
    with torch.cuda.device(index):
        return _lib.forge_qkv_bwd_workspace_size(d)
