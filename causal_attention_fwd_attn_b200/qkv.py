"""torch front end of the stage between the QKV projection and the attention
(forge_qkv_fwd / forge_qkv_bwd of include/forge_attn.h): per-head RMS norm of queries and
keys, rotary positions with one or several axes, and the attention's head layout.

The projection's tensors are [B, T, heads, d] views, usually slices of one packed
[B, T, H + 2 Hkv, d] tensor; only the last dimension has to be contiguous.
"""
from __future__ import annotations

import torch

from . import _lib
from ._front import DTYPES16, address, check, run

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_F64 = (torch.float64,)


def _view(t, name, B, T, heads, d, dtype, device):
    """A projection-side tensor as the C ABI's descriptor."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (B, T, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, T, heads, d)}")
    sb, st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _lib.QkvTensor(t.data_ptr(), sb, st, sh)


def _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, device):
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            check(w, name, _F32, device, (d,))
    rot, axes = 0, 1
    if inv_freq is not None:
        check(inv_freq, "inv_freq", _F64, device)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be one-dimensional")
        pairs = inv_freq.numel()
        rot = 2 * pairs
        if positions is not None:
            check(positions, "positions", _I32, device)
            if positions.dim() == 3:
                axes = positions.shape[0]
            if axes < 1 or positions.shape[-2:] != (B, T) or positions.dim() not in (2, 3):
                raise ValueError(f"positions has shape {tuple(positions.shape)}, expected "
                                 f"{(B, T)} or (axes, {B}, {T})")
        if pair_axis is not None:
            check(pair_axis, "pair_axis", _I32, device, (pairs,))
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    return _lib.QkvConfig(B, T, H, Hkv, d, rot, axes, float(eps), address(inv_freq),
                          address(positions), address(pair_axis), address(q_weight),
                          address(k_weight))


def qkv_fwd(q, k, v, q_weight=None, k_weight=None, *, eps=1e-6, inv_freq=None, positions=None,
            pair_axis=None, adjacent=False, out=None):
    """The attention's q, k, v [B, H, T, d] from the projection's q [B, T, H, d] and k, v
    [B, T, Hkv, d] (bf16 or fp16, d 64 or 128, H a multiple of Hkv; key / value heads are
    repeated H / Hkv times).

    q_weight, k_weight: fp32 [d] weights of an RMS norm of every head (None: no norm).
    inv_freq: float64 [rot / 2], the angle per position of each pair of the first rot
    elements (None: no rotation).  positions: int32 [B, T] or [axes, B, T] (None: 0 .. T - 1 on
    every axis); pair_axis: int32 [rot / 2], the axis of each pair (None: axis 0).  Pairs are
    (j, j + rot / 2), or with `adjacent` (2j, 2j + 1).  out: (q, k, v) to write into."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not isinstance(k, torch.Tensor) \
            or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d] tensors")
    B, T, H, d = q.shape
    Hkv, dt, dev = k.shape[2], q.dtype, q.device
    if dt not in DTYPES16:
        raise ValueError(f"q has dtype {dt}, expected one of {DTYPES16}")
    vq = _view(q, "q", B, T, H, d, dt, None)
    vk = _view(k, "k", B, T, Hkv, d, dt, dev)
    vv = _view(v, "v", B, T, Hkv, d, dt, dev)
    cfg = _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, dev)
    if out is None:
        out = tuple(torch.empty((B, H, T, d), dtype=dt, device=dev) for _ in range(3))
    elif len(out) != 3:
        raise ValueError("out must be (q, k, v)")
    else:
        for name, t in zip(("q", "k", "v"), out):
            check(t, f"out {name}", (dt,), dev, (B, H, T, d))
    flags = (_lib.FP16 if dt == torch.float16 else 0) | (_lib.QKV_ADJACENT if adjacent else 0)
    run(dev, "forge_qkv_fwd", _lib.forge_qkv_fwd, cfg, vq, vk, vv, out[0].data_ptr(),
        out[1].data_ptr(), out[2].data_ptr(), flags)
    return tuple(out)


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
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not isinstance(k, torch.Tensor) \
            or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d] tensors")
    B, T, H, d = q.shape
    Hkv, dt, dev = k.shape[2], q.dtype, q.device
    if dt not in DTYPES16:
        raise ValueError(f"q has dtype {dt}, expected one of {DTYPES16}")
    vq = _view(q, "q", B, T, H, d, dt, None)
    vk = _view(k, "k", B, T, Hkv, d, dt, dev)
    check(dq, "dq", (dt, torch.float32), dev, (B, H, T, d))
    check(dk, "dk", (dq.dtype,), dev, (B, H, T, d))
    check(dv, "dv", (dq.dtype,), dev, (B, H, T, d))
    cfg = _config(B, T, H, Hkv, d, eps, q_weight, k_weight, inv_freq, positions, pair_axis, dev)
    if out is None:
        packed = torch.empty((B, T, H + 2 * Hkv, d), dtype=dt, device=dev)
        out = (packed[:, :, :H], packed[:, :, H:H + Hkv], packed[:, :, H + Hkv:])
    elif len(out) != 3:
        raise ValueError("out must be (q, k, v)")
    views = [_view(t, f"out {n}", B, T, h, d, dt, dev)
             for n, t, h in zip(("q", "k", "v"), out, (H, Hkv, Hkv))]
    gw = [None, None]
    ws = None
    if accumulate and weight_out is None:
        raise ValueError("accumulate needs weight_out")
    if q_weight is not None or k_weight is not None:
        if weight_out is None:
            weight_out = (None, None)
        elif len(weight_out) != 2:
            raise ValueError("weight_out must be (q_weight, k_weight)")
        for j, w in enumerate((q_weight, k_weight)):
            if w is None:
                continue
            if weight_out[j] is None:
                if accumulate:
                    raise ValueError("accumulate needs weight_out")
                gw[j] = torch.empty(d, dtype=torch.float32, device=dev)
            else:
                gw[j] = check(weight_out[j], "weight_out", _F32, dev, (d,))
        ws = workspace
        if ws is None:
            ws = torch.empty(qkv_workspace_bytes(d, dev), dtype=torch.uint8, device=dev)
        else:
            check(ws, "workspace", (torch.uint8,), dev)
    flags = ((_lib.FP16 if dt == torch.float16 else 0) | (_lib.QKV_ADJACENT if adjacent else 0)
             | (_lib.QKV_GRAD_F32 if dq.dtype == torch.float32 else 0))
    run(dev, "forge_qkv_bwd", _lib.forge_qkv_bwd, cfg, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        vq, vk, *views, address(gw[0]), address(gw[1]), int(bool(accumulate)), address(ws),
        0 if ws is None else ws.numel(), flags)
    return (*out, *gw)


def qkv_workspace_bytes(d, device=None) -> int:
    """Bytes of qkv_bwd's workspace for head dimension d on `device` (default: the current)."""
    if device is None or device.index is None or torch.cuda.current_device() == device.index:
        return int(_lib.forge_qkv_bwd_workspace_size(d))
    with torch.cuda.device(device):
        return int(_lib.forge_qkv_bwd_workspace_size(d))
