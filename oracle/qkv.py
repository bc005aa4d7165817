"""fp64 CPU oracle of the stage between a QKV projection and the attention: per-head RMS
norm, rotary positions over several axes, head layout; forward and backward.

TEST INFRASTRUCTURE ONLY: the tests are the only callers; the CUDA library never imports or
calls anything here, and this module imports nothing from the library.

For a head x of d elements of token (b, t):
  r = 1 / sqrt(mean x^2 + eps),  n = r x * w                       (w None: n = x)
  pair j of the first 2 * len(freq) elements is a complex number, multiplied by
  exp(i pos[axis_j][b][t] freq_j)
and head g of k and v becomes the heads [g rep, (g + 1) rep) of the result, rep = H / Hkv.
Backward: the transposed maps in reverse order, written out below.
"""
from __future__ import annotations

import numpy as np


def angles(freq, positions, pair_axis, B, T):
    """[B, T, pairs]; positions [axes, B, T] or None (the token's index)."""
    freq = np.asarray(freq, dtype=np.float64)
    if positions is None:
        positions = np.broadcast_to(np.arange(T), (1, B, T))
        pair_axis = None
    p = np.asarray(positions, dtype=np.float64)
    axis = np.zeros(len(freq), dtype=int) if pair_axis is None else np.asarray(pair_axis)
    return np.moveaxis(p[axis], 0, -1) * freq


def rotate(x, phi, adjacent):
    """x: [B, T, heads, d]; phi: [B, T, pairs]."""
    pairs = phi.shape[-1]
    y = np.array(x, dtype=np.float64)
    if adjacent:
        a, b = y[..., 0:2 * pairs:2].copy(), y[..., 1:2 * pairs:2].copy()
    else:
        a, b = y[..., :pairs].copy(), y[..., pairs:2 * pairs].copy()
    z = (a + 1j * b) * np.exp(1j * phi)[:, :, None, :]
    if adjacent:
        y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2] = z.real, z.imag
    else:
        y[..., :pairs], y[..., pairs:2 * pairs] = z.real, z.imag
    return y


def head_fwd(x, w, phi, adjacent, eps, rep=1):
    """One projection [B, T, heads, d] to [B, heads * rep, T, d].  phi None: no rotation."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(w)
    if phi is not None:
        y = rotate(y, phi, adjacent)
    return np.repeat(np.swapaxes(y, 1, 2), rep, axis=1)


def head_bwd(dy, x, w, phi, adjacent, eps, rep=1):
    """Gradients (of x, of w or None) of head_fwd for dy [B, heads * rep, T, d]."""
    dy = np.asarray(dy, dtype=np.float64)
    B, H, T, d = dy.shape
    g = np.swapaxes(dy.reshape(B, H // rep, rep, T, d).sum(axis=2), 1, 2)
    if phi is not None:
        g = rotate(g, -phi, adjacent)
    if w is None:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r
    u = g * np.asarray(w, dtype=np.float64)
    return r * (u - n * np.mean(u * n, axis=-1, keepdims=True)), (g * n).sum(axis=(0, 1, 2))
