"""Pins of the fp64 oracles of the operators around the attention (CPU): the QKV stage, the
grouped products and gradient clipping.  None re-types an oracle: plain loops, central
differences, torch autograd in float64 and closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import grads as og
from oracle import linear as ol
from oracle import qkv as oq


def _stage(seed, B=2, T=3, heads=2, d=8, pairs=3, axes=2):
    r = np.random.default_rng(seed)
    x = r.normal(size=(B, T, heads, d))
    w = 1 + 0.3 * r.normal(size=d)
    freq = r.uniform(0.1, 2.0, size=pairs)
    pos = r.integers(-50, 50, size=(axes, B, T))
    axis = r.integers(0, axes, size=pairs)
    return x, w, freq, pos, axis


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_stage_forward_by_loops(adjacent, normed):
    x, w, freq, pos, axis = _stage(1)
    B, T, heads, d = x.shape
    eps = 0.01
    got = oq.head_fwd(x, w if normed else None, oq.angles(freq, pos, axis, B, T), adjacent, eps, 2)
    for b in range(B):
        for t in range(T):
            for h in range(2 * heads):
                v = [float(e) for e in x[b, t, h // 2]]
                if normed:
                    rms = math.sqrt(math.fsum(e * e for e in v) / d + eps)
                    v = [e / rms * float(g) for e, g in zip(v, w)]
                for j, f in enumerate(freq):
                    a, c = (2 * j, 2 * j + 1) if adjacent else (j, j + len(freq))
                    phi = float(pos[axis[j], b, t]) * float(f)
                    v[a], v[c] = (v[a] * math.cos(phi) - v[c] * math.sin(phi),
                                  v[a] * math.sin(phi) + v[c] * math.cos(phi))
                np.testing.assert_allclose(got[b, h, t], v, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_stage_backward_by_differences(adjacent, normed):
    x, w, freq, pos, axis = _stage(2)
    B, T, heads, d = x.shape
    phi = oq.angles(freq, pos, axis, B, T)
    dy = np.random.default_rng(3).normal(size=(B, heads * 3, T, d))
    gx, gw = oq.head_bwd(dy, x, w if normed else None, phi, adjacent, 0.02, 3)

    def loss(xx, ww):
        return float(np.sum(dy * oq.head_fwd(xx, ww if normed else None, phi, adjacent, 0.02, 3)))

    h = 1e-5
    num = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        num[i] = (loss(x + e, w) - loss(x - e, w)) / (2 * h)
    np.testing.assert_allclose(gx, num, rtol=1e-6, atol=1e-7)
    if not normed:
        assert gw is None
        return
    num = np.zeros_like(w)
    for i in range(d):
        e = np.zeros_like(w)
        e[i] = h
        num[i] = (loss(x, w + e) - loss(x, w - e)) / (2 * h)
    np.testing.assert_allclose(gw, num, rtol=1e-6, atol=1e-7)


def test_rotation_keeps_lengths_and_relative_positions():
    x, _, freq, _, _ = _stage(4)
    B, T, heads, d = x.shape
    a = oq.head_fwd(x, None, oq.angles(freq, None, None, B, T), False, 0.0)
    np.testing.assert_allclose((a * a).sum(-1), np.swapaxes((x * x).sum(-1), 1, 2), rtol=1e-12)
    # products of two tokens depend on the difference of their positions only
    far = np.broadcast_to(np.arange(T) + 1000, (1, B, T))
    b = oq.head_fwd(x, None, oq.angles(freq, far, None, B, T), False, 0.0)
    np.testing.assert_allclose(a @ np.swapaxes(a, 2, 3), b @ np.swapaxes(b, 2, 3), rtol=1e-9,
                               atol=1e-10)


def test_grouped_products_by_autograd():
    r = np.random.default_rng(5)
    offsets = [0, 3, 3, 7, 8]
    x, dy, w = r.normal(size=(9, 4)), r.normal(size=(9, 5)), r.normal(size=(4, 5, 4))
    tx, tw = (torch.tensor(t, requires_grad=True) for t in (x, w))
    y = torch.cat([tx[a:b] @ tw[e].T for e, (a, b) in enumerate(zip(offsets[:-1], offsets[1:]))])
    np.testing.assert_allclose(ol.grouped_fwd(x, w, offsets)[:8], y.detach().numpy(), rtol=1e-12)
    assert np.isnan(ol.grouped_fwd(x, w, offsets)[8]).all()
    gx, gw = torch.autograd.grad(y, (tx, tw), torch.tensor(dy[:8]))
    np.testing.assert_allclose(ol.grouped_bwd_dx(dy, w, offsets)[:8], gx[:8].numpy(), rtol=1e-12)
    np.testing.assert_allclose(ol.grouped_bwd_dw(dy, x, offsets), gw.numpy(), rtol=1e-12)
    assert (ol.grouped_bwd_dw(dy, x, offsets)[1] == 0).all()


def test_clipping_by_hand():
    norm, out = og.grad_clip([np.array([3.0]), np.array([0.0, -4.0])], 2.5)
    assert norm == pytest.approx(5.0, rel=1e-15)
    np.testing.assert_allclose(np.concatenate(out), [1.5, 0.0, -2.0], rtol=1e-15)
    norm, out = og.grad_clip([np.array([3.0]), np.array([0.0, -4.0])], 5.0)
    np.testing.assert_array_equal(np.concatenate(out), [3.0, 0.0, -4.0])
    assert og.grad_norm([np.zeros(3), np.zeros(0)]) == 0.0
    assert og.grad_norm([np.full(4, 1e200)]) == pytest.approx(2e200, rel=1e-14)
    p = [torch.randn(7, 3, dtype=torch.float64, requires_grad=True), torch.randn(5, dtype=torch.float64,
                                                                                 requires_grad=True)]
    for t in p:
        t.grad = torch.randn_like(t)
    g = [t.grad.numpy().copy() for t in p]
    want = torch.nn.utils.clip_grad_norm_(p, 0.5)
    norm, out = og.grad_clip(g, 0.5)
    assert norm == pytest.approx(float(want), rel=1e-12)
    for t, o in zip(p, out):  # torch adds 1e-6 to the norm
        np.testing.assert_allclose(t.grad.numpy(), o, rtol=1e-5)
