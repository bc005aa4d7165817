"""One training step of a decoder layer with the operators as they are used together (GPU):
QKV projection, per-head norm and rotation into the attention's layout, attention, experts
over rows sorted by a router, all of it backward, clipping, AdamW; against torch autograd in
float64 on the same values.

Tolerances, from the arithmetic: a bf16 rounding is off by at most 2^-8 and 2^-8 / sqrt(3) in
the mean square; the longest chain (input gradients of the projection) passes 12 of them
(projection, rotation, P, O, two expert products, their three gradients, dS, dQ, its rotation),
each of full relative size at most once: sqrt(12) 2^-8 / sqrt(3) = 7.9e-3.  Terms that cancel
(P (dP - D), the norm's backward) may double it twice; relative L2 errors are held to 3.2e-2.
The step after that is fp32: the update p - p_old follows gradients that agree to 3.2e-2, and
from zero moments its size is lr in every element, so it is compared by its sign where the
gradient is not small.
"""
import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = torch.bfloat16


def linear(x, w, fn, shape, tokens, fin, fout):
    y = torch.empty(shape, dtype=BF, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    _lib.check(fn(x.data_ptr(), w.data_ptr(), y.data_ptr(), tokens, fin, fout, 0, s), "linear")
    return y


def test_a_training_step():
    B, T, H, Hkv, d, E, hidden = 2, 200, 4, 2, 64, 5, 136
    dm, n = H * d, B * T
    qkv_w = (H + 2 * Hkv) * d
    g = torch.Generator().manual_seed(31)

    def rnd(*shape, sigma=1.0, dtype=BF):
        return (torch.randn(shape, generator=g) * sigma).to(dtype).to(DEV)

    x, wqkv = rnd(n, dm), rnd(qkv_w, dm, sigma=dm ** -0.5)
    up, down = rnd(E, hidden, dm, sigma=dm ** -0.5), rnd(E, dm, hidden, sigma=hidden ** -0.5)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g)).to(DEV), (1 + 0.1 * torch.randn(d, generator=g)).to(DEV)
    freq = (10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    expert = torch.randint(0, E - 1, (n,), generator=g)  # the last expert gets no rows
    order = torch.argsort(expert, stable=True).to(DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(expert, minlength=E).cumsum(0)
    offsets = offsets.to(DEV)
    dout = rnd(n, dm)

    # forward
    proj = linear(x, wqkv, _lib.forge_linear_fwd, (n, qkv_w), n, dm, qkv_w).view(B, T, -1, d)
    xq, xk, xv = proj[:, :, :H], proj[:, :, H:H + Hkv], proj[:, :, H + Hkv:]
    rope = dict(inv_freq=freq, positions=pos)
    q, k, v = fa.qkv_fwd(xq, xk, xv, wq, wk, **rope)
    o, lse = fa.attn_fwd(q, k, v)
    rows = o.transpose(1, 2).reshape(n, dm)[order].contiguous()
    h = fa.linear_grouped_fwd(rows, up, offsets)
    y = fa.linear_grouped_fwd(h, down, offsets)
    # backward
    dy = dout[order].contiguous()
    dh = fa.linear_grouped_bwd_dx(dy, down, offsets)
    d_down = fa.linear_grouped_bwd_dw(dy, h, offsets)
    drows = fa.linear_grouped_bwd_dx(dh, up, offsets)
    d_up = fa.linear_grouped_bwd_dw(dh, rows, offsets)
    do = torch.empty_like(drows)
    do[order] = drows
    do = do.view(B, T, H, d).transpose(1, 2).contiguous()
    dq, dk, dv = fa.attn_bwd(q, k, v, o, do, lse, grad_dtype=torch.float32)
    dproj = torch.empty_like(proj)
    out = (dproj[:, :, :H], dproj[:, :, H:H + Hkv], dproj[:, :, H + Hkv:])
    *_, d_wq, d_wk = fa.qkv_bwd(dq, dk, dv, xq, xk, wq, wk, out=out, **rope)
    d_wqkv = torch.empty((qkv_w, dm), device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    _lib.check(_lib.forge_linear_bwd_dw(dproj.data_ptr(), x.data_ptr(), d_wqkv.data_ptr(), n, dm, qkv_w,
                                        1, 0, 0, s), "dw")
    dx = linear(dproj, wqkv, _lib.forge_linear_bwd_dx, (n, dm), n, dm, qkv_w)
    grads = [d_wqkv, d_up, d_down, d_wq, d_wk]
    before = [t.clone() for t in grads]
    norm = fa.grad_clip(grads, 1.0)
    masters = [t.float() for t in (wqkv, up, down, wq, wk)]
    old = [m.clone() for m in masters]
    mom = [[torch.zeros_like(m) for m in masters] for _ in range(2)]
    table = [(p.data_ptr(), gr.data_ptr(), m1.data_ptr(), m2.data_ptr(), p.numel(), int(p.dim() > 1))
             for p, gr, m1, m2 in zip(masters, grads, *mom)]
    ws = torch.empty(_lib.forge_adamw_workspace_size(5), dtype=torch.uint8, device=DEV)
    _lib.check(_lib.forge_adamw_step(table, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-12, weight_decay=0.0,
                                     step=1, max_norm=0.0, grad_norm_out=None, workspace=ws.data_ptr(),
                                     workspace_bytes=ws.numel(), stream=s), "adamw")
    fa.check_device_error()

    # the same in float64 by autograd
    X, WQKV, UP, DOWN, WQ, WK = (t.double().cpu().requires_grad_() for t in (x, wqkv, up, down, wq, wk))
    P = (X @ WQKV.T).view(B, T, -1, d)
    phi = pos.cpu().double()[..., None, None] * freq.cpu()

    def turned(a, w):
        a = a / (a.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a1, a2 = a[..., :d // 2], a[..., d // 2:]
        c, sn = phi.cos(), phi.sin()
        return torch.cat((a1 * c - a2 * sn, a1 * sn + a2 * c), -1).transpose(1, 2)

    Q = turned(P[:, :, :H], WQ)
    K = turned(P[:, :, H:H + Hkv], WK).repeat_interleave(H // Hkv, 1)
    V = P[:, :, H + Hkv:].transpose(1, 2).repeat_interleave(H // Hkv, 1)
    S = Q @ K.transpose(2, 3) * d ** -0.5
    S = S.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), float("-inf"))
    O = (S.softmax(-1) @ V).transpose(1, 2).reshape(n, dm)[order.cpu()]
    off = offsets.tolist()
    Y = torch.cat([O[a:b] @ UP[e].T @ DOWN[e].T for e, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    want = torch.autograd.grad(Y, (X, WQKV, UP, DOWN, WQ, WK), dout[order].double().cpu())

    def rel(a, b):
        b = b.detach()
        return float((a.double().cpu() - b).norm() / b.norm())

    errs = {"y": rel(y, Y), "dx": rel(dx, want[0])}
    errs.update({n_: rel(b, w) for n_, b, w in zip(("wqkv", "up", "down", "wq", "wk"), before, want[1:])})
    assert max(errs.values()) <= 3.2e-2, errs
    assert not before[1][E - 1].any() and not before[2][E - 1].any()
    full = np.sqrt(sum(float(w.square().sum()) for w in want[1:]))
    assert norm.item() == pytest.approx(full, rel=3.2e-2)
    assert fa.grad_norm(grads).item() == pytest.approx(1.0, rel=1e-5)
    for p, p0, w in zip(masters, old, want[1:]):
        sure = (w.abs() > 0.2 * w.abs().max()).to(DEV)
        assert torch.equal(torch.sign(p - p0)[sure], -torch.sign(w).float().to(DEV)[sure])
