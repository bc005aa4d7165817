"""The operators around the attention at sizes whose offsets pass 2^31 bytes, or 2^31 elements
where they may (GPU): values are compared at the ends and at random places between, with the
bounds of the operators' own tests."""
import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from oracle import linear as ol
from oracle import qkv as oq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 1e-6


def f64(t):
    return t.double().cpu().numpy()


def normal(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_qkv_stage_just_below_its_limit():
    """B T H d = 2^31 - 2^12.  The norm weight's gradient: a thread adds up at most 512 rows in
    fp32, 8 warps follow and the rest is in 64 bits: (4e-6 + 520 u) of the sum of magnitudes,
    bounded by 4e-5 of it."""
    T, H, d = 2 ** 19 - 1, 32, 128
    q, k, v = (normal((1, T, h, d), n, torch.bfloat16) for n, h in enumerate((H, 1, 1)))
    wq, wk = (1 + 0.3 * normal((d,), n, torch.float32) for n in (3, 4))
    freq = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).to(DEV)
    at = torch.tensor([0, 1, 2 ** 18 - 1, 2 ** 18, 400_001, T - 17, T - 2, T - 1], device=DEV)
    phi = f64(at)[None, :, None] * f64(freq)
    out = fa.qkv_fwd(q, k, v, wq, wk, eps=EPS, inv_freq=freq)
    for x, w, o, rep in ((q, wq, out[0], 1), (k, wk, out[1], H)):
        xs, os = f64(x[:, at]), f64(o[:, :, at])
        ref = oq.head_fwd(xs, f64(w), phi, False, EPS, rep)
        n = np.abs(xs / np.sqrt(np.mean(xs * xs, -1, keepdims=True) + EPS) * f64(w)).max(-1)
        slack = 4e-6 * np.repeat(np.swapaxes(n, 1, 2), rep, axis=1)[..., None]
        assert (np.abs(os - ref) <= 2.0 ** -8 * np.abs(ref) + slack).all()
    assert torch.equal(out[2], v.transpose(1, 2).expand(1, H, T, d))

    dq, dk, dv = (t.normal_() for t in out)  # (their room is needed)
    gq, gk, gv, gwq, gwk = fa.qkv_bwd(dq, dk, dv, q, k, wq, wk, eps=EPS, inv_freq=freq)
    for x, w, dy, gx, rep in ((q, wq, dq, gq, 1), (k, wk, dk, gk, H)):
        xs, dys = f64(x[:, at]), f64(dy[:, :, at])
        ref = oq.head_bwd(dys, xs, f64(w), phi, False, EPS, rep)[0]
        top = np.abs(dys).reshape(1, H // rep, rep, len(at), d).sum(2).max(-1, keepdims=True)
        u = 1.5 * np.swapaxes(top, 1, 2) * np.abs(f64(w)).max()
        r = 1 / np.sqrt(np.mean(xs * xs, -1, keepdims=True) + EPS)
        n = np.abs(xs * r)
        slack = 8e-6 * r * (u + n.max(-1, keepdims=True) * u * n.mean(-1, keepdims=True))
        assert (np.abs(f64(gx[:, at]) - ref) <= 2.0 ** -8 * np.abs(ref) + slack).all()
    ref = dv[:, :, at].double().sum(1, keepdim=True).transpose(1, 2)
    total = dv[:, :, at].double().abs().sum(1, keepdim=True).transpose(1, 2)
    assert ((gv[:, at].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 8e-6 * total).all()

    for x, dy, gw in ((q, dq, gwq), (k, dk, gwk)):
        want, sizes = torch.zeros(d, dtype=torch.float64, device=DEV), 0
        for t0 in range(0, T, 1 << 14):
            t = slice(t0, min(t0 + (1 << 14), T))
            turn = torch.arange(t.start, t.stop, device=DEV, dtype=torch.float64)[:, None] * freq
            g = dy[0, :, t].double()
            if x.shape[2] == 1:
                g = g.sum(0, keepdim=True)
            a, b = g[..., :d // 2], g[..., d // 2:]
            back = torch.cat([a * turn.cos() + b * turn.sin(), b * turn.cos() - a * turn.sin()], -1)
            n = x[0, t].double().transpose(0, 1)
            n = n / (n.square().mean(-1, keepdim=True) + EPS).sqrt()
            want += (back * n).sum((0, 1))
            sizes = sizes + (back * n).abs().sum((0, 1))
        assert ((gw.double() - want).abs() <= 4e-5 * sizes).all()


def test_qkv_strides_beyond_31_bits():
    """Two sequences 2^31 + 2^12 elements apart, and tokens 2^26 apart: the rows between are
    neither read nor written."""
    B, T, H, d = 2, 9, 2, 64
    far, step = 2 ** 31 + 2 ** 12, 2 ** 26
    store = torch.zeros(far + T * step, dtype=torch.bfloat16, device=DEV)
    x = store.as_strided((B, T, H, d), (far, step, d, 1))
    x.copy_(normal((B, T, H, d), 1, torch.bfloat16))
    near, w = x.clone(memory_format=torch.contiguous_format), 1 + 0.3 * normal((d,), 2, torch.float32)
    freq = torch.linspace(1, 0.01, d // 2, dtype=torch.float64, device=DEV)
    for a, b in zip(fa.qkv_fwd(x, x, x, w, w, inv_freq=freq), fa.qkv_fwd(near, near, near, w, w, inv_freq=freq)):
        assert torch.equal(a, b)
    dy = normal((B, H, T, d), 3, torch.bfloat16)
    gaps = torch.zeros(far + T * step, dtype=torch.bfloat16, device=DEV)
    out = [gaps[n * 4096:].as_strided((B, T, H, d), (far, step, d, 1)) for n in range(3)]
    got = fa.qkv_bwd(dy, dy, dy, x, x, w, w, inv_freq=freq, out=tuple(out))
    ref = fa.qkv_bwd(dy, dy, dy, near, near, w, w, inv_freq=freq)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert torch.count_nonzero(gaps) == sum(int(torch.count_nonzero(t)) for t in ref[:3])


def test_grouped_products_just_below_their_limit():
    """rows * features = 2^31 - 2^10; the long expert's weight gradient sums 2 million rows."""
    fin, fout = 1024, 72
    counts = [2 ** 21 - 1 - 300, 0, 131, 169]
    rows = sum(counts)
    o = [0] + np.cumsum(counts).tolist()
    off = torch.tensor(o, dtype=torch.int32, device=DEV)
    x, dy = normal((rows, fin), 1, torch.bfloat16), normal((rows, fout), 2, torch.bfloat16)
    w = normal((4, fout, fin), 3, torch.bfloat16)
    at = torch.cat([torch.arange(0, 70), torch.arange(rows // 2 - 40, rows // 2 + 40),
                    torch.arange(rows - 400, rows)])
    owner = np.searchsorted(np.asarray(o[1:]), at.numpy(), side="right")
    ends = [0] + [int((owner <= e).sum()) for e in range(4)]  # the experts' rows among these
    xs, dys, ws = f64(x[at.to(DEV)]), f64(dy[at.to(DEV)]), f64(w)
    for got, ref, size, K in (
            (fa.linear_grouped_fwd(x, w, off), ol.grouped_fwd(xs, ws, ends),
             ol.grouped_fwd(abs(xs), abs(ws), ends), fin),
            (fa.linear_grouped_bwd_dx(dy, w, off), ol.grouped_bwd_dx(dys, ws, ends),
             ol.grouped_bwd_dx(abs(dys), abs(ws), ends), fout)):
        err = np.abs(f64(got[at.to(DEV)]) - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -23 * (K / 16 + 2) * size).all()
    dw = fa.linear_grouped_bwd_dw(dy, x, off)
    fa.check_device_error()
    for e, n in enumerate(counts):
        ref = torch.zeros((fout, fin), dtype=torch.float64, device=DEV)
        size = torch.zeros_like(ref)
        for r in range(o[e], o[e + 1], 1 << 17):
            r = slice(r, min(r + (1 << 17), o[e + 1]))
            a, b = dy[r].double(), x[r].double()
            ref += a.t() @ b
            size += a.abs().t() @ b.abs()
        # chunks of 512 rows in the tensor core, their sums added one after the other
        bound = 2.0 ** -24 * ref.abs() + 2.0 ** -23 * (512 / 16 + 2 + n / 512) * size
        assert ((dw[e].double() - ref).abs() <= bound).all()


def test_the_longest_reduction_there_may_be():
    """One expert with 2^28 - 1 rows, the last 63 of them a tail, behind which nothing is left to
    do: 4 million k-blocks on one pair of SMs.  Partial sums of n chunks grow like sqrt(k) and are
    rounded to nearest: u sqrt(n / 6) = 1.8e-5 relative, beside 1.3e-6 within the chunks; four
    times their sum bounds the norm of 64 such errors."""
    rows, f = 2 ** 28 - 1, 8
    x, dy = normal((rows, f), 1, torch.bfloat16), normal((rows, f), 2, torch.bfloat16)
    off = torch.tensor([0, 0, rows], dtype=torch.int32, device=DEV)
    dw = fa.linear_grouped_bwd_dw(dy, x, off)
    fa.check_device_error()
    ref = torch.zeros((f, f), dtype=torch.float64, device=DEV)
    for r in range(0, rows, 1 << 23):
        ref += dy[r:r + (1 << 23)].double().t() @ x[r:r + (1 << 23)].double()
    assert not dw[0].any()
    assert (dw[1].double() - ref).norm() <= 8e-5 * ref.norm()


def test_a_gradient_of_more_than_2_31_values():
    n = 2 ** 31 + 12345
    big, small = torch.full((n,), 0.25, dtype=torch.float16, device=DEV), torch.ones(7, device=DEV)
    big[-1] = 16.0
    norm = (0.0625 * (n - 1) + 256.0 + 7.0) ** 0.5
    got = fa.grad_clip([big, small], norm / 2)
    assert abs(got.item() - norm) <= 4e-6 * norm
    assert (small == 0.5).all() and big[-1] == 8.0 and big[0] == 0.125
    assert torch.all(big[:-1] == 0.125)
