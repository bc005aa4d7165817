"""The stage between the QKV projection and the attention (CUDA) against the fp64 oracle on
the same inputs (GPU).

Tolerances, from the arithmetic (u = 2^-24, the half step of fp32; h = eps / 2 of the output's
type, its half step):
  forward   norm: the sum of d squares, rsqrtf (2 ulp) and two products: below 16 u relative;
            angles: at most 2^-24 turns in 64 bits, one rounding to fp32 and sincospif (2 ulp):
            below 16 u absolute; rotation: three roundings.  So before the last rounding the
            error is below 40 u = 2.4e-6 of the two members' magnitudes; the bound is
            h |ref| + 4e-6 max|n w| over the head (fp16: + 2^-25, its subnormal half step).
  backward  the same for the rotated gradients summed over the shared heads (8 more
            roundings); dx = r (u - n m) subtracts two such terms: the bound is
            h |ref| + 8e-6 r (max|u| + max|n| |m|).
  weights   fp32 sums of a thread's rows (at most 64 in these sizes) and of 8 warps, the rest in
            64 bits: 4e-6 + 72 u of the sum of magnitudes, bounded by 1e-5 of it.
"""
import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import _lib
from oracle import qkv as oq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 1e-6


def project(g, B, T, H, Hkv, d, dtype, layout):
    """q, k, v views [B, T, heads, d] in one of the layouts a projection may have."""
    if layout == "packed":
        x = torch.randn((B, T, H + 2 * Hkv, d), generator=g).to(dtype).to(DEV)
        return x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    if layout == "per_head":  # [B, T, heads, 3, d], equal heads
        x = torch.randn((B, T, H, 3, d), generator=g).to(dtype).to(DEV)
        return x[:, :, :, 0], x[:, :, :, 1], x[:, :, :, 2]
    if layout == "heads_first":  # [B, heads, T, d] seen as [B, T, heads, d]
        return tuple(torch.randn((B, h, T, d), generator=g).to(dtype).to(DEV).transpose(1, 2)
                     for h in (H, Hkv, Hkv))
    if layout == "one_batch":  # the same rows for every sequence (stride 0)
        return tuple(torch.randn((1, T, h, d), generator=g).to(dtype).to(DEV).expand(B, T, h, d)
                     for h in (H, Hkv, Hkv))
    return tuple(torch.randn((B, T, h, d), generator=g).to(dtype).to(DEV) for h in (H, Hkv, Hkv))


def rope_of(g, B, T, d, rot, axes, adjacent, far):
    if rot == 0:
        return {}, None
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    kw = dict(inv_freq=freq.to(DEV), adjacent=adjacent)
    if axes == 0:  # the token's index
        return kw, oq.angles(freq.numpy(), None, None, B, T)
    pos = torch.randint(-2 ** 31 if far else -99, 2 ** 31 - 1 if far else 999, (axes, B, T), generator=g,
                        dtype=torch.int64).to(torch.int32)
    axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.int32)
    kw.update(positions=pos.to(DEV), pair_axis=axis.to(DEV))
    return kw, oq.angles(freq.numpy(), pos.numpy(), axis.numpy(), B, T)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def bound_head(x, w, dtype, eps=EPS):
    """Largest |n w| of each head, [B, T, heads, 1]."""
    x = f64(x)
    n = x if w is None else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * f64(w)
    return np.max(np.abs(n), -1, keepdims=True)


def within(got, ref, slack, dtype, what):
    h = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = np.abs(f64(got) - ref)
    excess = err - (h * np.abs(ref) + slack + tiny)
    assert np.isfinite(f64(got)).all(), f"{what}: non-finite"
    assert excess.max() <= 0, f"{what}: off by {err.max():.3e}, {excess.max():.3e} too much"


CASES = [
    # B, T, H, Hkv, d, rot, axes, dtype, adjacent, layout, normed, far
    (1, 1, 1, 1, 64, 64, 1, torch.bfloat16, False, "packed", True, False),
    (1, 1, 32, 8, 128, 128, 1, torch.bfloat16, False, "packed", True, True),
    (5, 1, 12, 4, 64, 64, 1, torch.float16, True, "packed", True, True),
    (2, 130, 6, 2, 64, 64, 0, torch.bfloat16, False, "packed", True, False),
    (3, 77, 5, 5, 128, 128, 3, torch.float16, False, "per_head", True, True),
    (2, 33, 17, 1, 128, 64, 2, torch.bfloat16, False, "heads_first", True, False),
    (4, 19, 3, 3, 64, 16, 2, torch.bfloat16, False, "one_batch", True, False),
    (1, 200, 8, 8, 128, 14, 2, torch.float16, True, "own", True, False),
    (2, 40, 16, 2, 64, 0, 1, torch.bfloat16, False, "packed", True, False),
    (2, 41, 4, 4, 128, 128, 1, torch.bfloat16, True, "packed", False, True),
    (1, 9, 40, 20, 64, 0, 1, torch.float16, False, "packed", False, False),
    (1, 1023, 12, 4, 64, 32, 2, torch.bfloat16, False, "own", True, False),
]


def make(case, seed):
    B, T, H, Hkv, d, rot, axes, dtype, adjacent, layout, normed, far = case
    g = torch.Generator().manual_seed(seed)
    q, k, v = project(g, B, T, H, Hkv, d, dtype, layout)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(DEV) if normed else None for _ in range(2))
    kw, phi = rope_of(g, B, T, d, rot, axes, adjacent, far)
    return g, q, k, v, wq, wk, kw, phi


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    B, T, H, Hkv, d, dtype, adjacent = *case[:5], case[7], case[8]
    _, q, k, v, wq, wk, kw, phi = make(case, 7)
    got = fa.qkv_fwd(q, k, v, wq, wk, eps=EPS, **kw)
    for name, x, w, o, turn in (("q", q, wq, got[0], phi), ("k", k, wk, got[1], phi),
                                ("v", v, None, got[2], None)):
        rep = H // x.shape[2]
        ref = oq.head_fwd(f64(x), f64(w), turn, adjacent, EPS, rep)
        assert o.shape == (B, H, T, d) and o.dtype == dtype
        if name == "v":
            assert np.array_equal(f64(o), ref)  # moved, not computed
            continue
        slack = 4e-6 * np.repeat(np.swapaxes(bound_head(x, w, dtype), 1, 2), rep, axis=1)
        within(o, ref, slack, dtype, f"{name} {case}")


@pytest.mark.parametrize("grad32", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, grad32):
    B, T, H, Hkv, d, dtype, adjacent, layout = *case[:5], *case[7:10]
    g, q, k, v, wq, wk, kw, phi = make(case, 11)
    grads = [torch.randn((B, H, T, d), generator=g).to(torch.float32 if grad32 else dtype).to(DEV)
             for _ in range(3)]
    out = None
    if layout == "heads_first":
        out = tuple(torch.empty_like(t) for t in (q, k, v))
    gq, gk, gv, gwq, gwk = fa.qkv_bwd(*grads, q, k, wq, wk, eps=EPS, out=out, **kw)
    for name, x, w, dy, gx, gw, turn in (("q", q, wq, grads[0], gq, gwq, phi),
                                         ("k", k, wk, grads[1], gk, gwk, phi),
                                         ("v", v, None, grads[2], gv, None, None)):
        rep = H // x.shape[2]
        ref, ref_w = oq.head_bwd(f64(dy), f64(x), f64(w), turn, adjacent, EPS, rep)
        dy_sum = np.abs(f64(dy)).reshape(B, H // rep, rep, T, d).sum(2).max(-1, keepdims=True)
        dy_max = 1.5 * np.swapaxes(dy_sum, 1, 2)  # a rotation's rows add up to sqrt(2) at most
        assert gx.shape == x.shape and gx.dtype == dtype
        if w is None:
            assert gw is None
            within(gx, ref, 8e-6 * dy_max, dtype, f"{name} {case}")
            continue
        xd, wd = f64(x), f64(w)
        r = 1 / np.sqrt(np.mean(xd * xd, -1, keepdims=True) + EPS)
        n = xd * r
        u_max = dy_max * np.abs(wd).max()
        m = u_max * np.mean(np.abs(n), -1, keepdims=True)
        within(gx, ref, 8e-6 * r * (u_max + np.abs(n).max(-1, keepdims=True) * m), dtype,
               f"{name} {case}")
        total = (dy_max * np.abs(n)).sum((0, 1, 2))
        err = np.abs(f64(gw) - ref_w)
        assert (err <= 1e-5 * total).all(), f"{name} weight {case}: {np.max(err / total):.2e}"


def test_gradients_against_differences():
    """The kernel's gradients along random directions against central differences of the fp64
    forward: |sum grad * dir - difference| within the gradients' rounding (h sum |grad dir|)
    and the difference's own error (1e-6 of it, step 1e-4)."""
    case = (2, 21, 4, 2, 64, 64, 2, torch.bfloat16, False, "packed", True, False)
    g, q, k, v, wq, wk, kw, phi = make(case, 13)
    grads = [torch.randn((2, 4, 21, 64), generator=g).to(DEV) for _ in range(3)]
    gq, gk, _, gwq, gwk = fa.qkv_bwd(*grads, q, k, wq, wk, eps=EPS, **kw)
    r = np.random.default_rng(3)
    for x, w, dy, gx, gw, rep in ((q, wq, grads[0], gq, gwq, 1), (k, wk, grads[1], gk, gwk, 2)):
        xd, wd, dyd = f64(x), f64(w), f64(dy)
        dx, dw = r.normal(size=xd.shape), r.normal(size=wd.shape)

        def loss(s):
            return float(np.sum(dyd * oq.head_fwd(xd + s * dx, wd + s * dw, phi, False, EPS, rep)))

        num = (loss(1e-4) - loss(-1e-4)) / 2e-4
        terms = np.concatenate([(f64(gx) * dx).ravel(), (f64(gw) * dw).ravel()])
        tol = 2.0 ** -8 * np.abs(f64(gx) * dx).sum() ** 0.5 * np.abs(f64(gx) * dx).max() ** 0.5 * 8
        assert abs(terms.sum() - num) <= tol + 1e-6 * np.abs(terms).sum()


def test_far_positions_keep_their_phase():
    """At positions near 2^31 a 32-bit angle would be off by tens of radians."""
    d = 64
    x = torch.zeros((1, 3, 1, d), dtype=torch.float16, device=DEV)
    x[..., 0] = 1.0
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 12345679]], dtype=torch.int32, device=DEV)
    freq = torch.full((32,), 0.7391, dtype=torch.float64, device=DEV)
    q, _, _ = fa.qkv_fwd(x, x, x, inv_freq=freq, positions=pos)
    phi = pos.cpu().double().numpy()[0] * 0.7391
    np.testing.assert_allclose(f64(q)[0, 0, :, 0], np.cos(phi), atol=2.0 ** -11 + 1e-6)
    np.testing.assert_allclose(f64(q)[0, 0, :, 32], np.sin(phi), atol=2.0 ** -11 + 1e-6)


def test_values_that_are_not_finite_stay_in_their_place():
    d = 64
    x = torch.ones((1, 9, 2, d), dtype=torch.bfloat16, device=DEV)
    x[0, 4, 0, 50] = float("inf")  # past the rotated elements
    x[0, 5, 1, 3] = float("nan")
    freq = torch.full((8,), 0.1, dtype=torch.float64, device=DEV)
    q, k, v = fa.qkv_fwd(x, x, x, inv_freq=freq)
    bad = ~torch.isfinite(q)
    want = torch.zeros_like(bad)
    want[0, 0, 4, 50] = True
    want[0, 1, 5, [3, 11]] = True  # a rotated pair shares a NaN
    assert torch.equal(bad, want) and torch.equal(bad, ~torch.isfinite(k))
    assert torch.equal(torch.isfinite(v), torch.isfinite(x.transpose(1, 2)))
    # zero heads: the norm is finite, their gradient too
    z = torch.zeros((1, 9, 2, d), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(d, device=DEV)
    assert not fa.qkv_fwd(z, z, z, w, w)[0].any()
    g = torch.ones((1, 2, 9, d), device=DEV)
    for t in fa.qkv_bwd(g, g, g, z, z, w, w):
        assert torch.isfinite(t).all()


def test_a_norm_without_eps_beside_rows_that_are_not_there():
    """Tokens past the last and heads past the last must not enter the weights' gradients."""
    B, T, H, d = 1, 19, 3, 64
    x = torch.randn((B, T, H, d), device=DEV).to(torch.bfloat16)
    g = torch.randn((B, H, T, d), device=DEV)
    w = torch.ones(d, device=DEV)
    gq, gk, gv, gwq, gwk = fa.qkv_bwd(g, g, g, x, x, w, w, eps=0.0)
    ref, ref_w = oq.head_bwd(f64(g), f64(x), f64(w), None, False, 0.0)
    total = np.abs(f64(g)).sum((0, 1, 2)) * 4
    assert (np.abs(f64(gwq) - ref_w) <= 1e-5 * total).all() and torch.equal(gwq, gwk)
    assert torch.isfinite(gq).all() and torch.equal(gq, gk)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("grad32", [False, True])
def test_what_shared_memory_held_before_does_not_matter(d, adjacent, grad32):
    """Calls whose rows, weights and angles are NaN leave NaN in every SM's shared memory; the
    tokens that a later call's last tile lacks must not bring them into its sums."""
    bad = torch.full((1, 6000, 4, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    wbad = torch.full((d,), float("nan"), device=DEV)
    fbad = torch.full((d // 2,), float("nan"), dtype=torch.float64, device=DEV)
    gbad = torch.full((1, 4, 6000, d), float("nan"), device=DEV)
    x = torch.randn((1, 3, 3, d), device=DEV).to(torch.bfloat16)
    g = torch.randn((1, 3, 3, d), device=DEV).to(torch.float32 if grad32 else torch.bfloat16)
    w = torch.ones(d, device=DEV)
    f = torch.rand(d // 2, dtype=torch.float64, device=DEV)
    ref, ref_w = oq.head_bwd(f64(g), f64(x), f64(w), oq.angles(f64(f), None, None, 1, 3), adjacent, EPS)
    for _ in range(3):
        fa.qkv_fwd(bad, bad, bad, wbad, wbad, inv_freq=fbad, adjacent=adjacent)
        fa.qkv_bwd(gbad, gbad, gbad, bad, bad, wbad, wbad, inv_freq=fbad, adjacent=adjacent)
        gq, gk, gv, gwq, gwk = fa.qkv_bwd(g, g, g, x, x, w, w, inv_freq=f, adjacent=adjacent)
        q, _, _ = fa.qkv_fwd(x, x, x, w, w, inv_freq=f, adjacent=adjacent)
        assert all(torch.isfinite(t).all() for t in (gq, gk, gv, gwq, gwk, q))
        total = 4 * np.abs(f64(g)).sum((0, 1, 2))
        assert (np.abs(f64(gwq) - ref_w) <= 1e-5 * total.max()).all()


@pytest.mark.parametrize("H,Hkv,d,rot,adjacent,dtype", [
    (1, 1, 64, 64, False, torch.bfloat16), (2, 1, 64, 32, False, torch.float16),
    (3, 3, 128, 128, False, torch.bfloat16), (4, 1, 128, 54, True, torch.bfloat16),
    (5, 5, 64, 64, True, torch.float16), (16, 2, 128, 128, False, torch.float16),
    (17, 1, 64, 64, False, torch.bfloat16), (8, 4, 64, 0, False, torch.bfloat16)])
def test_few_heads_of_many_tokens(H, Hkv, d, rot, adjacent, dtype):
    """Token tiles whose heads one block takes whole, and a list just too long for that: the same bits
    as a call on each sequence, and within the bounds at a sequence's first and last tokens."""
    B, T = 8, 4099
    g, q, k, v, wq, wk, kw, phi = make((B, T, H, Hkv, d, rot, 2 if rot else 0, dtype, adjacent, "packed",
                                        True, True), 23)
    n, few = 70, {name: kw[name] for name in kw if name != "positions"}
    for weights in ((wq, wk), (None, wk), (wq, None)):
        got = fa.qkv_fwd(q, k, v, *weights, eps=EPS, **kw)
        for b in range(B):
            if rot:
                few["positions"] = kw["positions"][:, b:b + 1].contiguous()
            own = fa.qkv_fwd(q[b:b + 1], k[b:b + 1], v[b:b + 1], *weights, eps=EPS, **few)
            assert all(torch.equal(x[b:b + 1], y) for x, y in zip(got, own)), b
        for part in (slice(0, n), slice(T - n, T)):
            turn = None if phi is None else phi[B - 1:, part]
            for x, w, o, a in ((q, weights[0], got[0], turn), (k, weights[1], got[1], turn),
                               (v, None, got[2], None)):
                x, o = x[B - 1:, part], o[B - 1:, :, part]
                rep = H // x.shape[2]
                ref = oq.head_fwd(f64(x), f64(w), a, adjacent, EPS, rep)
                slack = 4e-6 * np.repeat(np.swapaxes(bound_head(x, w, dtype), 1, 2), rep, axis=1)
                within(o, ref, slack, dtype, f"{H} {Hkv} {d}")


def test_pair_axes_out_of_range_count_as_the_nearest():
    x = torch.randn((1, 5, 1, 64), device=DEV).to(torch.bfloat16)
    freq = torch.rand(32, dtype=torch.float64, device=DEV)
    pos = torch.randint(0, 99, (2, 1, 5), dtype=torch.int32, device=DEV)
    wild = torch.tensor([-7, 0, 1, 900] * 8, dtype=torch.int32, device=DEV)
    a = fa.qkv_fwd(x, x, x, inv_freq=freq, positions=pos, pair_axis=wild)
    b = fa.qkv_fwd(x, x, x, inv_freq=freq, positions=pos, pair_axis=wild.clamp(0, 1))
    assert torch.equal(a[0], b[0])


def test_weight_gradients_accumulate_and_repeat():
    case = CASES[3]
    g, q, k, v, wq, wk, kw, _ = make(case, 17)
    grads = [torch.randn((2, 6, 130, 64), generator=g).to(DEV) for _ in range(3)]
    first = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    again = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(first, again))  # no atomics
    acc = (first[3].clone(), first[4].clone())
    fa.qkv_bwd(*grads, q, k, wq, wk, weight_out=acc, accumulate=True, **kw)
    for a, f in zip(acc, first[3:]):
        assert torch.allclose(a, 2 * f, rtol=2.0 ** -23, atol=0)
    with pytest.raises(ValueError, match="accumulate"):
        fa.qkv_bwd(*grads, q, k, wq, wk, accumulate=True, **kw)


def test_weights_of_queries_only():
    case = CASES[3]
    g, q, k, v, wq, _, kw, phi = make(case, 19)
    got = fa.qkv_fwd(q, k, v, wq, None, eps=EPS, **kw)
    ref = oq.head_fwd(f64(k), None, phi, False, EPS, 3)
    within(got[1], ref, 4e-6 * np.abs(ref).max(), torch.bfloat16, "k without norm")
    grads = [torch.randn((2, 6, 130, 64), generator=g).to(DEV) for _ in range(3)]
    *_, gwq, gwk = fa.qkv_bwd(*grads, q, k, wq, None, eps=EPS, **kw)
    assert gwk is None
    ref_w = oq.head_bwd(f64(grads[0]), f64(q), f64(wq), phi, False, EPS)[1]
    assert np.abs(f64(gwq) - ref_w).max() <= 1e-5 * np.abs(f64(grads[0])).sum()


def test_another_stream_and_a_captured_graph():
    case = CASES[4]
    g, q, k, v, wq, wk, kw, _ = make(case, 23)
    want = fa.qkv_fwd(q, k, v, wq, wk, **kw)
    grads = [torch.randn(t.shape, generator=g).to(DEV) for t in want]
    want_b = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fa.qkv_fwd(q, k, v, wq, wk, **kw)
        got_b = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *want_b), (*got, *got_b)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qkv_fwd(q, k, v, wq, wk, **kw)
        got_b = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    q.copy_(torch.randn(q.shape, generator=g).to(q.dtype))
    graph.replay()
    torch.cuda.synchronize()
    want = (*fa.qkv_fwd(q, k, v, wq, wk, **kw), *fa.qkv_bwd(*grads, q, k, wq, wk, **kw))
    assert all(torch.equal(a, b) for a, b in zip(want, (*got, *got_b)))


def test_parts_may_be_left_out():
    """The C ABI on queries alone, and on values alone."""
    B, T, H, d = 2, 7, 3, 64
    x = torch.randn((B, T, H, d), device=DEV).to(torch.bfloat16)
    y = torch.empty((B, H, T, d), dtype=torch.bfloat16, device=DEV)
    cfg = _lib.QkvConfig(B, T, H, H, d, 0, 1, 1e-6, None, None, None, None, None)
    tx = _lib.QkvTensor(x.data_ptr(), *x.stride()[:3])
    s = torch.cuda.current_stream().cuda_stream
    for args in ((tx, None, None, y.data_ptr(), None, None),
                 (None, None, tx, None, None, y.data_ptr())):
        y.zero_()
        assert _lib.forge_qkv_fwd(cfg, *args, 0, s) == _lib.OK
        assert torch.equal(y, x.transpose(1, 2))
    back = torch.zeros_like(x)
    tb = _lib.QkvTensor(back.data_ptr(), *back.stride()[:3])
    assert _lib.forge_qkv_bwd(cfg, None, None, y.data_ptr(), None, None, None, None, tb, None, None, 0,
                              None, 0, 0, s) == _lib.OK
    assert torch.equal(back, x)


def test_parts_of_few_heads_may_be_left_out():
    B, T, H, Hkv, d = 8, 4099, 3, 1, 64
    _, q, k, v, wq, wk, kw, _ = make((B, T, H, Hkv, d, d, 1, torch.bfloat16, False, "packed", True, True), 29)
    want = fa.qkv_fwd(q, k, v, wq, wk, eps=EPS, **kw)
    cfg = _lib.QkvConfig(B, T, H, Hkv, d, d, 1, EPS, kw["inv_freq"].data_ptr(), kw["positions"].data_ptr(),
                         kw["pair_axis"].data_ptr(), wq.data_ptr(), wk.data_ptr())
    ins = [_lib.QkvTensor(x.data_ptr(), *x.stride()[:3]) for x in (q, k, v)]
    for keep in range(1, 8):
        outs = [torch.full_like(o, -7.0) for o in want]
        on = [keep >> j & 1 for j in range(3)]
        assert _lib.forge_qkv_fwd(cfg, *(t if f else None for t, f in zip(ins, on)),
                                  *(o.data_ptr() if f else None for o, f in zip(outs, on)), 0,
                                  torch.cuda.current_stream().cuda_stream) == _lib.OK
        for o, w, f in zip(outs, want, on):
            assert torch.equal(o, w) if f else (o == -7).all(), keep


def test_one_graph_beside_eager_calls_of_the_same_tensors():
    """A captured backward shares nothing with eager calls: they may alternate."""
    case = CASES[3]
    g, q, k, v, wq, wk, kw, _ = make(case, 29)
    grads = [torch.randn((2, 6, 130, 64), generator=g).to(DEV) for _ in range(3)]
    want = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
    for _ in range(3):
        graph.replay()
        eager = fa.qkv_bwd(*grads, q, k, wq, wk, **kw)
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, eager):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_more_units_than_partial_sums():
    """Enough tokens that the backward's blocks take several units each."""
    B, T, H, d = 1, 40000, 1, 64
    x = torch.randn((B, T, H, d), device=DEV).to(torch.bfloat16)
    g = torch.randn((B, H, T, d), device=DEV)
    w = torch.ones(d, device=DEV)
    gq, _, _, gw, _ = fa.qkv_bwd(g, g, g, x, x, w, w, eps=EPS)
    ref, ref_w = oq.head_bwd(f64(g), f64(x), f64(w), None, False, EPS)
    bound = 1e-5 * np.abs(f64(g).transpose(0, 2, 1, 3) * f64(x)).sum((0, 1, 2)) * 1.5
    assert (np.abs(f64(gw) - ref_w) <= bound).all()
    assert np.abs(f64(gq) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4


def test_front_end_refusals_on_cuda_tensors():
    x = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device=DEV)
    freq = torch.ones(32, dtype=torch.float64, device=DEV)
    bad = [
        (dict(k=x.half()), "dtype"), (dict(v=x[:, :2]), "shape"),
        (dict(k=x[:, :, :3], v=x[:, :, :3]), "invalid argument"),   # 4 heads over 3
        (dict(q=x.transpose(2, 3)[..., :4, :], k=x, v=x), None),
        (dict(inv_freq=freq.float()), "dtype"), (dict(inv_freq=freq[:20]), "unsupported"),
        (dict(inv_freq=freq, positions=torch.zeros((2, 3), device=DEV)), "dtype"),
        (dict(inv_freq=freq, positions=torch.zeros((3, 2), dtype=torch.int32, device=DEV)), "shape"),
        (dict(positions=torch.zeros((2, 3), dtype=torch.int32, device=DEV)), "inv_freq"),
        (dict(q_weight=torch.ones(64, device=DEV).half()), "dtype"),
        (dict(q_weight=torch.ones(32, device=DEV)), "shape"),
        (dict(out=(x, x)), "out"), (dict(out=(x, x, x)), "shape"),
    ]
    for change, msg in bad:
        args = dict(q=x, k=x, v=x)
        args.update(change)
        with pytest.raises((ValueError, fa.ForgeAttnError), match=msg):
            fa.qkv_fwd(args.pop("q"), args.pop("k"), args.pop("v"), **args)
    odd = torch.zeros(2 * 3 * 4 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 3, 4, 64)
    with pytest.raises(fa.ForgeAttnError, match="misaligned"):
        fa.qkv_fwd(odd, odd, odd)


def test_overlapping_outputs_are_refused():
    """What two parts of the kernel would both write: one of the results would be lost."""
    B, T, H, d = 1, 70, 2, 64
    x = torch.randn((B, T, H, d), device=DEV).to(torch.bfloat16)
    w = torch.ones(d, device=DEV)
    room = torch.zeros(4 * B * H * T * d, dtype=torch.bfloat16, device=DEV)
    n = B * H * T * d
    o = [room[j * n:(j + 1) * n].view(B, H, T, d) for j in range(3)]
    late = room[2 * n - 8:3 * n - 8].view(B, H, T, d)
    for out in ((o[0], o[0], o[2]), (o[0], o[1], o[0]), (o[0], o[1], late)):
        with pytest.raises(fa.ForgeAttnError, match="invalid argument"):
            fa.qkv_fwd(x, x, x, w, w, out=out)
    assert not room.any()
    want = fa.qkv_fwd(x, x, x, w, w)
    assert all(torch.equal(a, b) for a, b in zip(want, fa.qkv_fwd(x, x, x, w, w, out=tuple(o))))
    g = torch.randn((B, H, T, d), device=DEV)
    both = torch.zeros(2 * d, device=DEV)
    for dq, dk in ((both[:d], both[:d]), (both[:d], both[4:d + 4])):
        with pytest.raises(fa.ForgeAttnError, match="invalid argument"):
            fa.qkv_bwd(g, g, g, x, x, w, w, weight_out=(dq, dk), accumulate=True)
    assert not both.any()
    *_, gq, gk = fa.qkv_bwd(g, g, g, x, x, w, w, weight_out=(both[:d], both[d:]), accumulate=True)
    assert torch.equal(gq, gk) and gq.any()
