"""The gradient norm and clipping (CUDA) against the fp64 oracle on the same values (GPU).

Tolerances, from the arithmetic (u = 2^-24): a thread sums at most 128 squares in fp32, each
addition and square off by at most u relative (all terms are positive): below 130 u on its
share, 65 u on the root, plus one rounding: the norm to 4e-6 relative.  A clipped value is
c (two roundings and the norm's error) times g, rounded to its type: eps / 2 + 5e-6 relative,
and half of the smallest subnormal where it is tiny.
"""
import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import _lib
from causal_attention_fwd_attn_b200 import workloads as wl
from oracle import grads as og

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
KINDS = (torch.float32, torch.bfloat16, torch.float16)


def make(sizes, kinds, seed, sigma=0.01):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * sigma).to(kinds[j % len(kinds)]).to(DEV)
            for j, n in enumerate(sizes)]


def f64(ts):
    return [t.double().cpu().numpy() for t in ts]


def check(grads, max_norm, in_place):
    norm, ref = og.grad_clip(f64(grads), max_norm)
    shown = norm if norm < float(np.finfo(np.float32).max) else float("inf")
    assert fa.grad_norm(grads).item() == pytest.approx(shown, rel=4e-6)
    if in_place:
        out = grads
        got = fa.grad_clip(grads, max_norm)
    else:
        out = [torch.full_like(t, 77.0) for t in grads]
        before = [t.clone() for t in grads]
        got = fa.grad_clip(grads, max_norm, out=out)
        assert all(torch.equal(a, b) for a, b in zip(before, grads))
    assert got.dtype == torch.float32 and got.shape == ()
    assert got.item() == pytest.approx(shown, rel=4e-6)
    for t, r in zip(out, ref):
        h = torch.finfo(t.dtype).eps / 2
        err = np.abs(t.double().cpu().numpy() - r)
        assert (err <= (h + 5e-6) * np.abs(r) + TINY[t.dtype]).all()


SETS = [[1], [3], [0, 5, 0], [8], [4095, 4096, 4097], [65536 + 7, 1, 30011], [300000, 9],
        [(k * 977) % 5000 for k in range(64)]]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kinds", [KINDS[:1], KINDS[1:2], KINDS[2:], KINDS])
@pytest.mark.parametrize("sizes", SETS)
def test_sets(sizes, kinds, in_place):
    for clipped in (True, False):
        grads = make(sizes, kinds, len(sizes) + sizes[0])
        full = og.grad_norm(f64(grads))
        check(grads, (0.3 if clipped else 3.0) * full + 1e-30, in_place)


def test_nothing_at_all():
    empty = [torch.zeros(0, device=DEV), torch.zeros((0, 5), dtype=torch.bfloat16, device=DEV)]
    assert fa.grad_norm(empty).item() == 0.0 and fa.grad_clip(empty, 1.0).item() == 0.0


def test_nothing_to_clip_leaves_every_bit():
    grads = make([70001, 13], KINDS, 3)
    before = [t.clone() for t in grads]
    out = [torch.zeros_like(t) for t in grads]
    fa.grad_clip(grads, 1e9, out=out)
    fa.grad_clip(grads, 1e9)
    for b, g, o in zip(before, grads, out):
        assert torch.equal(b, g) and torch.equal(b, o)


def test_more_tensors_than_one_launch_holds():
    n = _lib.ADAMW_MAX_TENSORS_PER_LAUNCH
    check(make([(37 * k) % 700 for k in range(2 * n + 5)], KINDS, 5), 0.2, False)
    check(make([(37 * k) % 700 for k in range(n + 1)], KINDS, 6), 0.2, True)


def test_gpt2_small_parameter_set():
    sizes = [int(np.prod(s)) for s in wl.gpt2small_param_shapes()]
    g = torch.Generator(device=DEV).manual_seed(7)
    grads = [torch.randn(n, generator=g, device=DEV) * 0.01 for n in sizes]
    check(grads, 1.0, True)


def test_squares_beyond_fp32s_range():
    for value, dtype in ((1e30, torch.float32), (3e-30, torch.float32), (1e-38, torch.bfloat16),
                         (2e37, torch.bfloat16)):
        grads = [torch.full((5000,), value, device=DEV).to(dtype), torch.zeros(70, device=DEV)]
        # 2e37 sqrt(5000) = 1.4e39 is past fp32's largest value: the norm shows as infinite,
        # the factor still comes from its 64-bit value; max_norm itself has to be finite
        check(grads, min(og.grad_norm(f64(grads)) * 0.5, 1e38), False)
    # small values beside large ones
    check([torch.full((5000,), 1e-30, device=DEV), torch.full((9,), 1e3, device=DEV)], 1.0, False)
    assert fa.grad_norm([torch.zeros(9000, device=DEV), -torch.zeros(9, device=DEV)]).item() == 0.0


@pytest.mark.parametrize("in_place", [False, True])
def test_factors_below_fp32s_normal_range(in_place):
    """max_norm / norm down to 1e-60 while the clipped values are ordinary: the factor keeps its
    bits (in fp32 it would be 0.05 % to 2 % off, or 0)."""
    for n, top, max_norm in ((5000, 3e38, 1e-3), (5000, 3e38, 1e-20), (70001, 3.3e38, 1e-2),
                             (40, 2e38, 1.0)):
        for kinds in (KINDS[:1], KINDS[1:2], KINDS):
            grads = [t.abs().add(0.1).mul(top / 10).to(t.dtype) if t.dtype != torch.float16 else t
                     for t in make([n, 333, 5], kinds, n, sigma=1.0)]
            assert all(torch.isfinite(t).all() for t in grads)
            check(grads, max_norm, in_place)


def test_values_that_are_not_finite():
    grads = make([5000, 300], KINDS, 9)
    grads[1][17] = float("inf")
    out = [torch.empty_like(t) for t in grads]
    assert fa.grad_clip(grads, 1.0, out=out).item() == float("inf")  # c = 0
    assert not out[0].any() and torch.isnan(out[1][17]) and int(torch.isnan(out[1]).sum()) == 1
    grads[0][4] = float("nan")
    assert torch.isnan(fa.grad_clip(grads, 1.0, out=out))  # c = 1
    assert torch.equal(out[0].nan_to_num(5.0), grads[0].nan_to_num(5.0))
    assert torch.isnan(fa.grad_norm(grads))


def test_results_repeat_on_another_stream_and_in_a_graph():
    grads = make([300001, 9, 4096], KINDS, 11)
    out, again = ([torch.empty_like(t) for t in grads] for _ in range(2))
    norm = fa.grad_clip(grads, 0.5, out=out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        norm2 = fa.grad_clip(grads, 0.5, out=again)
    side.synchronize()
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(out, again))
    # two graphs that share a workspace, replayed one after the other
    ws = torch.empty(fa.grad_workspace_bytes(3), dtype=torch.uint8, device=DEV)
    norms = [torch.zeros((), device=DEV) for _ in range(2)]
    graphs = []
    for j in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[j]):
            fa.grad_clip(grads, 0.5 + j, out=again, norm=norms[j], workspace=ws)
    for t in grads:
        t.mul_(1.5)
    for j in (0, 1, 0):
        graphs[j].replay()
    want = [torch.empty_like(t) for t in grads]
    norm = fa.grad_clip(grads, 0.5, out=want)
    torch.cuda.synchronize()
    assert torch.equal(norms[0], norm) and torch.equal(norms[1], norm)
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_matches_the_clip_inside_adamw():
    """forge_adamw_step's own factor and clipping first give the same step."""
    shapes = [(300, 70), (1000,), (65536 + 7,)]
    host = wl.make_adamw_inputs(shapes, 21)
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(_lib.forge_adamw_workspace_size(3), dtype=torch.uint8, device=DEV)
    res = []
    for first in (False, True):
        t = [{k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in host]
        if first:
            fa.grad_clip([x["grad"] for x in t], 0.5)
        table = [(x["param"].data_ptr(), x["grad"].data_ptr(), x["exp_avg"].data_ptr(),
                  x["exp_avg_sq"].data_ptr(), x["param"].numel(), int(x["decay"])) for x in t]
        _lib.check(_lib.forge_adamw_step(table, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8,
                                         weight_decay=0.1, step=3, max_norm=0.0 if first else 0.5,
                                         grad_norm_out=None, workspace=ws.data_ptr(),
                                         workspace_bytes=ws.numel(), stream=s), "adamw")
        res.append(t)
    for a, b in zip(*res):
        for n in ("param", "exp_avg", "exp_avg_sq"):
            assert torch.allclose(a[n], b[n], rtol=1e-5, atol=1e-6 * float(a[n].abs().max()))


def test_refusals():
    g = torch.zeros(9, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        fa.grad_clip([torch.zeros((4, 4), device=DEV).t()[:2]], 1.0)
    with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
        fa.grad_norm([g.double()])
    with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
        fa.grad_norm([g, g.cpu()])
    with pytest.raises(ValueError, match="outputs"):
        fa.grad_clip([g], 1.0, out=[g.half()])
    with pytest.raises(ValueError, match="1 gradients, 2 outputs"):
        fa.grad_clip([g], 1.0, out=[g, g])
    with pytest.raises(ValueError, match="twice"):
        fa.grad_clip([g, g], 1.0)
    with pytest.raises(fa.ForgeAttnError, match="invalid argument"):
        fa.grad_clip([g], 0.0)
    with pytest.raises(fa.ForgeAttnError, match="misaligned"):
        fa.grad_norm([g[1:]])
    with pytest.raises(fa.ForgeAttnError, match="workspace"):
        fa.grad_norm([g], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    # slices that overlap, in place and as outputs; neighbours do not
    whole, other = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="twice"):
        fa.grad_clip([whole[32:64], whole[:36]], 1.0)
    with pytest.raises(ValueError, match="twice"):
        fa.grad_clip([g[:8], whole[:8]], 1.0, out=[other[:8], other[4:12]])
    with pytest.raises(ValueError, match="read for another"):
        fa.grad_clip([whole[:16], whole[16:32]], 1.0, out=[other[:16], whole[8:24]])
    with pytest.raises(ValueError, match="read for another"):
        fa.grad_clip([whole[:16], whole[16:32]], 1.0, out=[whole[28:44], other[:16]])
    assert (whole == 1).all() and (other == 1).all()
    assert fa.grad_clip([whole[32:], whole[:32]], 4.0).item() == 8.0
    assert (whole == 0.5).all()
    assert fa.grad_clip([whole[:16], whole[16:32]], 4.0, out=[whole[:16], other[:16]]).item() < 4.0
    # any iterable of tensors is held until the launch
    grads, out = make([5000, 300], KINDS, 13), [torch.empty(5000, device=DEV), None]
    out[1] = torch.empty(300, dtype=KINDS[1], device=DEV)
    fa.grad_clip((t for t in grads), 0.1, out=(t for t in out))
    want = [t.clone() for t in grads]
    fa.grad_clip(want, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    # reading one tensor twice is a sum like any other
    one = torch.full((4,), 3.0, device=DEV)
    assert fa.grad_norm([one, one]).item() == pytest.approx(72 ** 0.5, rel=4e-6)
