"""The linear products grouped by expert (tcgen05) against the fp64 oracle on the same
inputs (GPU), over whole outputs.

Tolerances, from the arithmetic: products of 16-bit values are exact in fp32, and a tensor
core adds 16 of them to its accumulator at a time, aligned to the largest and cut off, so each
addition is off by at most 2^-23 of the magnitudes added so far.  K terms take K / 16 + 1 of
them and the last rounding (or the addition to earlier gradients) one more:
  |gpu - ref| <= h |ref| + 2^-23 (K / 16 + 2) sum |a b|
with h the half step of the output (2^-8 bf16, 2^-11 fp16, 2^-24 fp32).  Over a whole fp32
output, whose errors are not all of one sign, the relative L2 error stays below 2e-5.
"""
import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import workloads as wl
from oracle import linear as ol

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def gen(shape, seed, dtype=torch.bfloat16):
    return wl.gaussian_bf16(shape, 1.0, seed, dtype)


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32)


def within(got, ref, K, terms, what):
    """K: length of the sums; terms: the sums of the magnitudes."""
    g = got.double().cpu().numpy()
    if g.size == 0:
        return
    assert np.isfinite(g).all(), what
    err = np.abs(g - ref)
    excess = err - (HALF[got.dtype] * np.abs(ref) + 2.0 ** -23 * (np.asarray(K) / 16 + 2) * terms)
    assert excess.max() <= 0, f"{what}: off by {err.max():.3e}, {excess.max():.3e} too much"
    if got.dtype == torch.float32:
        assert np.linalg.norm(g - ref) <= 2e-5 * np.linalg.norm(ref), what


def run(counts, fin, fout, seed, dtype=torch.bfloat16, out_f32=False, first=0, spare=0,
        poison=False, what=("y", "dx", "dw", "dw+")):
    """All products over experts with `counts` rows; `first` and `spare` rows before and after
    them belong to nobody (poison: they hold infinities and NaN)."""
    E, rows = len(counts), first + int(sum(counts)) + spare
    off = offsets_of(counts, first)
    o = off.tolist()
    x, dy, w = gen((rows, fin), seed, dtype), gen((rows, fout), seed + 1, dtype), \
        gen((E, fout, fin), seed + 2, dtype)
    if poison:
        for t in (x, dy):
            t[:first] = float("nan")
            t[rows - spare:] = float("inf")
    xd, dyd, wd = (t.double().numpy() for t in (x, dy, w))
    X, DY, W, OFF = (t.to(DEV) for t in (x, dy, w, off))
    odt = torch.float32 if out_f32 else dtype
    xa, dya, wa = np.abs(xd), np.abs(dyd), np.abs(wd)
    say = f"counts={list(counts)[:9]} in={fin} out={fout} {dtype}"
    mine = slice(o[0], o[-1])
    if "y" in what:
        y = torch.full((rows, fout), -7.0, dtype=odt, device=DEV)
        assert fa.linear_grouped_fwd(X, W, OFF, out=y) is y
        within(y[mine], ol.grouped_fwd(xd, wd, o)[mine], fin, ol.grouped_fwd(xa, wa, o)[mine], f"y {say}")
        assert (y[:first] == -7).all() and (y[rows - spare:] == -7).all(), "rows of nobody"
    if "dx" in what:
        dx = torch.full((rows, fin), -7.0, dtype=odt, device=DEV)
        fa.linear_grouped_bwd_dx(DY, W, OFF, out=dx)
        within(dx[mine], ol.grouped_bwd_dx(dyd, wd, o)[mine], fout,
               ol.grouped_bwd_dx(dya, wa, o)[mine], f"dx {say}")
        assert (dx[:first] == -7).all() and (dx[rows - spare:] == -7).all(), "rows of nobody"
    K = np.asarray(counts, dtype=float)[:, None, None]
    ref, terms = ol.grouped_bwd_dw(dyd, xd, o), ol.grouped_bwd_dw(dya, xa, o)
    if "dw" in what:
        dw = torch.full((E, fout, fin), float("nan"), device=DEV)
        fa.linear_grouped_bwd_dw(DY, X, OFF, out=dw)
        within(dw, ref, K, terms, f"dw {say}")
        assert not dw[torch.tensor(counts) == 0].any()
    if "dw+" in what:
        prior = gen((E, fout, fin), seed + 3, torch.float32)
        dw = prior.to(DEV)
        fa.linear_grouped_bwd_dw(DY, X, OFF, out=dw, accumulate=True)
        prior = prior.double().numpy()
        within(dw, prior + ref, K, terms + np.abs(prior), f"dw+ {say}")
    fa.check_device_error()


@pytest.mark.parametrize("counts", [[1], [0], [3, 0, 1], [16, 17, 15], [64, 65, 63, 0, 1],
                                    [0, 0, 130], [255, 256, 257, 513], [31] * 9])
def test_counts(counts):
    run(counts, 72, 136, seed=sum(counts) + len(counts))


@pytest.mark.parametrize("fin,fout", [(8, 8), (64, 128), (120, 264), (520, 72), (256, 1032)])
def test_features(fin, fout):
    run([70, 5, 0, 140], fin, fout, seed=fin + fout)


def test_no_rows_at_all():
    run([0, 0, 0], 64, 72, seed=3)
    run([0, 0, 0], 64, 72, seed=3, first=5, spare=40)


def test_fp16_and_fp32_outputs():
    run([70, 129, 0, 33], 200, 136, seed=5, dtype=torch.float16)
    run([70, 129, 0, 33], 200, 136, seed=6, out_f32=True)
    run([70, 129, 0, 33], 136, 200, seed=7, dtype=torch.float16, out_f32=True)


def test_rows_of_nobody_are_neither_used_nor_written():
    run([40, 0, 90, 3], 136, 72, seed=9, first=13, spare=70, poison=True)
    run([1], 64, 64, seed=10, first=1, spare=1, poison=True)


def test_an_expert_with_values_that_are_not_finite_leaves_the_others_alone():
    counts, fin, fout = [33, 20, 70], 136, 200
    off = offsets_of(counts).to(DEV)
    x, dy = (gen((123, n), 11, torch.bfloat16).to(DEV) for n in (fin, fout))
    w = gen((3, fout, fin), 12).to(DEV)
    clean = (fa.linear_grouped_fwd(x, w, off), fa.linear_grouped_bwd_dx(dy, w, off),
             fa.linear_grouped_bwd_dw(dy, x, off))
    x[33:53], dy[33:53], w[1] = float("nan"), float("inf"), float("nan")
    y, dx, dw = (fa.linear_grouped_fwd(x, w, off), fa.linear_grouped_bwd_dx(dy, w, off),
                 fa.linear_grouped_bwd_dw(dy, x, off))
    for got, want in ((y, clean[0]), (dx, clean[1])):
        assert torch.equal(got[:33], want[:33]) and torch.equal(got[53:], want[53:])
        assert not torch.isfinite(got[33:53]).any()
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2])
    assert not torch.isfinite(dw[1]).any()


def test_many_experts():
    r = np.random.default_rng(1)
    run(r.integers(0, 3, size=1024), 24, 40, seed=15)
    run(r.integers(0, 40, size=130), 64, 264, seed=16)


def test_few_rows_of_many_experts():
    """A decoding step's shape: one or two rows to an expert."""
    run([1, 0, 2, 1, 0, 0, 1, 3, 0, 1, 1, 2, 0, 1, 1, 2], 1024, 520, seed=17)


def test_uneven_training_batch():
    r = np.random.default_rng(2)
    p = np.exp(r.normal(size=12))
    run(r.multinomial(6001, p / p.sum()), 520, 776, seed=19, spare=30)


def test_several_units_to_a_block():
    """More tiles than blocks: accumulators and stages are used again and again."""
    run([900, 1300, 20, 777], 264, 2056, seed=21)


def test_long_reductions_keep_fp32s_precision():
    """Chunks of 512 terms leave the tensor cores for sums rounded to nearest: 32 truncations of at
    most 2^-23 each, half of it on average and all towards zero, on partial sums that grow
    like sqrt(k) to the chunk's: 32 x 2^-24 x 2/3 = 1.3e-6 at most, however long the sum."""
    rows, fin, fout = 9000, 264, 136
    x, dy, w = gen((rows, fin), 1), gen((rows, fout), 2), gen((1, 1032, 8192), 3)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    dw = fa.linear_grouped_bwd_dw(dy.to(DEV), x.to(DEV), off).double().cpu()
    ref = dy.double().T @ x.double()
    assert float((dw[0] - ref).norm() / ref.norm()) <= 1.3e-6
    a = gen((40, 8192), 4)
    off = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    y = fa.linear_grouped_fwd(a.to(DEV), w.to(DEV), off, out_dtype=torch.float32).double().cpu()
    ref = a.double() @ w[0].double().T
    assert float((y - ref).norm() / ref.norm()) <= 1.3e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [4096, 4104, 8192, 65536 + 8, 2 ** 20])
def test_long_reductions_into_16_bit_outputs(K, dtype):
    """Terms of one sign, the worst for sums that are cut off: in chunks of 4096 terms at most
    4096 / 16 + 1 additions lose 2^-23 each, the chunks' sums lose 2^-24 each, and the output its
    half step, of sums of magnitudes that are the values themselves.  (In one piece 2^20 terms lost
    7e-3.)"""
    g = torch.Generator(device=DEV).manual_seed(K)
    a, w = ((torch.rand(s, generator=g, device=DEV) * 0.2).to(dtype) for s in ((40, K), (1, 72, K)))
    off = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    ref = a.double() @ w[0].double().t()
    assert ref.max() < 3e4
    bound = HALF[dtype] + 2.0 ** -23 * (4096 / 16 + 1) + 2.0 ** -24 * (K / 4096)
    y = fa.linear_grouped_fwd(a, w, off)
    dx = fa.linear_grouped_bwd_dx(a, w.transpose(1, 2).contiguous(), off)
    fa.check_device_error()
    for got in (y, dx):
        assert got.dtype == dtype
        assert float(((got.double() - ref) / ref).abs().max()) <= bound


def test_chunks_of_ragged_experts():
    """Reductions of several chunks and a rest, over tiles of several widths, empty ones between."""
    run([70, 5, 0, 300], 4104, 136, seed=41, what=("y",))
    run([33, 0, 257], 72, 8264, seed=42, dtype=torch.float16, what=("dx",), first=3, spare=9)


@pytest.mark.parametrize("rows", [130, 160, 190, 225, 250, 290, 330, 1000])
def test_every_tile_width(rows):
    """One expert: the device's choice of the tile's width goes through its range."""
    run([rows], 72, 1032, seed=rows, what=("y", "dx"))
    run([rows] * 20, 64, 264, seed=rows + 1, what=("y",))


def test_two_calls_at_once():
    """Products on two streams at a time, and attention beside them, give what each gives
    alone."""
    counts = [300, 0, 129, 33]
    off = offsets_of(counts).to(DEV)
    x, dy, w = gen((462, 136), 1).to(DEV), gen((462, 200), 2).to(DEV), gen((4, 200, 136), 3).to(DEV)
    q = gen((1, 4, 300, 64), 5).to(DEV)
    want = (fa.linear_grouped_fwd(x, w, off), fa.linear_grouped_bwd_dw(dy, x, off),
            fa.attn_fwd(q, q, q)[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(10):
        for s, call, res in zip(streams, (lambda: fa.linear_grouped_fwd(x, w, off),
                                          lambda: fa.linear_grouped_bwd_dw(dy, x, off),
                                          lambda: fa.attn_fwd(q, q, q)[0]), got):
            with torch.cuda.stream(s):
                res.append(call())
    torch.cuda.synchronize()
    for w_, res in zip(want, got):
        assert all(torch.equal(w_, r) for r in res)
    fa.check_device_error()


def test_wild_offsets_stay_inside_the_tensors():
    """Offsets past the rows, negative or decreasing are clamped: the calls end, and no row or
    gradient outside the tensors is touched."""
    x, w = gen((50, 64), 1).to(DEV), gen((4, 72, 64), 2).to(DEV)
    off = torch.tensor([-5, 20, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    guard = torch.full((70, 72), -7.0, dtype=torch.bfloat16, device=DEV)
    fa.linear_grouped_fwd(x, w, off, out=guard[10:60])
    assert (guard[:10] == -7).all() and (guard[60:] == -7).all()
    fa.linear_grouped_bwd_dx(gen((50, 72), 3).to(DEV), w, off)
    fa.linear_grouped_bwd_dw(gen((50, 72), 3).to(DEV), x, off)
    fa.check_device_error()


def test_results_repeat_on_another_stream_and_in_a_graph():
    counts = [70, 0, 129, 33]
    off = offsets_of(counts).to(DEV)
    x, dy, w = gen((232, 136), 1).to(DEV), gen((232, 200), 2).to(DEV), gen((4, 200, 136), 3).to(DEV)

    def all_three():
        return (fa.linear_grouped_fwd(x, w, off), fa.linear_grouped_bwd_dx(dy, w, off),
                fa.linear_grouped_bwd_dw(dy, x, off))

    want = all_three()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = all_three()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_three()
    # the counts are read at replay, not at capture
    off.copy_(offsets_of([100, 32, 0, 100]))
    graph.replay()
    torch.cuda.synchronize()
    want = all_three()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gradients_against_differences():
    """dx and dw along random directions against differences of the fp64 forward (which is
    linear in each: one step is exact), within the gradients' rounding."""
    counts, fin, fout = [20, 0, 33], 64, 72
    off = offsets_of(counts)
    o = off.tolist()
    x, dy, w = gen((53, fin), 1), gen((53, fout), 2), gen((3, fout, fin), 3)
    dx = fa.linear_grouped_bwd_dx(dy.to(DEV), w.to(DEV), off.to(DEV), out_dtype=torch.float32)
    dw = fa.linear_grouped_bwd_dw(dy.to(DEV), x.to(DEV), off.to(DEV))
    xd, dyd, wd = (t.double().numpy() for t in (x, dy, w))
    r = np.random.default_rng(5)
    ux, uw = r.normal(size=xd.shape), r.normal(size=wd.shape)
    for got, u, num in ((dx, ux, np.sum(dyd * ol.grouped_fwd(ux, wd, o))),
                        (dw, uw, np.sum(dyd * ol.grouped_fwd(xd, uw, o)))):
        terms = got.double().cpu().numpy() * u
        assert abs(terms.sum() - num) <= 2.0 ** -20 * np.abs(terms).sum()


def test_front_end_refusals_on_cuda_tensors():
    x, w = gen((8, 64), 1).to(DEV), gen((2, 72, 64), 2).to(DEV)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    dy = gen((8, 72), 3).to(DEV)
    for call, msg in [
            (lambda: fa.linear_grouped_fwd(x.half(), w, off), "dtype"),
            (lambda: fa.linear_grouped_fwd(x, w, off.long()), "dtype"),
            (lambda: fa.linear_grouped_fwd(x, w, off[:2]), "experts"),
            (lambda: fa.linear_grouped_fwd(x, w, off.cpu()), "CUDA"),
            (lambda: fa.linear_grouped_fwd(x[:, :56].contiguous(), w, off), "features"),
            (lambda: fa.linear_grouped_fwd(x[:, ::2], w, off), "contiguous"),
            (lambda: fa.linear_grouped_fwd(x, w, off, out=dy[:4]), "shape"),
            (lambda: fa.linear_grouped_fwd(x, w, off, out_dtype=torch.float16), "out_dtype"),
            (lambda: fa.linear_grouped_fwd(x, w, off, torch.empty_like(dy), torch.float32), "out_dtype"),
            (lambda: fa.linear_grouped_bwd_dx(dy, w, off, x.float(), x.dtype), "out_dtype"),
            (lambda: fa.linear_grouped_bwd_dx(x, w, off), "features"),
            (lambda: fa.linear_grouped_bwd_dw(dy[:7], x, off), "rows"),
            (lambda: fa.linear_grouped_bwd_dw(dy, x, off, accumulate=True), "out"),
            (lambda: fa.linear_grouped_bwd_dw(dy, x, off, out=w), "dtype")]:
        with pytest.raises(ValueError, match=msg):
            call()
