"""The front end of the operators around the attention beside other Python threads (GPU): calls
that wait for the device let them run, and calls of several threads on streams of their own
give what each gives alone."""
import threading
import time

import numpy as np
import pytest
import torch

import causal_attention_fwd_attn_b200 as fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def calls(seed=0):
    """One call of every entry point, all outputs and workspaces at hand."""
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g).to(dtype).to(DEV)

    x, w, freq = rnd(2, 40, 3, 64), rnd(64, dtype=torch.float32), torch.rand(32, generator=g).double().to(DEV)
    dy = [rnd(2, 3, 40, 64) for _ in range(3)]
    out, dx = [torch.empty_like(t) for t in dy], [torch.empty_like(x) for _ in range(3)]
    dws = [torch.empty_like(w) for _ in range(2)]
    ws_qkv = torch.empty(fa.qkv_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    off = torch.tensor([0, 30, 30, 70], dtype=torch.int32, device=DEV)
    rows, drows, weights = rnd(70, 72), rnd(70, 136), rnd(3, 136, 72)
    y, dxr, dwr = torch.empty_like(drows), torch.empty_like(rows), torch.empty((3, 136, 72), device=DEV)
    grads = [rnd(n, dtype=torch.float32) for n in (5000, 7)]
    clipped = [torch.empty_like(t) for t in grads]
    norm, ws = torch.empty((), device=DEV), torch.empty(fa.grad_workspace_bytes(2), dtype=torch.uint8, device=DEV)
    return {
        "qkv_fwd": lambda: fa.qkv_fwd(x, x, x, w, w, inv_freq=freq, out=tuple(out)),
        "qkv_bwd": lambda: fa.qkv_bwd(*dy, x, x, w, w, inv_freq=freq, out=tuple(dx), weight_out=tuple(dws),
                                      workspace=ws_qkv),
        "grouped_fwd": lambda: fa.linear_grouped_fwd(rows, weights, off, out=y),
        "grouped_dx": lambda: fa.linear_grouped_bwd_dx(drows, weights, off, out=dxr),
        "grouped_dw": lambda: fa.linear_grouped_bwd_dw(drows, rows, off, out=dwr),
        "grad_norm": lambda: fa.grad_norm(grads, norm=norm, workspace=ws),
        "grad_clip": lambda: fa.grad_clip(grads, 1.0, out=clipped, norm=norm, workspace=ws),
    }


def flat(res):
    return [t.clone() for t in (res if isinstance(res, (tuple, list)) else (res,))]


@pytest.mark.parametrize("name", ["qkv_fwd", "qkv_bwd", "grouped_fwd", "grouped_dx", "grouped_dw",
                                  "grad_norm", "grad_clip"])
def test_other_threads_run_while_a_launch_waits(name):
    """The stream is busy for about half a second, and calls are sent until its queue is full and
    a launch waits: a thread that only keeps time goes on meanwhile."""
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def keep_time():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.001)

    thread = threading.Thread(target=keep_time)
    thread.start()
    try:
        longest = 0.0
        busy = torch.cuda.Event()
        torch.cuda._sleep(10 ** 9)
        busy.record()
        begin = time.perf_counter()
        for _ in range(4000):
            t0 = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - t0)
            if busy.query():
                break
        end = time.perf_counter()
    finally:
        stop.set()
        thread.join()
    torch.cuda.synchronize()
    inside = [begin] + [t for t in ticks if begin < t < end] + [end]
    gap = float(np.max(np.diff(inside)))
    assert longest < 0.1 or gap < 0.5 * longest, f"a call took {longest:.3f} s, no tick for {gap:.3f} s"


def test_threads_on_streams_of_their_own():
    want = [{n: flat(c()) for n, c in calls(seed).items()} for seed in range(3)]
    torch.cuda.synchronize()
    wrong = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                mine = calls(seed)
                for _ in range(60):
                    for n, call in mine.items():
                        got = flat(call())
                        if not all(torch.equal(a, b) for a, b in zip(want[seed][n], got)):
                            wrong.append((seed, n))
        except Exception as e:  # shown by the main thread
            wrong.append((seed, repr(e)))

    threads = [threading.Thread(target=work, args=(seed,)) for seed in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    fa.check_device_error()
    assert not wrong, wrong[:3]


def test_a_list_that_changes_during_the_call():
    """Another thread empties the lists of gradients and outputs again and again: a call takes
    them as they were, whole or (empty) refused."""
    start = [torch.full((3000 + n,), 2.0, device=DEV) for n in range(300)]
    full = float(sum(4.0 * t.numel() for t in start)) ** 0.5
    grads, stop = [], threading.Event()

    def change():
        while not stop.is_set():
            grads[:] = start
            time.sleep(0)
            grads.clear()

    thread = threading.Thread(target=change)
    thread.start()
    try:
        for _ in range(2000):
            try:
                norm = fa.grad_norm(grads)
            except ValueError as e:
                assert "no gradients" in str(e)
                continue
            assert abs(norm.item() - full) <= 4e-6 * full
    finally:
        stop.set()
        thread.join()
    assert abs(fa.grad_norm(start).item() - full) <= 4e-6 * full
