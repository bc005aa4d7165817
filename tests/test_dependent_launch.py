"""Kernels that start beside the one ahead of them in the stream read what it writes by ordinary
loads: the read-only path (__ldg, const __restrict__) is for data that nothing writes during
the kernel's lifetime (CPU: the sources; GPU: chains of such calls)."""
import os
import re

import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import build


@pytest.mark.parametrize("source", ["qkv.cu", "gemm_grouped.cu", "grad.cu"])
def test_no_read_only_loads(source):
    with open(os.path.join(build.CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "launch_dependent(" in text and "allow_dependents_launch();" in text
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict", text)


@pytest.mark.gpu
def test_chains_of_small_calls_see_each_others_writes():
    """Gradients clipped in place again and again, and norm weights' gradients through one
    workspace, without a synchronisation between: as with one after every call."""
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(3)
    start = [torch.randn(n, generator=g).to(dev) for n in (5000, 37, 70001)]
    x = torch.randn((1, 300, 2, 64), generator=g).to(torch.bfloat16).to(dev)
    dys = [torch.randn((1, 2, 300, 64), generator=g).to(dev) for _ in range(4)]
    w = torch.ones(64, device=dev)
    ws = torch.empty(fa.grad_workspace_bytes(3), dtype=torch.uint8, device=dev)
    ws_qkv = torch.empty(fa.qkv_workspace_bytes(64), dtype=torch.uint8, device=dev)

    def chain(between):
        grads, norms, acc = [t.clone() for t in start], [], (torch.zeros_like(w), torch.zeros_like(w))
        torch.cuda.synchronize()
        for n in range(200):
            norms.append(fa.grad_clip(grads, 200.0 * 0.99 ** n, workspace=ws))
            between()
            dy = dys[n % 4]
            fa.qkv_bwd(dy, dy, dy, x, x, w, w, weight_out=acc, accumulate=n > 0, workspace=ws_qkv)
            between()
        return torch.stack(norms), *grads, *acc

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, chain(lambda: None)))


@pytest.mark.gpu
def test_captured_between_memsets_copies_and_another_stream():
    """In a graph the kernels' neighbours are nodes of other kinds, and several of them: replays
    give what the same calls give eagerly."""
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(5)

    def rnd(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g).to(dtype).to(dev)

    x, w, rows, weights = rnd(1, 300, 2, 64), rnd(64, dtype=torch.float32), rnd(300, 128), rnd(3, 72, 128)
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device=dev)
    none = torch.zeros(4, dtype=torch.int32, device=dev)
    big = torch.zeros(300 * 128, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        big.zero_()  # a memset
        q, k, v = fa.qkv_fwd(x, x, x, w, w)
        big.copy_(rows.view(-1))  # a copy
        side.wait_stream(here)
        y = fa.linear_grouped_fwd(big.view(300, 128), weights, off)
        with torch.cuda.stream(side):
            gq, gk, gv, gwq, gwk = fa.qkv_bwd(q, k, v, x, x, w, w)
        dw = fa.linear_grouped_bwd_dw(y, rows, off)
        empty = fa.linear_grouped_bwd_dw(y[:0], rows[:0], none)  # a memset
        here.wait_stream(side)  # two nodes ahead of the next kernel
        norm = fa.grad_clip([dw, gwq, gwk, empty], 0.5)
        return q, k, v, y, gq, gk, gv, gwq, gwk, dw, empty, norm

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    fa.check_device_error()
