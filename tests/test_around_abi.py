"""Refusals of the operators around the attention, through the C ABI and the torch front
ends (CPU: every call here is refused before any launch)."""
import ctypes

import pytest
import torch

import causal_attention_fwd_attn_b200 as fa
from causal_attention_fwd_attn_b200 import _lib, build

P = 4096  # a 16-byte aligned fake address; never dereferenced (rejected first)
BIG = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def config(**kw):
    c = dict(B=2, T=5, H=4, Hkv=2, d=64, rot=64, axes=1, eps=1e-6, inv_freq=P, positions=P,
             pair_axis=None, q_weight=P, k_weight=P)
    c.update(kw)
    return _lib.QkvConfig(*(c[n] for n, _ in _lib.QkvConfig._fields_))


def tensor(data=P, b=5 * 8 * 64, t=8 * 64, h=64):
    return _lib.QkvTensor(data, b, t, h)


def fwd(cfg=None, q=None, k=None, v=None, outs=(P, P, P), flags=0):
    return _lib.forge_qkv_fwd(cfg or config(), q or tensor(), k or tensor(), v or tensor(), *outs,
                              flags, None)


@pytest.mark.parametrize("change,want", [
    (dict(B=0), _lib.ERR_INVALID_ARG), (dict(T=0), _lib.ERR_INVALID_ARG),
    (dict(H=0), _lib.ERR_INVALID_ARG), (dict(Hkv=0), _lib.ERR_INVALID_ARG),
    (dict(H=5), _lib.ERR_INVALID_ARG),                      # not a multiple of Hkv
    (dict(d=96), _lib.ERR_UNSUPPORTED), (dict(rot=66), _lib.ERR_INVALID_ARG),
    (dict(rot=-2), _lib.ERR_INVALID_ARG), (dict(rot=31), _lib.ERR_INVALID_ARG),
    (dict(rot=40), _lib.ERR_UNSUPPORTED),                   # halves need multiples of 16
    (dict(axes=0), _lib.ERR_INVALID_ARG), (dict(inv_freq=None), _lib.ERR_INVALID_ARG),
    (dict(inv_freq=P + 4), _lib.ERR_MISALIGNED), (dict(positions=P + 2), _lib.ERR_MISALIGNED),
    (dict(pair_axis=P + 1), _lib.ERR_MISALIGNED), (dict(q_weight=P + 2), _lib.ERR_MISALIGNED),
    (dict(eps=-1e-6), _lib.ERR_INVALID_ARG), (dict(eps=float("nan")), _lib.ERR_INVALID_ARG),
    (dict(B=1 << 12, T=1 << 12, H=2), _lib.ERR_UNSUPPORTED),  # 2^31 elements
    (dict(B=1 << 20, T=1 << 20), _lib.ERR_UNSUPPORTED),
])
def test_qkv_rejects_bad_configs(change, want):
    assert fwd(config(**change)) == want
    ws = _lib.forge_qkv_bwd_workspace_size(64)
    assert _lib.forge_qkv_bwd(config(**change), P, P, P, tensor(), tensor(), tensor(), tensor(),
                              tensor(), P, P, 0, P, ws, 0, None) == want


def test_qkv_rejects_bad_tensors():
    assert fwd(flags=1) == _lib.ERR_INVALID_ARG
    assert fwd(flags=_lib.QKV_GRAD_F32) == _lib.ERR_INVALID_ARG  # the backward's
    assert fwd(q=tensor(data=None)) == _lib.ERR_INVALID_ARG
    assert fwd(q=tensor(data=P + 8)) == _lib.ERR_MISALIGNED
    assert fwd(k=tensor(t=-64)) == _lib.ERR_INVALID_ARG
    assert fwd(v=tensor(h=68)) == _lib.ERR_MISALIGNED
    assert fwd(outs=(P, P + 8, P)) == _lib.ERR_MISALIGNED
    assert fwd(outs=(P, None, P)) == _lib.ERR_INVALID_ARG
    assert _lib.forge_qkv_fwd(config(), None, None, None, None, None, None, 0, None) == \
        _lib.ERR_INVALID_ARG
    assert _lib.forge_qkv_fwd(None, tensor(), None, None, P, None, None, 0, None) == \
        _lib.ERR_INVALID_ARG


def test_qkv_backward_rejects_bad_arguments():
    ws = _lib.forge_qkv_bwd_workspace_size(64)
    assert ws > 0 and _lib.forge_qkv_bwd_workspace_size(128) == 2 * ws
    assert _lib.forge_qkv_bwd_workspace_size(96) == 0

    def bwd(cfg=None, grads=(P, P, P), q=tensor(), k=tensor(), outs=None, dw=(P, P), acc=0,
            workspace=P, n=ws, flags=0):
        outs = outs or (tensor(), tensor(), tensor())
        return _lib.forge_qkv_bwd(cfg or config(), *grads, q, k, *outs, *dw, acc, workspace, n, flags,
                                  None)

    assert bwd(acc=2) == _lib.ERR_INVALID_ARG
    assert bwd(flags=64) == _lib.ERR_INVALID_ARG
    assert bwd(grads=(P, None, P)) == _lib.ERR_INVALID_ARG
    assert bwd(grads=(P + 2, P, P)) == _lib.ERR_MISALIGNED
    assert bwd(q=None) == _lib.ERR_INVALID_ARG            # the norm's source
    assert bwd(dw=(None, P)) == _lib.ERR_INVALID_ARG
    assert bwd(dw=(P, P + 2)) == _lib.ERR_MISALIGNED
    assert bwd(workspace=None) == _lib.ERR_WORKSPACE
    assert bwd(n=ws - 1) == _lib.ERR_WORKSPACE
    assert bwd(workspace=P + 8) == _lib.ERR_MISALIGNED
    # gradients whose elements coincide: a broadcast batch, overlapping heads
    assert bwd(outs=(tensor(b=0), tensor(), tensor())) == _lib.ERR_INVALID_ARG
    assert bwd(outs=(tensor(h=32), tensor(), tensor())) == _lib.ERR_INVALID_ARG
    assert bwd(outs=(tensor(t=3 * 64), tensor(), tensor())) == _lib.ERR_INVALID_ARG
    assert _lib.forge_qkv_bwd(config(), None, None, None, None, None, None, None, None, None, None, 0,
                              P, ws, 0, None) == _lib.ERR_INVALID_ARG


def test_qkv_rejects_outputs_that_overlap():
    """The same tensor twice, or neighbours that share their ends."""
    size = 2 * 2 * 5 * 4 * 64  # bytes of an output
    far = [P + n * (size + 16) for n in range(3)]
    for outs in ((far[0], far[0], far[2]), (far[0], far[1], far[1]), (far[0], far[1], far[0]),
                 (far[1] - 32, far[1], far[2]), (far[0], far[2] + 32, far[2])):
        assert fwd(outs=outs) == _lib.ERR_INVALID_ARG
    # far apart, nothing else is wrong: the launch itself fails without a device
    if not torch.cuda.is_available():
        assert fwd(outs=far) == _lib.ERR_CUDA
    # both weights' gradients: one would be lost
    ws = _lib.forge_qkv_bwd_workspace_size(64)

    def bwd(dq_weight, dk_weight, cfg=None):
        return _lib.forge_qkv_bwd(cfg or config(), P, P, P, tensor(), tensor(), tensor(), tensor(), tensor(),
                                  dq_weight, dk_weight, 1, P, ws, 0, None)

    assert bwd(P, P) == _lib.ERR_INVALID_ARG
    assert bwd(P, P + 252) == _lib.ERR_INVALID_ARG
    assert bwd(P + 128, P) == _lib.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert bwd(P, P + 256) == _lib.ERR_CUDA
        assert bwd(P, P, config(k_weight=None)) == _lib.ERR_CUDA  # only one is written


def test_grouped_rejects_bad_arguments():
    for fn in (_lib.forge_linear_grouped_fwd, _lib.forge_linear_grouped_bwd_dx):
        assert fn(P, P, P, P, 0, 4, 64, 64, 0, None) == _lib.OK  # no rows: nothing to do
        assert fn(None, P, None, P, 0, 4, 64, 64, 0, None) == _lib.OK
        assert fn(P, P, P, None, 8, 4, 64, 64, 0, None) == _lib.ERR_INVALID_ARG
        assert fn(None, P, P, P, 8, 4, 64, 64, 0, None) == _lib.ERR_INVALID_ARG
        assert fn(P, None, P, P, 8, 4, 64, 64, 0, None) == _lib.ERR_INVALID_ARG
        assert fn(P, P, P, P, -1, 4, 64, 64, 0, None) == _lib.ERR_INVALID_ARG
        assert fn(P, P, P, P, 8, 0, 64, 64, 0, None) == _lib.ERR_INVALID_ARG
        assert fn(P, P, P, P, 8, 1025, 64, 64, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 8, 4, 60, 64, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 8, 4, 64, 12, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 1 << 25, 4, 64, 64, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 8, 4, 1 << 21, 64, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 8, 4, 64, 1 << 21, 0, None) == _lib.ERR_UNSUPPORTED
        assert fn(P, P, P, P, 8, 4, 64, 64, _lib.PRECISE, None) == _lib.ERR_INVALID_ARG
        assert fn(P, P + 8, P, P, 8, 4, 64, 64, 0, None) == _lib.ERR_MISALIGNED
        assert fn(P, P, P, P + 2, 8, 4, 64, 64, 0, None) == _lib.ERR_MISALIGNED
    dw = _lib.forge_linear_grouped_bwd_dw
    assert dw(None, None, P, P, 0, 4, 64, 64, 1, 0, None) == _lib.OK  # nothing to add
    assert dw(P, P, None, P, 8, 4, 64, 64, 0, 0, None) == _lib.ERR_INVALID_ARG
    assert dw(P, P, P, P, 8, 4, 64, 64, 2, 0, None) == _lib.ERR_INVALID_ARG
    assert dw(P, P, P, P, 8, 4, 64, 64, 0, _lib.OUT_F32, None) == _lib.ERR_INVALID_ARG
    assert dw(P, P + 2, P, P, 8, 4, 64, 64, 0, 0, None) == _lib.ERR_MISALIGNED
    assert dw(P, P, P + 4, P, 8, 4, 64, 64, 0, 0, None) == _lib.ERR_MISALIGNED
    assert dw(None, P, P, P, 8, 4, 64, 64, 0, 0, None) == _lib.ERR_INVALID_ARG


def test_grad_rejects_bad_arguments():
    n = _lib.forge_grad_workspace_size(1)
    assert n > 0 and _lib.forge_grad_workspace_size(0) == 0
    assert _lib.forge_grad_workspace_size(257) == 2 * _lib.forge_grad_workspace_size(256)

    def clip(fields, count=1, max_norm=1.0, norm=P, ws=P, size=n):
        return _lib.forge_grad_clip(_lib.grad_table(fields, len(fields) // 4), count, max_norm, norm,
                                    ws, size, None)

    ok = [P, P + BIG, 8, 0]
    assert clip(ok, count=0) == _lib.ERR_INVALID_ARG
    assert clip(ok, max_norm=0.0) == _lib.ERR_INVALID_ARG
    assert clip(ok, max_norm=float("inf")) == _lib.ERR_INVALID_ARG
    assert clip(ok, ws=None) == _lib.ERR_WORKSPACE
    assert clip(ok, size=n - 1) == _lib.ERR_WORKSPACE
    assert clip(ok, ws=P + 8) == _lib.ERR_MISALIGNED
    assert clip(ok, norm=P + 2) == _lib.ERR_MISALIGNED
    assert clip([P, P + BIG, -1, 0]) == _lib.ERR_INVALID_ARG
    assert clip([P, P + BIG, 8, 3]) == _lib.ERR_INVALID_ARG
    assert clip([0, P, 8, 0]) == _lib.ERR_INVALID_ARG
    assert clip([P, 0, 8, 0]) == _lib.ERR_INVALID_ARG
    assert clip([P + 4, P + BIG, 8, 0]) == _lib.ERR_MISALIGNED
    assert clip([P, P + 16, 8, 0]) == _lib.ERR_INVALID_ARG  # partly overlapping
    assert clip([P, P + BIG, 1 << 45, 0]) == _lib.ERR_UNSUPPORTED
    t = _lib.grad_table(ok, 1)
    assert _lib.forge_grad_norm(t, 1, None, P, n, None) == _lib.ERR_INVALID_ARG
    assert _lib.forge_grad_norm(t, 1, P, P, n - 1, None) == _lib.ERR_WORKSPACE


def test_structures_match_the_header():
    assert ctypes.sizeof(_lib.QkvConfig) == 72 and ctypes.sizeof(_lib.QkvTensor) == 32
    assert len(_lib.grad_table([P, P, 8, 0], 1)) == 32


def test_front_ends_refuse_cpu_tensors_and_wrong_shapes():
    x = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qkv_fwd(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qkv_bwd(x, x, x, x, x)
    with pytest.raises(ValueError, match=r"\[B, T, heads, d\]"):
        fa.qkv_fwd(x[0], x, x)
    with pytest.raises(ValueError, match="dtype"):
        fa.qkv_fwd(x.float(), x, x)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.linear_grouped_fwd(x[0, 0], x[0], o)
    with pytest.raises(ValueError, match="CUDA"):
        fa.linear_grouped_bwd_dx(x[0, 0], x[0], o)
    with pytest.raises(ValueError, match="CUDA"):
        fa.linear_grouped_bwd_dw(x[0, 0], x[0, 0], o)
    with pytest.raises(ValueError, match="CUDA"):
        fa.grad_clip([x.float()], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        fa.grad_norm([])
