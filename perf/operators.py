"""Cases of the operators around the attention, for measurement: the stage from a QKV projection
to the attention (per-head norm, rotation, head layout) forward and backward, the linear products
grouped by expert, and the clipping of gradients at a global norm.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the calls a user makes
of the package.  ``exact`` is the operators' definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases --
def listed():
    return [
        # one new token for each of 48 sequences, at far positions, shared key/value heads:
        # a decoding step, where the launch is what counts
        dict(name="qkv_fwd_decode", op="qkv_fwd", B=48, T=1, H=32, Hkv=8, d=128, rot=128, axes=1,
             dtype="bf16", adjacent=False, packed=True, norm=True, far=True),
        # the attention layer of a small language model in training, fp16, adjacent pairs
        dict(name="qkv_fwd_b8h12t1024d64", op="qkv_fwd", B=8, T=1024, H=12, Hkv=12, d=64, rot=64,
             axes=1, dtype="fp16", adjacent=True, packed=True, norm=True, far=False),
        # one long ragged sequence of video patches: time, height and width positions
        dict(name="qkv_fwd_video_t8000d128", op="qkv_fwd", B=1, T=8000, H=32, Hkv=32, d=128, rot=128,
             axes=3, dtype="bf16", adjacent=False, packed=True, norm=True, far=False),
        # the backward of a layer with head dimension 128, with its norm weights' gradients
        dict(name="qkv_bwd_b2h16t4096d128", op="qkv_bwd", B=2, T=4096, H=16, Hkv=16, d=128, rot=128,
             axes=1, dtype="bf16", grad="bf16", adjacent=False, packed=True, norm=True, far=False),
        # images of odd token counts: two axes, half of each head rotated, three query heads to
        # a key/value head, the attention's fp32 gradients
        dict(name="qkv_bwd_image_t1023d64", op="qkv_bwd", B=3, T=1023, H=12, Hkv=4, d=64, rot=32,
             axes=2, dtype="fp16", grad="fp32", adjacent=False, packed=False, norm=True, far=False),
        # decoding with experts: 16 tokens, two experts each; the weights of 20 experts are read
        dict(name="grouped_fwd_decode", op="grouped_fwd", rows=32, spare=0, E=32, active=20, fin=2048,
             fout=4096, dtype="bf16", out="bf16", skew=0.5),
        # the up projection of 16 experts over a training batch of routed rows
        dict(name="grouped_fwd_train", op="grouped_fwd", rows=16384, spare=0, E=16, active=16, fin=2048,
             fout=4096, dtype="bf16", out="bf16", skew=0.5),
        # input gradients: odd row counts, one expert without rows, rows routed to nobody at the end
        dict(name="grouped_dx_ragged", op="grouped_dx", rows=12001, spare=77, E=24, active=23, fin=1024,
             fout=2816, dtype="fp16", out="fp16", skew=1.0),
        # weight gradients of a training batch
        dict(name="grouped_dw_train", op="grouped_dw", rows=16384, spare=0, E=8, active=8, fin=2048,
             fout=4096, dtype="bf16", accumulate=False, skew=0.5),
        # weight gradients of a small ragged micro-batch, added to earlier ones
        dict(name="grouped_dw_accumulate", op="grouped_dw", rows=1501, spare=3, E=12, active=10, fin=776,
             fout=520, dtype="fp16", accumulate=True, skew=1.0),
        # all gradients of a 124M-parameter model in fp32 (148 tensors), clipped
        dict(name="grad_clip_124m", op="grad_clip", tensors="gpt2small", kind="fp32", clipped=True),
        # the gradients of a few adapters: odd sizes, bf16 and fp32 side by side
        dict(name="grad_clip_adapters", op="grad_clip", tensors="24x30011", kind="mixed", clipped=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qkv_fwd", "qkv_bwd", "grouped_fwd", "grouped_dx", "grouped_dw", "grad_clip"])
    if op.startswith("qkv"):
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        H = min(32, Hkv * rng.choice([1, 1, 2, 3, 4, 8]))
        H = H // Hkv * Hkv
        T = _log(rng, 1, 8191)
        most = 32 * 8000 * 128 // (H * d)  # tokens of the largest listed case
        B = _log(rng, 1, max(1, min(64, most // T)))
        c = dict(op=op, B=B, T=T, H=H, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                 axes=rng.choice([1, 1, 2, 3]), dtype=rng.choice(["bf16", "fp16"]),
                 adjacent=rng.random() < 0.3, packed=rng.random() < 0.7, norm=rng.random() < 0.8,
                 far=rng.random() < 0.3)
        if op == "qkv_bwd":
            c["grad"] = rng.choice([c["dtype"], "fp32"])
            c["B"] = max(1, B // 2)
        return c
    if op.startswith("grouped"):
        E = _log(rng, 2, 64)
        rows = _log(rng, 4, 16384)
        active = max(1, min(rows, E, round(E * rng.uniform(0.6, 1.0))))
        fin, fout = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512)
        while E * fin * fout > 16 * 2048 * 4096:
            E, active = max(2, E // 2), max(1, min(active, E // 2))
        c = dict(op=op, rows=rows, spare=rng.choice([0, 0, 1, 130]), E=E, active=active, fin=fin,
                 fout=fout, dtype=rng.choice(["bf16", "fp16"]), skew=rng.choice([0.0, 0.5, 1.0]))
        if op == "grouped_dw":
            c["accumulate"] = rng.random() < 0.5
        else:
            c["out"] = rng.choice([c["dtype"], c["dtype"], "fp32"])
        return c
    n = _log(rng, 1, 300)
    return dict(op=op, tensors="%dx%d" % (n, _log(rng, 7, max(8, 60_000_000 // n))),
                kind=rng.choice(["fp32", "bf16", "fp16", "mixed"]), clipped=rng.random() < 0.8)


# ------------------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype)


def _heads(g, case):
    """The projection's output as q, k, v views [B, T, heads, d]: parts of one packed tensor, or
    tensors of their own."""
    B, T, H, Hkv, d = (case[n] for n in ("B", "T", "H", "Hkv", "d"))
    dt = DTYPES[case["dtype"]]
    if case["packed"]:
        x = _randn(g, (B, T, H + 2 * Hkv, d), dt)
        return x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    return tuple(_randn(g, (B, T, h, d), dt) for h in (H, Hkv, Hkv))


def _positions(g, case):
    """Positions of every token on each axis, and the axis of each frequency pair: sections of
    the pairs, as multi-axis models share them out."""
    B, T, axes, pairs = case["B"], case["T"], case["axes"], case["rot"] // 2
    t = torch.arange(T, device=DEV)
    shift = torch.randint(0, 1_000_000 if case["far"] else 64, (B, 1), generator=g, device=DEV)
    if axes == 1:
        return (shift + t).to(torch.int32)[None].contiguous(), None
    wide = max(1, int(math.sqrt(T / 4)))
    grid = [t // wide, t % wide] if axes == 2 else [t // (wide * wide), t // wide % wide, t % wide]
    pos = torch.stack([(shift + p) for p in grid]).to(torch.int32).contiguous()
    axis = torch.div(torch.arange(pairs, device=DEV) * axes, pairs, rounding_mode="floor")
    return pos, axis.to(torch.int32)


def _counts(case, seed):
    """Rows of each expert, as a router with uneven preferences gives them: `active` experts
    have some."""
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    E, active, rows = case["E"], case["active"], case["rows"]
    p = np.exp(case["skew"] * r.randn(active))
    n = np.zeros(E, dtype=np.int64)
    n[r.permutation(E)[:active]] = 1 + r.multinomial(rows - active, p / p.sum())
    return n


def _sizes(case):
    if case["tensors"] == "gpt2small":
        e, layers, vocab, ctx = 768, 12, 50257, 1024
        block = [e, e, 3 * e * e, 3 * e, e * e, e, e, e, 4 * e * e, 4 * e, 4 * e * e, e]
        return [vocab * e, ctx * e] + block * layers + [e, e]
    n, most = (int(x) for x in case["tensors"].split("x"))
    return [1 + (k * 7919 + most) % most for k in range(n)]


def _flat(g, sizes, dtype):
    """Gradients as slices of one buffer (16-byte aligned, zeros between), and room for the
    clipped ones."""
    at = np.concatenate([[0], np.cumsum([-(-n // 8) * 8 for n in sizes])]).tolist()
    keep = np.zeros(at[-1], dtype=bool)
    for a, n in zip(at, sizes):
        keep[a:a + n] = True
    flat = torch.where(torch.from_numpy(keep).to(DEV),
                       torch.randn(at[-1], generator=g, device=DEV) * 0.01, 0.0).to(dtype)
    out = torch.zeros_like(flat)
    return (flat, out, [flat[a:a + n] for a, n in zip(at, sizes)],
            [out[a:a + n] for a, n in zip(at, sizes)])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op.startswith("qkv"):
        B, T, H, Hkv, d, rot = (case[n] for n in ("B", "T", "H", "Hkv", "d", "rot"))
        dt = DTYPES[case["dtype"]]
        s["q"], s["k"], s["v"] = _heads(g, case)
        s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
                            for _ in range(2))
        s["pos"], s["axis"] = _positions(g, case)
        j = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
        s["freq"] = 10000.0 ** (-2.0 * j / rot)
        if op == "qkv_fwd":
            s["out"] = tuple(torch.empty((B, H, T, d), dtype=dt, device=DEV) for _ in range(3))
        else:
            s["grads"] = tuple(_randn(g, (B, H, T, d), DTYPES[case["grad"]]) for _ in range(3))
            s["dx"] = torch.empty((B, T, H + 2 * Hkv, d), dtype=dt, device=DEV)
    elif op.startswith("grouped"):
        n = _counts(case, seed)
        dt = DTYPES[case["dtype"]]
        E, fin, fout, all_rows = case["E"], case["fin"], case["fout"], case["rows"] + case["spare"]
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
        s["most"] = int(n.max())  # rows of the fullest expert, for the plain form's padding
        if op != "grouped_dx":
            s["x"] = _randn(g, (all_rows, fin), dt)
        if op != "grouped_fwd":
            s["dy"] = _randn(g, (all_rows, fout), dt)
        if op == "grouped_dw":
            s["dw"] = torch.randn((E, fout, fin), generator=g, device=DEV)
        else:
            s["w"] = _randn(g, (E, fout, fin), dt, fin ** -0.5)
            s["y"] = torch.zeros((all_rows, fout if op == "grouped_fwd" else fin),
                                 dtype=DTYPES[case["out"]], device=DEV)
    else:
        sizes = _sizes(case)
        half = len(sizes) // 2 if case["kind"] == "mixed" else len(sizes)
        kinds = ("bf16", "fp32") if case["kind"] == "mixed" else (case["kind"], case["kind"])
        parts = [_flat(g, n, DTYPES[k]) for n, k in zip((sizes[:half], sizes[half:]), kinds) if n]
        s["flats"] = [p[0] for p in parts]
        s["outs"] = [p[1] for p in parts]
        s["grad"] = [t for p in parts for t in p[2]]
        s["clip"] = [t for p in parts for t in p[3]]
        full = 0.01 * math.sqrt(sum(sizes))  # about what the norm is
        s["max_norm"] = 0.25 * full if case["clipped"] else 4.0 * full
    return s


# --------------------------------------------------------------------------- plain form --
def _angles(s):
    """cos and sin of every token's angles, [B, T, 1, rot / 2]; the angles in 64 bits."""
    pos = s["pos"].double()
    p = pos[0][..., None] if s["axis"] is None else pos[s["axis"].long()].movedim(0, -1)
    a = (p * s["freq"])[:, :, None]
    return a.cos().float(), a.sin().float()


def _turn(x, cos, sin, adjacent):
    """Rotates the first 2 * pairs elements of every head of x."""
    n = 2 * cos.shape[-1]
    y, rest = x[..., :n], x[..., n:]
    if adjacent:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = y[..., :n // 2], y[..., n // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, rest), dim=-1)


def _plain_head(x, w, cos, sin, case):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _turn(x, cos, sin, case["adjacent"])


def _spread(x, case):
    """[B, T, heads, d] to the attention's [B, H, T, d], key/value heads repeated, rounded."""
    x = x.transpose(1, 2).repeat_interleave(case["H"] // x.shape[2], dim=1)
    return x.to(DTYPES[case["dtype"]]).contiguous()


def _plain_qkv_fwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    return (_spread(_plain_head(s["q"], s["wq"], cos, sin, c), c),
            _spread(_plain_head(s["k"], s["wk"], cos, sin, c), c), _spread(s["v"], c))


def _plain_back(dy, x, w, cos, sin, case):
    """Gradients of one projection's heads and of its norm weight."""
    dy = _gather(dy, x.shape[2])
    g = _turn(dy, cos, -sin, case["adjacent"])
    if w is None:
        return g, None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n, gw = x * r, g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1, 2), dtype=torch.float64).float()


def _gather(dy, heads):
    """[B, H, T, d] gradients to [B, T, heads, d] in 32 bits, summed over shared heads."""
    B, H, T, d = dy.shape
    return dy.float().reshape(B, heads, H // heads, T, d).sum(2).transpose(1, 2)


def _plain_qkv_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    dq, dk, dv = s["grads"]
    gq, gwq = _plain_back(dq, s["q"], s["wq"], cos, sin, c)
    gk, gwk = _plain_back(dk, s["k"], s["wk"], cos, sin, c)
    dx = torch.cat((gq, gk, _gather(dv, c["Hkv"])), dim=2).to(DTYPES[c["dtype"]])
    return (dx, gwq, gwk) if gwq is not None else (dx,)


def _padded(x, s):
    """Rows of each expert side by side, [E, most, features] in 32 bits, zeros after the last."""
    o = s["offsets"].long()
    at = torch.arange(s["most"], device=DEV)
    n = (o[1:] - o[:-1])[:, None]
    rows = (o[:-1, None] + at).clamp(max=x.shape[0] - 1)
    return torch.where((at < n)[..., None], x[rows].float(), 0.0)


def _plain_grouped(s, x, transposed):
    """y of the rows that belong to an expert, the others as they were."""
    w = s["w"].float()
    yp = _padded(x, s) @ (w if transposed else w.transpose(1, 2))
    o = s["offsets"].long()
    row = torch.arange(x.shape[0], device=DEV)
    e = torch.bucketize(row, o[1:], right=True).clamp(max=o.shape[0] - 2)
    y = yp[e, (row - o[e]).clamp(max=s["most"] - 1)].to(s["y"].dtype)
    return torch.where((row < o[-1])[:, None], y, s["y"])


def _plain_dw(s):
    dw = _padded(s["dy"], s).transpose(1, 2) @ _padded(s["x"], s)
    return s["dw"] + dw if s["case"]["accumulate"] else dw


def _plain_clip(s):
    total = torch.stack([torch.sum(f.float().square(), dtype=torch.float64) for f in s["flats"]]).sum()
    norm = total.sqrt().float()
    c = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    return [norm] + [(f.float() * c).to(f.dtype) for f in s["flats"]]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "qkv_fwd":
        return _plain_qkv_fwd(s)
    if op == "qkv_bwd":
        return _plain_qkv_bwd(s)
    if op == "grouped_fwd":
        return _plain_grouped(s, s["x"], False)
    if op == "grouped_dx":
        return _plain_grouped(s, s["dy"], True)
    if op == "grouped_dw":
        return _plain_dw(s)
    return _plain_clip(s)


# --------------------------------------------------------------------- the user's calls --
def _run_own(s):
    import causal_attention_fwd_attn_b200 as fa

    case = s["case"]
    op = case["op"]
    if op.startswith("qkv"):
        rope = dict(eps=EPS, inv_freq=s["freq"], positions=s["pos"], pair_axis=s["axis"],
                    adjacent=case["adjacent"])
    if op == "qkv_fwd":
        return fa.qkv_fwd(s["q"], s["k"], s["v"], s["wq"], s["wk"], out=s["out"], **rope)
    if op == "qkv_bwd":
        H, Hkv, dx = case["H"], case["Hkv"], s["dx"]
        out = (dx[:, :, :H], dx[:, :, H:H + Hkv], dx[:, :, H + Hkv:])
        _, _, _, gwq, gwk = fa.qkv_bwd(*s["grads"], s["q"], s["k"], s["wq"], s["wk"], out=out, **rope)
        return (dx, gwq, gwk) if gwq is not None else (dx,)
    if op == "grouped_fwd":
        return fa.linear_grouped_fwd(s["x"], s["w"], s["offsets"], out=s["y"])
    if op == "grouped_dx":
        return fa.linear_grouped_bwd_dx(s["dy"], s["w"], s["offsets"], out=s["y"])
    if op == "grouped_dw":
        if not case["accumulate"]:
            return fa.linear_grouped_bwd_dw(s["dy"], s["x"], s["offsets"], out=s["dw"])
        dw = s["dw"].clone()  # the earlier sum, kept so that a pass can be repeated
        return fa.linear_grouped_bwd_dw(s["dy"], s["x"], s["offsets"], out=dw, accumulate=True)
    norm = fa.grad_clip(s["grad"], s["max_norm"], out=s["clip"])
    return [norm] + s["outs"]


def run(s):
    return _run_own(s) if own else _run_plain(s)


# --------------------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op.startswith("qkv"):
        B, T, H, Hkv, d = (case[n] for n in ("B", "T", "H", "Hkv", "d"))
        row = B * T * d
        side = 4 * B * T * case["axes"] + 4 * case["rot"] + 8 * d  # positions, frequencies, weights
        if op == "qkv_fwd":
            return {"bytes": 2 * row * (H + 2 * Hkv) + 2 * row * 3 * H + side, "flops": 8 * row * (H + Hkv)}
        read = SIZE[case["grad"]] * row * 3 * H + (2 * row * (H + Hkv) if case["norm"] else 0)
        return {"bytes": read + 2 * row * (H + 2 * Hkv) + side + 8 * d, "flops": 16 * row * (H + Hkv)}
    if op.startswith("grouped"):
        rows, E, active, fin, fout = (case[n] for n in ("rows", "E", "active", "fin", "fout"))
        flops = 2 * rows * fin * fout
        if op == "grouped_dw":
            return {"bytes": 2 * rows * (fin + fout) + 4 * E * fin * fout * (2 if case["accumulate"] else 1),
                    "flops": flops}
        a, b = (fin, fout) if op == "grouped_fwd" else (fout, fin)
        return {"bytes": 2 * rows * a + 2 * active * fin * fout + SIZE[case["out"]] * rows * b, "flops": flops}
    sizes = _sizes(case)
    half = len(sizes) // 2 if case["kind"] == "mixed" else 0
    kinds = ["bf16"] * half + [case["kind"] if half == 0 and case["kind"] != "mixed" else "fp32"] * (len(sizes) - half)
    return {"bytes": sum(2 * SIZE[k] * n for k, n in zip(kinds, sizes)), "flops": 3 * sum(sizes)}


# ----------------------------------------------------------------------- 64-bit results --
def _exact_head(x, w, s):
    """One projection's heads [B, T, heads, d] normed and turned, in 64 bits: each pair is a
    complex number times e^(i position frequency)."""
    case = s["case"]
    B, T, heads, d = x.shape
    pairs = case["rot"] // 2
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / d + EPS).sqrt() * w
    axis = torch.zeros(pairs, dtype=torch.int64, device=DEV) if s["axis"] is None else s["axis"].to(torch.int64)
    phi = torch.einsum("jbt,j->btj", s["pos"].to(torch.float64)[axis], s["freq"])
    unit = torch.polar(torch.ones_like(phi), phi)[:, :, None, :]
    head = x[..., :2 * pairs]
    if case["adjacent"]:
        z = torch.view_as_real(torch.view_as_complex(head.reshape(B, T, heads, pairs, 2).contiguous()) * unit)
        head = z.reshape(B, T, heads, 2 * pairs)
    else:
        z = torch.complex(head[..., :pairs], head[..., pairs:]) * unit
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., 2 * pairs:]), -1)


def _exact_qkv(s, q, k, v, wq, wk):
    H = s["case"]["H"]
    outs = []
    for x in (_exact_head(q, wq, s), _exact_head(k, wk, s), v):
        B, T, heads, d = x.shape
        x = x[:, :, :, None].expand(B, T, heads, H // heads, d).reshape(B, T, H, d)
        outs.append(x.permute(0, 2, 1, 3))
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("qkv"):
        ins = [s[n].double() for n in ("q", "k", "v")]
        ws = [s[n].double() if s[n] is not None else None for n in ("wq", "wk")]
        if op == "qkv_fwd":
            return tuple(t.contiguous() for t in _exact_qkv(s, *ins, *ws))
        need = [t.requires_grad_() for t in ins + ws if t is not None]
        outs = _exact_qkv(s, *ins, *ws)
        got = torch.autograd.grad(outs, need, [g.double() for g in s["grads"]])
        dx = torch.cat(got[:3], dim=2)
        return (dx, *got[3:])
    if op.startswith("grouped"):
        o = s["offsets"].tolist()
        out = s["y"].double() if op != "grouped_dw" else s["dw"].double() * (1.0 if case["accumulate"] else 0.0)
        for e, (a, b) in enumerate(zip(o[:-1], o[1:])):
            if a == b:
                continue
            if op == "grouped_fwd":
                out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
            elif op == "grouped_dx":
                out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
            else:
                out[e] += s["dy"][a:b].double().T @ s["x"][a:b].double()
        return out
    norm = math.sqrt(math.fsum(float(torch.sum(t.double() ** 2)) for t in s["grad"]))
    c = min(1.0, s["max_norm"] / norm)
    return [torch.tensor(norm, dtype=torch.float64)] + [f.double() * c for f in s["flats"]]
