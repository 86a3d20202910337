"""The norms around a block on the GPU against their fp64 definition (block_norm_reference.py).

Tolerances, u = 2^-24.  A mean over up to 16384 channels: 32 sums in a thread, at most 5 + 16
joins; its root's inverse and products 6 more: 60 u of the norm's factor, half of it through the
root.  The gate's factor is within 2^-21 = 8 u (bf16) or 6 u (fp32) relative; where z is far
below zero the exponential's argument adds |z| u.  A value passes two norms at most, forward and
again backward: below 256 u of the magnitude of its terms (the *_s of the reference), and half a
step of its type.  A weight's gradient adds the fp32 sum over the rows: rows * u of its terms'
magnitudes at most.
"""
import itertools

import pytest
import torch

import block_norm_reference as R
import linear_attention_head_gb300 as la

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF_STEP = {BF: 2.0 ** -8, F32: U}


def near(got, ref, scale, dtype, label, u=256 * U):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    tol = u * scale + HALF_STEP[dtype] * (ref.abs() + u * scale) + 1e-37
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        label, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol).max()))


def make(shape, dt, wt, gate, residual, post, pre, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)
    D = shape[-1]
    return {"x": rnd(*shape).to(dt), "gate": (2 * rnd(*shape)).to(dt) if gate else None,
            "residual": (3 * rnd(*shape)).to(dt) if residual else None,
            "post": (1 + 0.2 * rnd(D)).to(wt) if post else None,
            "pre": (1 + 0.2 * rnd(D)).to(wt) if pre else None,
            "dh": rnd(*shape).to(dt), "dy": rnd(*shape).to(dt) if pre else None}


def call(d, **kw):
    return dict(gate=d["gate"], residual=d["residual"], post_weight=d["post"],
                pre_weight=d["pre"], **kw)


def check(x, activation="silu", scale=0.7, label="", dev=None, dh=True):
    dt = x["x"].dtype
    d = dev if dev is not None else {n: t.cuda() if t is not None else None for n, t in x.items()}
    kw = dict(activation=activation, scale=scale)
    ref = R.block_norm(**{**x, "dh": x["dh"] if dh else None}, **kw)
    h, y = la.block_norm_fwd(d["x"], **call(d, **kw))
    near(h, ref["h"], ref["h_s"], dt, label + " h")
    assert (y is None) == (x["pre"] is None)
    if y is not None:
        near(y, ref["y"], ref["y_s"], dt, label + " y")
    got = la.block_norm_bwd(d["x"], d["dh"] if dh else None, d["dy"], **call(d, **kw))
    rows = x["x"].numel() // max(1, x["x"].shape[-1])
    for name, t in zip(("dx", "dgate", "dres", "dpost", "dpre"), got):
        given = {"dx": True, "dgate": x["gate"] is not None, "dres": x["residual"] is not None,
                 "dpost": x["post"] is not None, "dpre": x["pre"] is not None}[name]
        assert (t is not None) == given, (label, name)
        if not given:
            continue
        weight = name in ("dpost", "dpre")
        wt = (x["post"] if x["post"] is not None else x["pre"]).dtype if weight else dt
        near(t, ref[name], ref[name + "_s"], wt, label + " " + name,
             (256 + (rows if weight else 0)) * U)


TYPES = [(BF, BF), (BF, F32), (F32, F32)]
SHAPES = [(1, 1, 1), (2, 3, 7), (3, 5, 64), (2, 9, 3, 128), (1, 4, 2, 250), (2, 2, 256),
          (1, 7, 512), (3, 2, 1000), (1, 5, 2048), (1, 3, 4096), (2, 2, 4104), (1, 2, 8192),
          (1, 2, 16384), (1, 2, 9001)]
USES = [(g, r, a, b) for g, r, a, b in itertools.product((0, 1), repeat=4)]


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dt, wt):
    check(make(shape, dt, wt, 1, 1, 1, 1, sum(shape)), label=str(shape))
    check(make(shape, dt, wt, 0, 1, 0, 1, sum(shape)), label=str(shape), scale=1.0)


@pytest.mark.parametrize("use", USES)
@pytest.mark.parametrize("activation", ["none", "sigmoid", "silu"])
def test_uses(use, activation):
    gate, residual, post, pre = use
    for shape, dt in (((2, 5, 96), BF), ((2, 3, 37), F32)):
        x = make(shape, dt, dt, gate, residual, post, pre, 11)
        check(x, activation, label="%s" % (use,))
        if pre:
            check(x, activation, label="%s no dh" % (use,), dh=False)


@pytest.mark.parametrize("dt", [BF, F32])
def test_many_rows(dt):
    # more rows than one wave of CTAs takes at once
    check(make((2, 3001, 2, 64), dt, F32, 1, 0, 1, 0, 1), label="short rows")
    check(make((1, 1300, 1024), dt, F32, 1, 1, 1, 1, 2), label="long rows")


@pytest.mark.parametrize("dt", [BF, F32])
def test_layouts(dt):
    # slices of wider tensors (16-byte aligned or not), heads before tokens, repeated rows
    gen = torch.Generator().manual_seed(5)
    x = make((2, 6, 3, 64), dt, dt, 1, 1, 1, 1, 6)
    for shift in (0, 1):
        d = {n: t.cuda() if t is not None else None for n, t in x.items()}
        for n in ("x", "gate", "residual", "dh"):
            wide = torch.randn((2, 6, 3, 96 + shift), generator=gen).to(dt).cuda()
            wide[..., shift:64 + shift] = d[n]
            d[n] = wide[..., shift:64 + shift]
        d["dy"] = d["dy"].transpose(1, 2).contiguous().transpose(1, 2)
        check(x, label="shift %d" % shift, dev=d)
    y = make((2, 6, 3, 64), dt, dt, 1, 1, 1, 1, 6)
    y["gate"] = y["gate"][:1, :1].expand(2, 6, 3, 64)
    d = {n: t.cuda() if t is not None else None for n, t in y.items()}
    d["gate"] = y["gate"][:1, :1].contiguous().cuda().expand(2, 6, 3, 64)
    check(y, label="repeated gate", dev=d)


def test_zero_rows_and_extremes():
    x = make((1, 4, 32), F32, F32, 1, 1, 1, 1, 3)
    x["x"][0, 0] = 0
    x["residual"][0, 1] = 0
    x["gate"][0, 2] = -60.0
    x["gate"][0, 3] = 60.0
    check(x, label="zeros")
    x = make((1, 4, 32), BF, BF, 1, 0, 1, 0, 3)
    x["x"][0, 0] = 0
    x["gate"][0, 2] = -60.0
    x["gate"][0, 3] = 60.0
    check(x, label="zeros bf16")


def test_nothing_to_do():
    w = torch.ones(8, device="cuda")
    x = torch.empty((0, 5, 8), device="cuda")
    h, y = la.block_norm_fwd(x, residual=x, pre_weight=w)
    assert h.shape == y.shape == x.shape
    g = la.block_norm_bwd(x, x, x, residual=x, pre_weight=w, post_weight=w)
    assert torch.equal(g[3], torch.zeros_like(w)) and torch.equal(g[4], torch.zeros_like(w))


def test_in_place():
    x = make((2, 5, 200), BF, BF, 1, 1, 1, 1, 9)
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    h, y = la.block_norm_fwd(d["x"], **call(d))
    for name in ("residual", "x"):
        e = {n: t.clone() if t is not None else None for n, t in d.items()}
        h2, y2 = la.block_norm_fwd(e["x"], **call(e), out=(e[name], None))
        assert h2.data_ptr() == e[name].data_ptr()
        assert torch.equal(h2, h) and torch.equal(y2, y)


def test_same_bits_again():
    # the weights' gradients are summed in a fixed order
    x = make((4, 500, 512), BF, F32, 1, 1, 1, 1, 4)
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    first = la.block_norm_bwd(d["x"], d["dh"], d["dy"], **call(d))
    for _ in range(3):
        for a, b in zip(first, la.block_norm_bwd(d["x"], d["dh"], d["dy"], **call(d))):
            assert torch.equal(a, b)


def test_autograd():
    x = make((2, 4, 40), F32, F32, 1, 1, 1, 1, 8)
    leaves = {n: x[n].cuda().requires_grad_() for n in ("x", "gate", "residual", "post", "pre")}
    kw = dict(activation="sigmoid", scale=0.5)
    dh, dy = x["dh"].cuda(), x["dy"].cuda()
    for parts in ("hy", "h", "y"):
        h, y = la.block_norm(leaves["x"], leaves["gate"], leaves["residual"], leaves["post"],
                             leaves["pre"], **kw)
        loss = (h * dh).sum() if "h" in parts else 0
        loss = loss + ((y * dy).sum() if "y" in parts else 0)
        for t in leaves.values():
            t.grad = None
        loss.backward()
        ref = R.block_norm(**{**x, "dh": x["dh"] if "h" in parts else torch.zeros_like(x["dh"]),
                              "dy": x["dy"] if "y" in parts else torch.zeros_like(x["dy"])}, **kw)
        for n, g in (("x", "dx"), ("gate", "dgate"), ("residual", "dres"), ("post", "dpost"),
                     ("pre", "dpre")):
            near(leaves[n].grad, ref[g], ref[g + "_s"], F32, "%s %s" % (parts, g), 300 * U)
    # a gate of one row for all tokens: its gradient is the sum over them
    gate = torch.randn(1, 1, 40, device="cuda", requires_grad=True)
    h, _ = la.block_norm(leaves["x"], gate.expand(2, 4, 40), post_weight=leaves["post"])
    h.backward(dh)
    ref = R.block_norm(x["x"], gate.detach().cpu().expand(2, 4, 40), post=x["post"], dh=x["dh"])
    near(gate.grad, ref["dgate"].sum((0, 1), keepdim=True),
         ref["dgate_s"].sum((0, 1), keepdim=True), F32, "broadcast gate")


def test_captured():
    x = make((2, 64, 256), BF, F32, 1, 1, 1, 1, 2)
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    run = lambda: (la.block_norm_fwd(d["x"], **call(d)) +
                   la.block_norm_bwd(d["x"], d["dh"], d["dy"], **call(d)))
    want = run()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.zero_()
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 5, 2, 64), (1, 3, 250), (2, 3, 7), (1, 1, 16)])
def test_no_eps_and_fewer_rows_than_groups(shape, dt):
    # eps 0: the groups of a CTA that have no row add nothing to the weights' gradients
    x = make(shape, dt, F32, 1, 1, 1, 1, 21)
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    ref = R.block_norm(**x, eps=0.0)
    got = la.block_norm_bwd(d["x"], d["dh"], d["dy"], **call(d, eps=0.0))
    rows = x["x"].numel() // shape[-1]
    for name, t in zip(("dx", "dgate", "dres", "dpost", "dpre"), got):
        weight = name in ("dpost", "dpre")
        near(t, ref[name], ref[name + "_s"], F32 if weight else dt, "%s %s" % (shape, name),
             (256 + (rows if weight else 0)) * U)
