"""The operators beside the attention on the GPU against their fp64 definitions
(layer_reference.py): the gated recurrence and the norms with the rotation, forward and
backward, each alone and in a run together with the attention.

Tolerances.  An output rounded to its type is off by at most half a step (bf16 2^-8, fp32
2^-24, relative to the value).  Before it, the recurrence in fp32 makes at most 8 relative
roundings of u = 2^-24 a token of the running magnitude.  The decay a enters with a times its
relative error: for |g| < 1/4 below 2 u (a series whose last addition rounds); else 2^x within
4 u and its argument's rounding, |g| u, so a (4 + |g|) u <= 3.4 u, the most at |g| = 1/4.  The
token's own sum in each of the two passes over it, the product of decays: 3 u.  The joins of
16 (or 8) tokens to a thread's map, of those to a tile's and to the state: fewer than 12 for
those tokens together, below 1.5 u each.  layer_reference.scan carries them on as the
recurrence does (the *_e scales).  The rotation: sin and cos within 2^-22 (the angle's fraction
of a turn kept to 2^-32; its remainder as fp32 and the series' last steps 3 u), the norm's
factor within 2^-22 (a sum of up to 256 squares by 8 and then pairwise, the root, the product:
13 + 2 roundings of 2^-24), three products: together below 2^-20 of the pair's magnitude, which
the row's largest value times sqrt 2 bounds.
"""
import math

import pytest
import torch

import layer_reference as R
import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import _native as N

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCAN_U = 8 * R.U
ROT_U = 2.0 ** -20 * math.sqrt(2.0)


def _close(got, ref, scale, dtype, label):
    """|got - ref| within the arithmetic's scale and half a step of the rounded value."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    tol = scale + R.HALF_STEP[dtype] * (ref.abs() + scale) + 1e-37
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        label, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol).max()))


# ---------------------------------------------------------------------------
# gated recurrence

def _scan_inputs(B, T, H, D, dt, gt, n, seed, state=True, near=0.7):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, H, D), generator=gen).to(dt)
    # forget gates from a few tokens to thousands of tokens of memory
    z = torch.randn((B, T, H, D), generator=gen) + 8 * near * torch.rand((H, D), generator=gen)
    g = torch.nn.functional.logsigmoid(z).to(gt)
    do = torch.randn((B, T, H, D), generator=gen).to(dt)
    init = torch.randn((n, H, D), generator=gen) if state else None
    dfin = torch.randn((n, H, D), generator=gen) if state else None
    return x, g, do, init, dfin


def _cuda(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def _scan_check(x, g, do, init, dfin, reverse=False, cu=None, label="", dev=None):
    """Forward and backward (with the forward's states, and without) against the definition."""
    dt, gt = x.dtype, g.dtype
    ref = R.scan(x, g, init, reverse, cu, do, dfin)
    xd, gd, dod, initd, dfind = dev if dev is not None else _cuda(x, g, do, init, dfin)
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    kw = dict(reverse=reverse, cu_seqlens=cu_t.cuda() if cu is not None else None,
              cu_seqlens_host=cu_t)
    o, fin, states = la.gated_scan_fwd(xd, gd, initd, keep_states=True, **kw)
    _close(o, ref["o"], SCAN_U * ref["o_e"], dt, label + " o")
    _close(fin, ref["final"], SCAN_U * ref["final_e"], F32, label + " final_state")
    plain = la.gated_scan_fwd(xd, gd, initd, **kw)
    assert torch.equal(plain[0], o) and torch.equal(plain[1], fin)
    got = la.gated_scan_bwd(xd, gd, dod, initd, dfind, states=states, **kw)
    for name, t, d in zip(("dx", "dg", "dinit"), got, (dt, gt, F32)):
        _close(t, ref[name], SCAN_U * ref[name + "_e"], d, label + " " + name)
    again = la.gated_scan_bwd(xd, gd, dod, initd, dfind, **kw)
    for a, b in zip(got, again):
        assert torch.equal(a, b), label + ": the recomputed states differ"
    torch.cuda.synchronize()
    la.get_device_error()


TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("B,T,H,D", [
    (1, 1, 1, 1), (5, 1, 2, 128), (2, 2, 1, 4), (3, 15, 2, 64), (2, 16, 1, 128), (3, 17, 2, 64),
    (2, 127, 1, 32), (1, 128, 2, 33), (2, 129, 1, 256), (3, 300, 5, 36), (1, 700, 1, 250)])
def test_scan_dense(B, T, H, D, dt, gt):
    for reverse in (False, True):
        x, g, do, init, dfin = _scan_inputs(B, T, H, D, dt, gt, B, 10 * T + D, state=not reverse)
        _scan_check(x, g, do, init, dfin, reverse, label="%s rev %d" % ((B, T, H, D), reverse))


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_long(dt, gt, reverse):
    # dozens of tiles, in segments: the maps of those before a segment give its state
    x, g, do, init, dfin = _scan_inputs(1, 9001, 1, 8, dt, gt, 1, 3)
    _scan_check(x, g, do, init, dfin, reverse, label="long")


PACKS = [
    [0, 5], [0, 0, 0, 7, 7, 8, 9, 9], [0, 128, 256, 257, 384, 640], [0, 300, 301, 301, 1000],
    [0, 1, 2, 3, 4, 5, 130, 131, 132, 600], list(range(0, 41)), [0, 4500, 4500, 4700, 9001, 9001],
]


@pytest.mark.parametrize("dt,gt", [(BF, F32), (F32, F32)])
@pytest.mark.parametrize("pack", range(len(PACKS)))
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_packed(pack, dt, gt, reverse):
    cu = PACKS[pack]
    T, H, D = cu[-1], 2, 12
    for state in (True, False):
        x, g, do, init, dfin = _scan_inputs(1, T, H, D, dt, gt, len(cu) - 1, pack, state)
        _scan_check(x, g, do, init, dfin, reverse, cu, label="pack %d" % pack)


def test_scan_many_short_sequences():
    # more sequences than one dimension of a launch grid holds, most of one token, some empty
    n = 70000
    lens = torch.ones(n, dtype=torch.int64)
    lens[::7] = 0
    lens[3] = 40
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    T = int(cu[-1])
    x, g, do, init, dfin = _scan_inputs(1, T, 1, 4, F32, F32, n, 5)
    xd, gd, dod, initd, dfind = _cuda(x, g, do, init, dfin)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    o, fin = la.gated_scan_fwd(xd, gd, initd, **kw)
    dx, dg, dinit = la.gated_scan_bwd(xd, gd, dod, initd, dfind, **kw)
    ref = R.scan(x, g, init, False, cu.tolist(), do, dfin)
    for t, name, scale in ((o, "o", "o_e"), (fin, "final", "final_e"), (dx, "dx", "dx_e"),
                           (dg, "dg", "dg_e"), (dinit, "dinit", "dinit_e")):
        _close(t, ref[name], SCAN_U * ref[scale], F32, name)


@pytest.mark.parametrize("D,dt,gt,reverse", [
    (3, BF, F32, False), (8, BF, BF, True), (8, F32, F32, False), (3, F32, F32, True)])
def test_scan_many_sequences_of_some_tokens(D, dt, gt, reverse):
    # so many that a thread takes a sequence alone, in several blocks of tokens: whole blocks,
    # a last one of one token, sequences without tokens; dense too
    lens = [0, 1, 8, 9, 16, 17, 20] * 220
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x, g, do, init, dfin = _scan_inputs(1, cu[-1], 1, D, dt, gt, len(lens), 21)
    _scan_check(x, g, do, init, dfin, reverse, cu, label="packed")
    x, g, do, init, dfin = _scan_inputs(1400, 17, 1, D, dt, gt, 1400, 22, state=not reverse)
    _scan_check(x, g, do, init, dfin, reverse, label="dense")


@pytest.mark.parametrize("B,T,H,D", [
    (2, 1500, 2, 64), (3, 300, 4, 6), (2, 140, 8, 250), (1, 2500, 1, 200), (2, 400, 3, 33)])
@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_rows_of_all_heads(B, T, H, D, dt, gt, reverse):
    # heads whose channels are one row together, whatever a head's own width; several rows
    x, g, do, init, dfin = _scan_inputs(B, T, H, D, dt, gt, B, 23)
    _scan_check(x, g, do, init, dfin, reverse, label="%s" % ((B, T, H, D),))


@pytest.mark.parametrize("H,dt,gt", [(40, BF, BF), (50, F32, F32), (80, BF, F32), (100, BF, BF)])
@pytest.mark.parametrize("cu", [None, [0, 900], [0, 1, 130, 130, 900]])
def test_scan_chains_of_several_teams(H, dt, gt, cu):
    # 64 to 300 chains (sequences x 64 channels): two or four teams take a chain's tiles in
    # turn, whole and ragged runs, rows of 16-byte pieces and (D 127) others
    B, T, D = (1, 900, 128) if H != 50 else (1, 900, 127)
    n = 1 if cu is None else len(cu) - 1
    x, g, do, init, dfin = _scan_inputs(B, T, H if n == 1 else H // 2, D, dt, gt, n, 28)
    _scan_check(x, g, do, init, dfin, H == 80, cu, label="%d heads" % H)


@pytest.mark.parametrize("dt,gt", [(BF, F32), (F32, F32)])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("D", [64, 72, 192])
def test_scan_head_major_in_segments(D, dt, gt, reverse):
    # heads apart, in tiles that are whole heads' parts (64, 192) or cross them (72), packed
    cu = [0, 700, 701, 2000]
    x, g, do, init, dfin = _scan_inputs(1, 2000, 2, D, dt, gt, 3, 24)
    dev = [_relayout(t, "head_major") for t in (x, g, do)] + _cuda(init, dfin)
    _scan_check(x, g, do, init, dfin, reverse, cu, label="head major", dev=dev)


def test_scan_rows_far_apart():
    # offsets beyond 2^31 elements, between batch rows and between tokens (whose distance is
    # beyond the steps that fit 32 bits of bytes)
    x, g, do, init, dfin = _scan_inputs(2, 150, 1, 64, BF, BF, 2, 25)
    far = 1 << 31
    big = torch.empty(far + 150 * 64, dtype=BF, device="cuda")
    xd = big.as_strided((2, 150, 1, 64), (far, 64, 64, 1))
    xd.copy_(x)
    _scan_check(x, g, do, init, dfin, label="rows", dev=[xd] + _cuda(g, do, init, dfin))
    del xd, big
    step = (1 << 24) + 8
    big = torch.empty(149 * step + 64, dtype=BF, device="cuda")
    out = big.as_strided((1, 150, 1, 64), (0, step, 64, 1))
    for reverse in (False, True):
        want, _ = la.gated_scan_fwd(x[:1].cuda(), g[:1].cuda(), reverse=reverse)
        got, _ = la.gated_scan_fwd(x[:1].cuda(), g[:1].cuda(), reverse=reverse, out=out)
        assert torch.equal(got, want)
    out.copy_(x[:1])
    for reverse in (False, True):
        want, _ = la.gated_scan_fwd(x[:1].cuda(), g[:1].cuda(), reverse=reverse)
        got, _ = la.gated_scan_fwd(out, g[:1].cuda(), reverse=reverse)
        assert torch.equal(got, want)


def test_scan_and_norms_from_threads():
    # two host threads, each on its own stream, the same inputs: the results of one alone
    import threading
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 3000, 2, 64, BF, F32, 1, 26))
    q, k, dq, dk, qw, kw = _cuda(*_rope_inputs(1, 700, 4, 2, 64, BF, 27))
    rope = la.Rope(la.rope_inv_freq(64))

    def calls():
        y = la.gated_scan_fwd(x, g, init, keep_states=True)
        z = la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw, rope=rope)
        return y + la.gated_scan_bwd(x, g, do, init, dfin, states=y[2])[:2] + z
    want = calls()
    torch.cuda.synchronize()
    got, threads = [None, None], []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = calls()
    for i in range(2):
        threads.append(threading.Thread(target=work, args=(i,)))
        threads[-1].start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    la.get_device_error()
    for r in got:
        # (the states of first tiles are not written)
        assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(r, want)) if i != 2)


def _relayout(t, kind):
    """The same values on the GPU in another layout."""
    B, T, H, D = t.shape
    if kind == "head_major":
        return t.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "odd_rows":       # rows of odd length, base off by one element: no wide loads
        big = torch.full((B, T, H, D + 3), float("nan"), dtype=t.dtype, device="cuda")
        big[..., 1:D + 1] = t.cuda()
        return big[..., 1:D + 1]
    if kind == "sliced":         # a part of a fused projection
        big = torch.full((B, T, 3 * H, D), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :, H:2 * H] = t.cuda()
        return big[:, :, H:2 * H]
    if kind == "channels_apart":
        return t.cuda().transpose(2, 3).contiguous().transpose(2, 3)
    return t.cuda()


@pytest.mark.parametrize("kind", ["head_major", "odd_rows", "sliced", "channels_apart"])
@pytest.mark.parametrize("dt,gt", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("T", [7, 260])
def test_scan_layouts(kind, dt, gt, T):
    x, g, do, init, dfin = _scan_inputs(2, T, 3, 40, dt, gt, 2, 7)
    dev = [_relayout(t, kind) for t in (x, g, do)] + _cuda(init, dfin)
    _scan_check(x, g, do, init, dfin, label=kind, dev=dev)
    # outputs into a strided buffer, other bytes of it untouched
    buf = torch.full((2, T, 3, 43), 7.0, dtype=dt, device="cuda")
    o, _ = la.gated_scan_fwd(dev[0], dev[1], dev[3], out=buf[..., 1:41])
    want, _ = la.gated_scan_fwd(dev[0], dev[1], dev[3])
    assert torch.equal(buf[..., 1:41], want)
    assert bool((buf[..., :1] == 7).all()) and bool((buf[..., 41:] == 7).all())


def test_scan_repeated_inputs_and_their_gradients():
    # one gate for all batch rows (stride 0) and one input for all heads: the gradients of a
    # repeated input are its uses' sum
    x, g, do, init, dfin = _scan_inputs(3, 200, 2, 16, F32, F32, 3, 8)
    xl = x[:, :, :1].cuda().requires_grad_()
    gl = g[:1].cuda().requires_grad_()
    o, fin = la.gated_scan(xl.expand(-1, -1, 2, -1), gl.expand(3, -1, -1, -1), init.cuda())
    dx, dg = torch.autograd.grad((o, fin), (xl, gl), (do.cuda(), dfin.cuda()))
    ref = R.scan(x[:, :, :1].expand_as(x), g[:1].expand_as(g), init, False, None, do, dfin)
    _close(dx, ref["dx"].sum(2, keepdim=True), SCAN_U * ref["dx_e"].sum(2, keepdim=True) +
           2 * R.U * ref["dx"].abs().sum(2, keepdim=True), F32, "dx")
    _close(dg, ref["dg"].sum(0, keepdim=True), SCAN_U * ref["dg_e"].sum(0, keepdim=True) +
           3 * R.U * ref["dg"].abs().sum(0, keepdim=True), F32, "dg")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_keeps_sequences_apart(bad, reverse):
    # a sequence full of NaN or infinities leaves its neighbours in the same tile as they were
    cu = [0, 50, 90, 130, 300, 320]
    x, g, do, init, dfin = _scan_inputs(1, 320, 1, 8, F32, F32, 5, 9)
    cut = torch.tensor(cu, dtype=torch.int32)
    kw = dict(reverse=reverse, cu_seqlens=cut.cuda(), cu_seqlens_host=cut)
    run = lambda t: (la.gated_scan_fwd(t[0], t[1], t[3], **kw) +
                     la.gated_scan_bwd(t[0], t[1], t[2], t[3], t[4], **kw))
    clean = run(_cuda(x, g, do, init, dfin))
    for seq in (1, 3):
        lo, hi = cu[seq], cu[seq + 1]
        y = [t.clone() for t in (x, g, do, init, dfin)]
        for t in y[:3]:
            t[:, lo:hi] = bad
        y[3][seq] = bad
        y[4][seq] = bad
        dirty = run(_cuda(*y))
        keep = torch.ones(320, dtype=torch.bool)
        keep[lo:hi] = False
        rest = [i for i in range(5) if i != seq]
        for name, a, b in zip(("o", "fin", "dx", "dg", "dinit"), clean, dirty):
            a, b = a.cpu(), b.cpu()
            if name in ("fin", "dinit"):
                assert torch.equal(a[rest], b[rest]), (name, seq)
            else:
                assert torch.equal(a[:, keep], b[:, keep]), (name, seq)


def test_scan_spreads_nan_and_infinities_as_the_definition():
    x, g, do, init, dfin = _scan_inputs(1, 400, 1, 6, F32, F32, 1, 12)
    x[0, 37, 0, 0] = float("inf")
    x[0, 90, 0, 1] = float("nan")
    x[0, 20, 0, 2], x[0, 300, 0, 2] = float("inf"), -float("inf")     # inf - inf = nan
    init[0, 0, 3] = -float("inf")
    g[0, :, 0, 4] = -1000.0             # exp underflows: every token starts anew
    g[0, 200, 0, 5] = -float("inf")     # the state is forgotten at once
    o, fin = la.gated_scan_fwd(*_cuda(x, g, init))
    ref = R.scan(x, g, init)
    o = o.cpu().double()
    assert torch.equal(o.isnan(), ref["o"].isnan())
    assert torch.equal(o.isinf(), ref["o"].isinf())
    ok = ref["o"].isfinite()
    assert torch.equal(o[~ok & ~o.isnan()], ref["o"][~ok & ~o.isnan()])
    assert torch.allclose(o[ok], ref["o"][ok], rtol=1e-4, atol=1e-5)
    assert torch.equal(o[0, :, 0, 4].float(), x[0, :, 0, 4])
    assert o[0, 200, 0, 5] == x[0, 200, 0, 5]


def test_scan_state_in_place_and_carried_on():
    # final_state may be initial_state; a sequence cut in two continues from the state
    x, g, _, init, _ = _scan_inputs(2, 333, 2, 24, BF, BF, 2, 13)
    xd, gd, s = _cuda(x, g, init)
    whole, fin = la.gated_scan_fwd(xd, gd, s.clone())
    for cut in (1, 16, 128, 200, 332):
        state = s.clone()
        a, st = la.gated_scan_fwd(xd[:, :cut], gd[:, :cut], state, final_state=state)
        assert st.data_ptr() == state.data_ptr()
        b, _ = la.gated_scan_fwd(xd[:, cut:], gd[:, cut:], state, final_state=state)
        # the same arithmetic in other tiles: within the roundings, then one bf16 step apart
        ref = R.scan(x, g, init)
        _close(torch.cat((a, b), 1), ref["o"], SCAN_U * ref["o_e"], BF, "cut %d" % cut)
        _close(state, ref["final"], SCAN_U * ref["final_e"], F32, "cut %d" % cut)
    # packed sequences shorter than a tile, updated in place
    cu = torch.tensor([0, 3, 3, 100, 333], dtype=torch.int32)
    p = torch.randn(4, 2, 24, device="cuda")
    want = la.gated_scan_fwd(xd[:1], gd[:1], p.clone(), cu_seqlens=cu.cuda())[1]
    la.gated_scan_fwd(xd[:1], gd[:1], p, cu_seqlens=cu.cuda(), final_state=p)
    assert torch.equal(p, want)


def test_scan_is_deterministic_and_takes_any_stream():
    x, g, do, init, dfin = _cuda(*_scan_inputs(2, 5000, 4, 64, BF, BF, 2, 14))
    run = lambda: la.gated_scan_fwd(x, g, init) + la.gated_scan_bwd(x, g, do, init, dfin)
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):      # two calls at once, each with its workspace
            other = run()
        here = run()
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, here):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_scan_withheld_tile_reports_timeout_and_context_survives():
    # a CTA's first tile is not handed over: its team waits, at most two seconds, and the call
    # reports it; the next call is right
    import time
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 6000, 1, 64, BF, BF, 1, 16))
    want = la.gated_scan_fwd(x, g, init) + la.gated_scan_bwd(x, g, do, init, dfin)
    la.get_device_error()
    _, _, states = la.gated_scan_fwd(x, g, init, keep_states=True)
    for call in (lambda: la.gated_scan_fwd(x, g, init),
                 lambda: la.gated_scan_bwd(x, g, do, init, dfin, states=states)):
        N.check(N.lib().la_debug_withhold_next_handoff(1))
        t0 = time.time()
        call()
        with pytest.raises(N.LaError) as err:
            la.get_device_error()
        assert err.value.status == N.LA_ERR_TIMEOUT and time.time() - t0 < 30
        la.get_device_error()
        got = la.gated_scan_fwd(x, g, init) + la.gated_scan_bwd(x, g, do, init, dfin)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        la.get_device_error()


def test_scan_withheld_tile_among_teams_that_wait_for_one_another():
    # the same where several teams take a chain's tiles in turn: all of them stop
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 900, 50, 128, BF, BF, 1, 17))
    want = la.gated_scan_fwd(x, g, init)
    la.get_device_error()
    N.check(N.lib().la_debug_withhold_next_handoff(1))
    la.gated_scan_fwd(x, g, init)
    with pytest.raises(N.LaError) as err:
        la.get_device_error()
    assert err.value.status == N.LA_ERR_TIMEOUT
    got = la.gated_scan_fwd(x, g, init)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    la.get_device_error()


def test_scan_refuses_foreign_states():
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 300, 1, 8, F32, F32, 1, 15))
    with pytest.raises(ValueError, match="states"):
        la.gated_scan_bwd(x, g, do, init, dfin, states=torch.zeros(5, device="cuda"))
    with pytest.raises(TypeError, match="g must have"):
        la.gated_scan_fwd(x, g.bfloat16())
    with pytest.raises(ValueError, match="initial_state"):
        la.gated_scan_fwd(x, g, init[:, :, :4])
    with pytest.raises(ValueError, match="out must"):
        la.gated_scan_fwd(x, g, out=x.bfloat16())


# ---------------------------------------------------------------------------
# norms and rotation

def _rope_inputs(B, T, Hq, Hk, D, dt, seed, weights=True, wdt=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    q, k, dq, dk = (r(B, T, h, D).to(dt) for h in (Hq, Hk, Hq, Hk))
    w = [(1 + 0.2 * r(D)).to(wdt or dt) for _ in range(2)] if weights else [None, None]
    return q, k, dq, dk, w[0], w[1]


def _row_scale(x):
    return x.abs().amax(-1, keepdim=True).expand_as(x)


def _rope_check(q, k, dqo, dko, qw, kw, rope, pos, kwargs, normalize=True, eps=1e-6, label="",
                dev=None):
    """Forward, backward and the weights' gradients; pos: the positions [axes, B, T] (fp64
    reference); kwargs: how the call is given them."""
    dt = q.dtype
    freq = rope.inv_freq.cpu() if rope is not None else None
    ref_kw = dict(eps=eps, normalize=normalize, inv_freq=freq,
                  axes=rope.axes if rope is not None else None, positions=pos,
                  interleaved=rope.interleaved if rope is not None else False)
    qd, kd, dqd, dkd = dev if dev is not None else _cuda(q, k, dqo, dko)
    qwd, kwd = _cuda(qw, kw)
    args = dict(rope=rope, **kwargs)
    if normalize:
        args.update(q_weight=qwd, k_weight=kwd, eps=eps)
        ys = la.qk_norm_rope_fwd(qd, kd, **args)
        got = la.qk_norm_rope_bwd(qd, kd, dqd, dkd, **args)
    else:
        ys = la.rotary_fwd(qd, kd, **args)
        got = la.rotary_bwd(dqd, dkd, **args)
    for i, (x, dy, w, name) in enumerate(((q, dqo, qw, "q"), (k, dko, kw, "k"))):
        xr = x.double().requires_grad_()
        wr = w.double().requires_grad_() if w is not None else None
        y = R.norm_rope(xr, wr, **ref_kw)
        grads = torch.autograd.grad(y, (xr,) + ((wr,) if wr is not None else ()), dy.double())
        _close(ys[i], y.detach(), ROT_U * _row_scale(y.detach()), dt, label + " " + name)
        # dx = r (z - x r^2 mean(z x)): the roundings of z and of the mean, times the factors
        rr = 1 / torch.sqrt((xr * xr).mean(-1, keepdim=True) + eps).detach() if normalize else 1.0
        wmax = float(w.abs().max()) if w is not None else 1.0
        n = (xr.detach() * rr).abs().amax(-1, keepdim=True) if normalize else 0.0
        size = _row_scale(dy.double()) * wmax * rr * (1 + n * n)
        _close(got[i], grads[0], 4 * ROT_U * size, dt, label + " d" + name)
        if w is not None and normalize:
            # fp32 sums of every row's term: each term's own roundings, and at most 88
            # additions on any path from a term to the sum (a lane's rows: 12, the CTA's lanes:
            # 32, a slice's CTAs: 4, the slices: 32)
            terms = (_row_scale(dy.double()) * (xr.detach() * rr).abs()).sum((0, 1, 2))
            _close(got[2 + i], grads[1], (ROT_U + 88 * R.U) * terms, w.dtype,
                   label + " d%s_weight" % name)
    la.get_device_error()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,rot,interleaved", [
    (2, 2, False), (16, 16, False), (33, 32, True), (40, 24, False), (64, 64, False),
    (64, 64, True), (96, 96, False), (128, 128, False), (128, 128, True), (128, 64, False),
    (128, 38, True), (192, 192, False), (192, 96, True), (250, 130, False), (256, 256, False),
    (256, 256, True)])
def test_norm_rotation_widths(D, rot, interleaved, dt):
    B, T, Hq, Hk = 2, 9, 6, 3
    q, k, dq, dk, qw, kw = _rope_inputs(B, T, Hq, Hk, D, dt, D + rot)
    rope = la.Rope(la.rope_inv_freq(rot), interleaved=interleaved)
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(B, T, None), {},
                label="%d/%d" % (D, rot))
    _rope_check(q, k, dq, dk, None, None, rope, R.positions_of(B, T, None), {}, normalize=False,
                label="rotary %d/%d" % (D, rot))


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, BF)])
def test_norms_without_rotation_and_weight_types(dt, wdt):
    q, k, dq, dk, qw, kw = _rope_inputs(3, 5, 4, 4, 128, dt, 3, wdt=wdt)
    _rope_check(q, k, dq, dk, qw, kw, None, None, {}, label="norms")
    _rope_check(q, k, dq, dk, None, kw, None, None, {}, eps=0.1, label="one weight")
    _rope_check(q, k, dq, dk, qw, None, None, None, {}, eps=0.0, label="other weight")


@pytest.mark.parametrize("Hq,Hk,B,T", [(1, 1, 1, 1), (40, 8, 1, 1), (7, 1, 33, 1), (3, 3, 2, 500),
                                       (32, 8, 3, 37), (12, 12, 1, 2047)])
def test_norm_rotation_counts(Hq, Hk, B, T):
    q, k, dq, dk, qw, kw = _rope_inputs(B, T, Hq, Hk, 64, BF, Hq * T)
    rope = la.Rope(la.rope_inv_freq(64))
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(B, T, None), {})


@pytest.mark.parametrize("ptype", [torch.int32, torch.int64])
def test_rotation_at_far_and_negative_positions(ptype):
    # the turns wrap exactly: fp32 products would be off by whole radians here
    B, T = 3, 5
    q, k, dq, dk, _, _ = _rope_inputs(B, T, 2, 2, 64, F32, 21)
    pos = torch.tensor([0, -1, 131071, 2 ** 31 - 1, -2 ** 31, 123456789, 7, -77777, 2 ** 24 + 1,
                        1, 2, 3, 4, 5, 2 ** 30], dtype=torch.int64).reshape(1, B, T)
    # frequencies that fp64 holds exactly, so that the reference's angles are exact products
    # of 53 bits: the reference itself is then off by 2^31 2^-53 radians
    freq = torch.tensor([2.0 ** -j for j in range(32)], dtype=torch.float64)
    rope = la.Rope(freq.cuda())
    given = pos.to(ptype).cuda()
    for p in (given, given[0]):
        _rope_check(q, k, dq, dk, None, None, rope, pos, dict(positions=p), normalize=False)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rotation_with_several_axes(axes, dt):
    B, T, D = 2, 24, 64
    gen = torch.Generator().manual_seed(axes)
    q, k, dq, dk, qw, kw = _rope_inputs(B, T, 4, 2, D, dt, axes)
    freq = la.rope_inv_freq(D)
    pos = torch.randint(0, 3000, (axes, B, T), generator=gen)
    cuts = [5, 7, 9, 32][:axes - 1]
    sections = tuple(cuts) + (32 - sum(cuts),) if axes < 4 else (5, 7, 9, 11)
    mixed = [j % axes for j in range(32)]
    for interleaved in (False, True):
        for rope in (la.Rope(freq, sections=sections, interleaved=interleaved),
                     la.Rope(freq, axes=mixed, interleaved=interleaved)):
            p = pos.to(torch.int32).cuda()
            _rope_check(q, k, dq, dk, qw, kw, rope, pos, dict(positions=p), label="norm")
            _rope_check(q, k, dq, dk, None, None, rope, pos, dict(positions=p),
                        normalize=False, label="rotary")
    # one grid for all batch rows, and an axis-last tensor seen through its strides
    one = pos[:, :1].to(torch.int64).cuda()
    want = pos[:, :1].expand(-1, B, -1)
    _rope_check(q, k, dq, dk, qw, kw, rope, want, dict(positions=one))
    last = pos.permute(1, 2, 0).contiguous().to(torch.int32).cuda().permute(2, 0, 1)
    _rope_check(q, k, dq, dk, qw, kw, rope, pos, dict(positions=last))


@pytest.mark.parametrize("cu", [[0, 4, 4, 5, 60], [0, 0, 0, 33], list(range(0, 51))])
def test_norm_rotation_packed(cu):
    T = cu[-1]
    q, k, dq, dk, qw, kw = _rope_inputs(1, T, 4, 2, 128, BF, T)
    rope = la.Rope(la.rope_inv_freq(128))
    cut = torch.tensor(cu, dtype=torch.int32)
    off = torch.arange(len(cu) - 1, dtype=torch.int32) * 1000
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(1, T, cu),
                dict(cu_seqlens=cut.cuda(), cu_seqlens_host=cut))
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(1, T, cu, off),
                dict(cu_seqlens=cut.cuda(), cu_seqlens_host=cut, position_offset=off.cuda()))
    # decoding on: one token a row, each row at its offset
    q, k, dq, dk, qw, kw = _rope_inputs(len(off), 1, 4, 2, 128, BF, T)
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(len(off), 1, None, off),
                dict(position_offset=off.cuda()))


@pytest.mark.parametrize("kind", ["head_major", "odd_rows", "sliced", "channels_apart"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_rotation_layouts(kind, dt):
    B, T = 2, 19
    q, k, dq, dk, qw, kw = _rope_inputs(B, T, 4, 4, 64, dt, 4)
    rope = la.Rope(la.rope_inv_freq(64))
    dev = [_relayout(t, kind) for t in (q, k, dq, dk)]
    _rope_check(q, k, dq, dk, qw, kw, rope, R.positions_of(B, T, None), {}, dev=dev)
    # q from one layout, k from another; outputs in place
    qd, kd = _relayout(q, kind), k.cuda()
    want = la.qk_norm_rope_fwd(qd, kd, rope=rope)
    if kind != "channels_apart":
        got = la.qk_norm_rope_fwd(qd, kd, rope=rope, out=(qd, kd))
        assert got[0].data_ptr() == qd.data_ptr()
        assert torch.equal(qd, want[0]) and torch.equal(kd, want[1])
    # one tensor alone
    alone = la.qk_norm_rope_fwd(_relayout(q, kind), rope=rope)
    assert torch.equal(alone, want[0])


def test_norm_of_zero_and_large_rows():
    # a row of zeros stays zero (eps), its gradient finite; large rows do not overflow in the
    # factors
    q = torch.zeros(1, 3, 1, 64)
    q[0, 1] = 1e18
    q[0, 2] = torch.randn(64)
    dy = torch.randn(1, 3, 1, 64)
    qd = q.cuda()
    y = la.qk_norm_rope_fwd(qd)
    dq = la.qk_norm_rope_bwd(qd, None, dy.cuda())[0]
    assert bool((y[0, 0] == 0).all()) and bool(torch.isfinite(y).all())
    assert torch.allclose(y[0, 1].cpu(), torch.ones(1, 64))
    assert torch.allclose(dq[0, 0].cpu(), dy[0, 0] * 1e3, rtol=1e-5)
    assert bool(torch.isfinite(dq).all())


def test_norm_rotation_keeps_rows_apart():
    # NaN and infinities stay in their row
    q, k, dq, dk, qw, kw = _cuda(*_rope_inputs(2, 5, 3, 3, 64, F32, 6))
    rope = la.Rope(la.rope_inv_freq(64))
    clean = la.qk_norm_rope_fwd(q, k, qw, kw, rope=rope)
    cg = la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw, rope=rope)
    for bad in (float("nan"), float("inf")):
        q2, dq2 = q.clone(), dq.clone()
        q2[0, 1, 2, 5] = bad
        dq2[1, 3, 0, 7] = bad
        y = la.qk_norm_rope_fwd(q2, k, qw, kw, rope=rope)
        g = la.qk_norm_rope_bwd(q2, k, dq2, dk, qw, kw, rope=rope)
        keep = torch.ones(2, 5, 3, dtype=torch.bool, device="cuda")
        keep[0, 1, 2] = False
        assert torch.equal(y[0][keep], clean[0][keep]) and torch.equal(y[1], clean[1])
        keep[1, 3, 0] = False
        assert torch.equal(g[0][keep], cg[0][keep]) and torch.equal(g[1], cg[1])
        assert torch.equal(g[3], cg[3])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 32), (36, 10)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rotation_leaves_the_other_channels_alone(D, rot, interleaved, dt):
    # NaN and infinities in rotated channels stay in their pair, so do those of the others
    q, k, dq, dk, _, _ = _cuda(*_rope_inputs(1, 9, 3, 2, D, dt, 12))
    rope = la.Rope(la.rope_inv_freq(rot), interleaved=interleaved)
    for call, x, y in ((la.rotary_fwd, q, k), (la.rotary_bwd, dq, dk)):
        clean = call(x, y, rope=rope)[0]
        for c in (0, rot - 1, rot, D - 1):
            for bad in (float("nan"), float("inf")):
                z = x.clone()
                z[0, 4, 1, c] = bad
                got = call(z, y, rope=rope)[0]
                keep = torch.ones_like(z, dtype=torch.bool)
                keep[0, 4, 1, c] = False
                if c < rot:
                    keep[0, 4, 1, c ^ 1 if interleaved else (c + rot // 2) % rot] = False
                assert torch.equal(got[keep], clean[keep]), (c, bad)


def test_norm_rotation_rows_far_apart():
    # offsets beyond 2^31 elements, between batch rows and between heads
    q, k, dqo, dko, qw, kw = _rope_inputs(2, 6, 2, 2, 64, BF, 13)
    rope = la.Rope(la.rope_inv_freq(64))
    far = 1 << 31
    big = torch.empty(far + 6 * 2 * 64, dtype=BF, device="cuda")
    args = dict(q_weight=qw.cuda(), k_weight=kw.cuda(), rope=rope)
    want = la.qk_norm_rope_fwd(q.cuda(), k.cuda(), **args)
    wantg = la.qk_norm_rope_bwd(q.cuda(), k.cuda(), dqo.cuda(), dko.cuda(), **args)
    for shape, strides in (((2, 6, 2, 64), (far, 128, 64, 1)), ((2, 6, 2, 64), (384, 64, far, 1))):
        if strides[2] == far:
            big = torch.empty(far + 2 * 384, dtype=BF, device="cuda")
        qd = big.as_strided(shape, strides)
        qd.copy_(q)
        got = la.qk_norm_rope_fwd(qd, k.cuda(), **args)
        gotg = la.qk_norm_rope_bwd(qd, k.cuda(), dqo.cuda(), dko.cuda(), **args)
        for a, b in zip(got + gotg, want + wantg):
            assert torch.equal(a, b)
        got = la.qk_norm_rope_fwd(qd, k.cuda(), out=(qd, None), **args)   # in place
        assert torch.equal(got[0], want[0]) and torch.equal(qd, want[0])


def test_weight_gradients_are_deterministic_and_empty_sums_are_zero():
    q, k, dq, dk, qw, kw = _cuda(*_rope_inputs(4, 777, 8, 2, 128, BF, 31, wdt=F32))
    first = la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in
                   zip(first, la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw)))
    e = torch.zeros(2, 0, 4, 128, device="cuda", dtype=BF)
    got = la.qk_norm_rope_bwd(e, e, e, e, qw, kw)
    assert got[0].shape == e.shape and bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_norm_rotation_refusals():
    q, k, dq, dk, qw, kw = _cuda(*_rope_inputs(2, 4, 4, 2, 64, BF, 3))
    rope = la.Rope(la.rope_inv_freq(64))
    pos = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="positions must be"):
        la.rotary_fwd(q, k, rope, pos)
    with pytest.raises(TypeError, match="int32 or int64"):
        la.rotary_fwd(q, k, rope, pos.float())
    with pytest.raises(ValueError, match="on cuda"):
        la.rotary_fwd(q, k, rope, pos[0].cpu())
    with pytest.raises(ValueError, match="exceeds"):
        la.rotary_fwd(q[..., :32], k[..., :32], rope)
    with pytest.raises(ValueError, match="inv_freq is on"):
        la.rotary_fwd(q, k, la.Rope(la.rope_inv_freq(64, device="cpu")))
    with pytest.raises(ValueError, match="needs positions"):
        la.rotary_fwd(q, k, la.Rope(la.rope_inv_freq(64), sections=(16, 16)))
    with pytest.raises(ValueError, match="one entry per sequence"):
        la.rotary_fwd(q, k, rope, position_offset=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="weights must be"):
        la.qk_norm_rope_fwd(q, k, qw[:32])
    with pytest.raises(TypeError, match="share one dtype"):
        la.qk_norm_rope_fwd(q, k.float())
    with pytest.raises(ValueError, match="share shape"):
        la.qk_norm_rope_bwd(q, k, dq[:, :2], dk[:, :2], qw, kw)
    with pytest.raises(ValueError, match="batch dimension"):
        la.rotary_fwd(q, k, rope, cu_seqlens=torch.tensor([0, 2, 4], dtype=torch.int32))


# ---------------------------------------------------------------------------
# differences, graphs, a run together

def test_gradients_against_differences_of_the_kernels():
    # along a random direction: (f(p + h v) - f(p - h v)) / 2h against grad . v, fp32, f summed
    # in fp64.  The difference's own error: the values' roundings (2^-20 of f's terms) over h
    # = 2^-8, and h^2 of the third derivative, which h = 2^-8 holds to 2^-16 of terms of order 1:
    # together 2^-11 of the root of the sum of the squared terms, of which there are 2 * 150 * 32
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    h = 2.0 ** -8
    x, do = r(2, 150, 2, 16), r(2, 150, 2, 16)
    g, init, dfin = -r(2, 150, 2, 16).abs(), r(2, 2, 16), r(2, 2, 16)

    def scan(x, g, init):
        o, fin = la.gated_scan_fwd(x, g, init)
        return float((o.double() * do).sum() + (fin.double() * dfin).sum())

    q, w, dy = r(2, 150, 2, 16), 1 + 0.2 * r(16), r(2, 150, 2, 16)
    rope = la.Rope(la.rope_inv_freq(16))

    def rot(q, w):
        return float((la.qk_norm_rope_fwd(q, None, w, rope=rope).double() * dy).sum())

    cases = ((scan, (x, g, init), la.gated_scan_bwd(x, g, do, init, dfin)),
             (rot, (q, w), [la.qk_norm_rope_bwd(q, None, dy, None, w, rope=rope)[i]
                            for i in (0, 2)]))
    for f, args, grads in cases:
        for i, grad in enumerate(grads):
            v = r(*args[i].shape)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * v, args[i] - h * v
            diff = (f(*up) - f(*down)) / (2 * h)
            terms = grad.double() * v
            size = float(terms.square().sum().sqrt())
            want = float(terms.sum())
            assert abs(diff - want) <= 2.0 ** -11 * (size * math.sqrt(2 * 150 * 32) + abs(want)), \
                (f.__name__, i, diff, want, size)


def test_autograd_equals_the_explicit_calls():
    x, g, do, init, dfin = _cuda(*_scan_inputs(2, 140, 2, 32, BF, F32, 2, 17))
    leaves = [t.clone().requires_grad_() for t in (x, g, init)]
    o, fin = la.gated_scan(*leaves)
    got = torch.autograd.grad((o, fin), leaves, (do, dfin))
    assert all(torch.equal(a, b) for a, b in zip(got, la.gated_scan_bwd(x, g, do, init, dfin)))
    o, _ = la.gated_scan(*leaves)        # the final state unused
    got = torch.autograd.grad(o, leaves, do)
    assert all(torch.equal(a, b) for a, b in zip(got, la.gated_scan_bwd(x, g, do, init)))
    q, k, dq, dk, qw, kw = _cuda(*_rope_inputs(2, 33, 4, 2, 64, BF, 18))
    rope = la.Rope(la.rope_inv_freq(64))
    leaves = [t.clone().requires_grad_() for t in (q, k, qw, kw)]
    yq, yk = la.qk_norm_rope(leaves[0], leaves[1], la.QkNorm(leaves[2], leaves[3]), rope)
    got = torch.autograd.grad((yq, yk), leaves, (dq, dk))
    want = la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw, rope=rope)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = la.rotary(leaves[0], rope=rope)
    assert torch.equal(torch.autograd.grad(y, leaves[0], dq)[0], la.rotary_bwd(dq, rope=rope))


def test_packed_calls_replay_from_two_graphs():
    # nothing is copied from the host: packed calls are captured too; two graphs of the same
    # calls hold their own workspaces and replay with new inputs, one after the other and on
    # two streams at once
    cu = torch.tensor([0, 700, 700, 705, 1500], dtype=torch.int32)
    cud = cu.cuda()
    kw = dict(cu_seqlens=cud, cu_seqlens_host=cu)
    rope = la.Rope(la.rope_inv_freq(64))

    def step(t):
        x, g, do, init, dfin, q, k, dq, dk, qw, kw_ = t
        o, fin, st = la.gated_scan_fwd(x, g, init, keep_states=True, **kw)
        a = la.gated_scan_bwd(x, g, do, init, dfin, states=st, **kw)
        y = la.qk_norm_rope_fwd(q, k, qw, kw_, rope=rope, **kw)
        b = la.qk_norm_rope_bwd(q, k, dq, dk, qw, kw_, rope=rope, **kw)
        return (o, fin) + tuple(a) + tuple(y) + tuple(b)

    draw = lambda seed: _cuda(*(_scan_inputs(1, 1500, 2, 64, BF, BF, 4, seed) +
                                _rope_inputs(1, 1500, 4, 2, 64, BF, seed)))
    held, graphs, outs = [draw(1), draw(2)], [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held[0])
    torch.cuda.current_stream().wait_stream(side)
    for t in held:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(t))
        graphs.append(gr)
    for seed in (3, 5):
        for i, t in enumerate(held):
            for a, b in zip(t, draw(seed + i)):
                a.copy_(b)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        la.get_device_error()
        for t, out in zip(held, outs):
            got = [y.clone() for y in out]
            assert all(torch.equal(a, b) for a, b in zip(got, step(t))), seed


def test_layer_run_together():
    # a layer as it is used, packed, fp32: values mixed along time by the gated recurrence,
    # queries and keys normalised and rotated, the decayed linear attention; outputs and every
    # gradient against fp64 autograd of the definitions, at the framework's own 1e-4 of the
    # largest value
    cu = [0, 40, 41, 41, 150]
    T, H, Hk, D = cu[-1], 4, 2, 32
    gen = torch.Generator().manual_seed(40)
    r = lambda *s: torch.randn(s, generator=gen)
    n = len(cu) - 1
    q, k, v = r(1, T, H, D), r(1, T, Hk, D), r(1, T, Hk, D)
    gate = torch.nn.functional.logsigmoid(r(1, T, Hk, D) + 2)
    qw, kw, s0, do = 1 + 0.1 * r(D), 1 + 0.1 * r(D), 0.1 * r(n, Hk, D), r(1, T, H, D)
    gg = -torch.tensor([0.02, 0.1, 0.3, 0.5])
    freq = la.rope_inv_freq(D)
    cut = torch.tensor(cu, dtype=torch.int32)
    off = torch.tensor([0, 7, 0, 100], dtype=torch.int32)

    dev = [t.cuda().requires_grad_() for t in (q, k, v, gate, qw, kw, s0)]
    mixed, carried = la.gated_scan(dev[2], dev[3], dev[6], cu_seqlens=cut)
    o, _ = la.recurrent(dev[0], dev[1], mixed, g_gamma=gg, cu_seqlens=cut,
                        qk_norm=la.QkNorm(dev[4], dev[5]), rope=la.Rope(freq),
                        position_offset=off)
    got = [o, carried] + list(torch.autograd.grad((o * do.cuda()).sum() + carried.sum(), dev))

    ref = [t.double().requires_grad_() for t in (q, k, v, gate, qw, kw, s0)]
    pos = R.positions_of(1, T, cu, off)
    qr = R.norm_rope(ref[0], ref[4], 1e-6, True, freq.cpu(), None, pos)
    kr = R.norm_rope(ref[1], ref[5], 1e-6, True, freq.cpu(), None, pos)
    rows, fins = [None] * T, []
    for i, (_, lo, hi) in enumerate(R.spans(1, T, cu)):
        m, S = ref[6][i], torch.zeros(H, D, D, dtype=torch.float64)
        for t in range(lo, hi):
            m = ref[3][0, t].exp() * m + ref[2][0, t]
            kk, vv = (z.repeat_interleave(H // Hk, 0) for z in (kr[0, t], m))
            S = gg.double().exp()[:, None, None] * S + kk[:, :, None] * vv[:, None, :]
            rows[t] = torch.einsum("hd,hde->he", qr[0, t] * D ** -0.5, S)
        fins.append(m)
    o_ref, c_ref = torch.stack(rows)[None], torch.stack(fins)
    want = [o_ref, c_ref] + list(torch.autograd.grad((o_ref * do.double()).sum() + c_ref.sum(),
                                                     ref))
    for name, a, b in zip(("o", "carried", "dq", "dk", "dv", "dgate", "dqw", "dkw", "ds0"), got,
                          want):
        err = float((a.detach().cpu().double() - b.detach()).abs().max() / b.detach().abs().max())
        assert err <= 1e-4, (name, err)


def test_decoding_continues_the_prompt():
    # the prompt in one call, then single tokens with the carried states and the positions'
    # offset: the same outputs as the whole sequence at once, within one bf16 step each
    B, T, H, D, P = 3, 60, 4, 64, 52
    gen = torch.Generator().manual_seed(50)
    r = lambda *s: torch.randn(s, generator=gen).to(BF).cuda()
    q, k, v = r(B, T, H, D), r(B, T, H, D), r(B, T, H, D)
    gate = torch.nn.functional.logsigmoid(r(B, T, H, D).float() + 2)
    norm, rope = la.QkNorm(), la.Rope(la.rope_inv_freq(D))
    gg = la.alibi_g_gamma(H)

    def layer(lo, hi, states):
        s, S = states
        m, s = la.gated_scan(v[:, lo:hi], gate[:, lo:hi], s)
        o, S = la.recurrent(q[:, lo:hi], k[:, lo:hi], m, g_gamma=gg, initial_state=S,
                            qk_norm=norm, rope=rope, position_offset=[lo] * B)
        return o, (s, S)

    whole, _ = layer(0, T, (None, None))
    o, states = layer(0, P, (None, None))
    parts = [o]
    for t in range(P, T):
        o, states = layer(t, t + 1, states)
        parts.append(o)
    got = torch.cat(parts, 1)
    err = float((got.float() - whole.float()).abs().max() / whole.float().abs().max())
    assert err <= 2e-2, err


@pytest.mark.parametrize("gated", [False, True])
def test_attention_calls_take_norms_and_rotation(gated):
    # recurrent_gla and lightning_attn with qk_norm= and rope= are the calls on normalised and
    # rotated inputs, gradients included
    B, T, H, D = 2, 70, 2, 64
    gen = torch.Generator().manual_seed(60)
    r = lambda *s: torch.randn(s, generator=gen).to(BF).cuda()
    leaves = [r(B, T, H, D).requires_grad_() for _ in range(3)]
    w = [(1 + 0.1 * r(D)).requires_grad_() for _ in range(2)]
    gate = torch.nn.functional.logsigmoid(r(B, T, H, D).float() + 2)
    norm, rope = la.QkNorm(w[0], w[1]), la.Rope(la.rope_inv_freq(D))
    pos = torch.randint(0, 1000, (B, T), generator=gen).cuda()
    gg = la.alibi_g_gamma(H)

    def attend(q, k, v, **kw):
        if gated:
            return la.recurrent_gla(q, k, v, g=gate, g_gamma=gg, **kw)[0]
        return la.lightning_attn(q, k, v, 1, 4, **kw)
    q, k, v = leaves
    o = attend(q, k, v, qk_norm=norm, rope=rope, positions=pos)
    q2, k2 = la.qk_norm_rope(q, k, norm, rope, pos)
    want = attend(q2, k2, v)
    o, want = (t[0] if isinstance(t, tuple) else t for t in (o, want))
    assert torch.equal(o, want)
    do = r(*o.shape)
    for a, b in zip(torch.autograd.grad(o, leaves + w, do),
                    torch.autograd.grad(want, leaves + w, do)):
        assert torch.equal(a, b)
