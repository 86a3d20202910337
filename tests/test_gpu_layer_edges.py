"""The operators beside the attention where fp32 runs out: infinite states under gates that
forget, decays over their range, angles at far positions and of any frequency; and the launches of
the gated recurrence that depend on the number of chains.  The tolerances are those of
test_gpu_layer.py unless a test derives its own."""
import ctypes
from fractions import Fraction
import math

import pytest
import torch

import layer_reference as R
import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import _native as N
from test_gpu_layer import (BF, F32, SCAN_U, _close, _cuda, _relayout, _scan_check,
                            _scan_inputs)

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (BF, F32), (F32, F32)]


# ---------------------------------------------------------------------------
# infinite states

def _same(got, ref, err, dtype, label):
    """NaN and infinities where the definition has them, the rest within the tolerance."""
    got = got.detach().cpu()
    assert torch.equal(got.isnan(), ref.isnan()), label + ": NaN"
    inf = ref.isinf()
    assert torch.equal(got.isinf(), inf), label + ": infinities"
    assert torch.equal(got[inf].double().sign(), ref[inf].sign()), label + ": signs"
    ok = ref.isfinite()
    _close(got[ok], ref[ok], SCAN_U * err[ok], dtype, label)


# a launch of each kind: segments, teams in turn, a team alone, a thread alone
@pytest.mark.parametrize("B,T,H,D", [(1, 1500, 1, 8), (1, 300, 121, 64), (3, 300, 110, 64),
                                     (1, 1500, 1, 9), (1400, 17, 1, 8)])
@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_infinite_states_stay_infinite_under_strong_gates(B, T, H, D, dt, gt, reverse):
    # the product of a few decays underflows to 0 although none of them is: what is infinite
    # stays so, as token by token; a decay that is 0 itself makes it NaN
    x, g, do, init, dfin = _scan_inputs(B, T, H, D, dt, gt, B, 31)
    c = torch.arange(H * D).reshape(H, D) % 9
    gates = torch.tensor([-3.4, -4.0, -7.0, -10.0, -80.0, -7.0, -7.0, -7.0, -7.0])
    g.copy_(gates[c].expand_as(g))
    sign = torch.where(init < 0, -math.inf, math.inf)
    init = torch.where((c < 5) | (c == 6), sign, init)
    dfin = torch.where(c < 5, torch.where(dfin < 0, -math.inf, math.inf), dfin)
    x[:, T // 3] = torch.where(c == 5, math.inf, x[:, T // 3])
    do[:, 2 * T // 3] = torch.where((c == 5) | (c == 7), -math.inf, do[:, 2 * T // 3])
    g[:, T // 2] = torch.where(c == 6, -math.inf, g[:, T // 2])
    ref = R.scan(x, g, init, reverse, None, do, dfin)
    xd, gd, dod, initd, dfind = _cuda(x, g, do, init, dfin)
    o, fin, states = la.gated_scan_fwd(xd, gd, initd, reverse, keep_states=True)
    _same(o, ref["o"], ref["o_e"], dt, "o")
    _same(fin, ref["final"], ref["final_e"], F32, "final_state")
    got = la.gated_scan_bwd(xd, gd, dod, initd, dfind, reverse, states=states)
    for name, t, d in zip(("dx", "dg", "dinit"), got, (dt, gt, F32)):
        _same(t, ref[name], ref[name + "_e"], d, name)
    la.get_device_error()


# ---------------------------------------------------------------------------
# decays

@pytest.mark.parametrize("T", [1, 300])
def test_scan_decays_over_their_range(T):
    # a state under one gate (and then gates of 0, whose decay is 1 itself): exp(g) within
    # 4 u (2^x within 2^-22; near 0 the series, 2 u) and, from the argument's product with a
    # rounded log2 e, 1.25 |g| u; below 2^-126 it is 0.  T = 1: a thread alone, 300: a tile.
    H, D = 64, 256
    gate = torch.linspace(-110.0, 88.0, H * D, dtype=torch.float64).float()
    gate[::4] = torch.linspace(-0.5, 0.5, 4096, dtype=torch.float64).float()
    g = torch.zeros(1, T, H, D)
    g[0, 0] = gate.reshape(H, D)
    x, init = torch.zeros(1, T, H, D), torch.ones(1, H, D)
    o, fin = la.gated_scan_fwd(*_cuda(x, g, init))
    want = gate.double().exp()
    for got in (o[0, T - 1], fin[0]):
        got = got.cpu().double().reshape(-1)
        gone = want < 2.0 ** -126 * (1 + 2.0 ** -16)    # (to where the argument may round)
        assert 0 < int(gone.sum()) < gone.numel()
        assert bool((got[gone] <= 2.0 ** -125).all())
        err = (got - want).abs()[~gone] / want[~gone]
        bound = (4 + 1.25 * gate.double().abs()[~gone]) * R.U
        assert bool((err <= bound).all()), float((err / bound).max())


# ---------------------------------------------------------------------------
# angles

_PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923,
               10 ** 64)


def _turn(position, freq):
    """The fraction of a turn in (-1/2, 1/2] of position * freq radians, freq the fp64 number
    itself, with 60 digits of pi."""
    t = Fraction(position) * Fraction(freq) / (2 * _PI)
    return float(t - round(t))


def _angles(positions, freqs):
    """cos and sin [position, frequency] of the kernel: pairs (1, 0) rotated."""
    n, R_ = len(freqs), len(positions)
    q = torch.zeros(1, R_, 1, 2 * n)
    q[..., :n] = 1
    rope = la.Rope(torch.tensor(freqs, dtype=torch.float64).cuda())
    y = la.rotary_fwd(q.cuda(), rope=rope,
                      positions=torch.tensor(positions, dtype=torch.int64).cuda())
    y = y[0, :, 0].cpu().double()
    return y[:, :n], y[:, n:]


FAR = [2 ** 31 - 1, -2 ** 31, 123456789, -77777777, 2 ** 28 + 1, 2 ** 24 + 1, 131071, 7, 0, -1]


def test_rotation_angles_of_any_frequency():
    # frequencies above 1 and below, negative ones and 0 too: cos and sin within 2^-22 of those
    # of the exact product (the angle itself: the next test)
    freqs = [1.0, 2.0, 3.7, 100.0, 12345.678, -5.5, 1e-4, 0.1, 0.0, 1e6]
    cos, sin = _angles(FAR, freqs)
    for i, p in enumerate(FAR):
        for j, f in enumerate(freqs):
            a = 2 * math.pi * _turn(p, f)
            assert abs(float(cos[i, j]) - math.cos(a)) <= 2.0 ** -22, (p, f)
            assert abs(float(sin[i, j]) - math.sin(a)) <= 2.0 ** -22, (p, f)


@pytest.mark.parametrize("position", [2 ** 31 - 1, -2 ** 31, 2 ** 28 + 1, 2 ** 24 + 1])
def test_rotation_angle_keeps_its_fraction_of_a_turn(position):
    # frequencies that take this position to almost whole turns: there the sine, a small number,
    # shows the angle itself.  The fraction of a turn is within 2^-32 (its lower bits are cut off)
    # and |position| 2^-64 <= 2^-33 (the two roundings of a frequency's fraction); sine and the
    # remainder as fp32 are within 2^-22 of their value.
    freqs = [2 * math.pi * round(abs(position) * f / (2 * math.pi)) / abs(position)
             for f in (1.0, 0.7, 0.3, 0.01, 2.0, 17.0)]
    _, sin = _angles([position], freqs)
    for j, f in enumerate(freqs):
        turn = _turn(position, f)
        assert abs(turn) < 2.0 ** -16       # (of these frequencies)
        want = math.sin(2 * math.pi * turn)
        bound = 2 * math.pi * 1.5 * 2.0 ** -32 + 2.0 ** -22 * abs(want)
        assert abs(float(sin[0, j]) - want) <= bound, (f, turn, float(sin[0, j]), want)


# ---------------------------------------------------------------------------
# teams that take a chain's tiles in turn, backward

def _chains():
    """Chains for which both directions have their teams take turns: fewer than the teams of
    the backward by half, more than are cut into segments."""
    return int(0.8 * torch.cuda.get_device_properties(0).multi_processor_count)


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 1, 130, 900], [0, 512, 512, 900]])
def test_scan_backward_of_teams_in_turn(dt, gt, reverse, cu):
    n = 1 if cu is None else len(cu) - 1
    x, g, do, init, dfin = _scan_inputs(1, 900, _chains() // n, 64, dt, gt, n, 33)
    _scan_check(x, g, do, init, dfin, reverse, cu, label="in turn")


@pytest.mark.parametrize("dt,gt,layout,D", [
    (BF, F32, "head_major", 72), (F32, F32, "head_major", 72), (BF, BF, "dense", 63),
    (F32, F32, "odd_rows", 64)])
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_backward_of_teams_in_turn_by_rows(dt, gt, layout, D, reverse):
    # tiles that cross heads which are apart (copied row by row), rows that no wide access fits
    H = _chains() * 64 // D - 1
    x, g, do, init, dfin = _scan_inputs(1, 700, H, D, dt, gt, 1, 34)
    dev = [_relayout(t, layout) for t in (x, g, do)] + _cuda(init, dfin)
    _scan_check(x, g, do, init, dfin, reverse, label=layout, dev=dev)


@pytest.mark.parametrize("dt", [BF, F32])
def test_scan_withheld_tile_among_backward_teams_that_wait_for_one_another(dt):
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 900, _chains(), 64, dt, dt, 1, 35))
    _, _, states = la.gated_scan_fwd(x, g, init, keep_states=True)
    want = la.gated_scan_bwd(x, g, do, init, dfin, states=states)
    la.get_device_error()
    N.check(N.lib().la_debug_withhold_next_handoff(1))
    la.gated_scan_bwd(x, g, do, init, dfin, states=states)
    with pytest.raises(N.LaError) as err:
        la.get_device_error()
    assert err.value.status == N.LA_ERR_TIMEOUT
    la.get_device_error()
    got = la.gated_scan_bwd(x, g, do, init, dfin, states=states)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    la.get_device_error()


@pytest.mark.parametrize("H", [1, 121])
def test_scan_backward_of_tokens_far_apart(H):
    # tokens further apart than the steps of whole groups that fit 32 bits of bytes, read and
    # (C call) written; one chain in segments, many in turn
    x, g, do, init, dfin = _cuda(*_scan_inputs(1, 140, H, 64, BF, BF, 1, 36))
    step = (1 << 24) + 64 * H
    room = 139 * step + 64 * H
    far = lambda buf: buf.as_strided((1, 140, H, 64), (0, step, 64, 1))
    for reverse in (False, True):
        want = la.gated_scan_bwd(x, g, do, init, dfin, reverse)
        for i in range(3):
            buf = torch.empty(room, dtype=BF, device="cuda")
            args = [x, g, do]
            args[i] = far(buf).copy_(args[i])
            got = la.gated_scan_bwd(*args, init, dfin, reverse)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (i, reverse)
            del buf, args
        # dx far apart
        lib, dg, dinit = N.lib(), torch.empty_like(g), torch.empty_like(init)
        buf = torch.zeros(room, dtype=BF, device="cuda")
        dx = far(buf)
        near = (ctypes.c_int64 * 3)(*x.stride()[:3])
        apart = (ctypes.c_int64 * 3)(0, step, 64)
        d = N.LaScanDims(1, 140, H, 64, 1, N.LA_DTYPE_BF16, near, near, near, near, apart, near)
        ws = torch.empty(int(lib.la_gated_scan_workspace_size(ctypes.byref(d), N.LA_DTYPE_BF16, 2)),
                         dtype=torch.uint8, device="cuda")
        ptr = [t.data_ptr() for t in (x, g, do, init, dfin, dx, dg, dinit, ws)]
        N.check(lib.la_gated_scan_bwd(ctypes.byref(d), N.LA_DTYPE_BF16, *ptr[:5], int(reverse),
                                      None, None, None, *ptr[5:9], ws.numel(),
                                      torch.cuda.current_stream().cuda_stream))
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, dinit), want)), reverse
        del buf, dx
    la.get_device_error()
