"""The operators beside the attention where fp32 runs out: infinite states under gates that
forget.  The tolerances are those of test_gpu_layer.py unless a test derives its own."""
import math

import pytest
import torch

import layer_reference as R
import linear_attention_head_gb300 as la
from test_gpu_layer import BF, F32, SCAN_U, _close, _cuda, _scan_inputs

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
