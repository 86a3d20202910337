"""The gated delta rule's outputs number by number against fp64, at bounds near their errors.

dv of the chunked backward is rounded once: a number is off by half a step, 2^-8 of it at most,
and by what R, made of operands held as two bf16, is off.  Such an operand is off by 2^-18 of
itself and the product left out is as much; a sum of random signs is off by that much of its
terms' root sum of squares.  R takes P^T dO, K K', B^T W, and K' as many again for every chunk:
below 20 such errors over four chunks, at 6 sigma 20 * 6 * 2^-18 = 4.6e-4 of the outputs' rms.
(Rounded twice, as R and as beta R, it would be off by up to 2^-7 of a number.)"""
import pytest
import torch

import delta_bounds as DB
import delta_reference as R
import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import delta
from test_gpu_delta import BF, F32, chunked, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,cu", [
    ((1, 64, 1, 1, 128, 128), None), ((2, 256, 2, 1, 128, 128), None),
    ((1, 200, 4, 2, 64, 40), None), ((1, 130, 2, 2, 24, 72), None),
    ((1, 211, 2, 1, 64, 128), [0, 64, 65, 100, 211]), ((1, 90, 3, 3, 96, 56), [0, 0, 30, 90]),
    ((1, 1500, 1, 1, 64, 64), None)])
def test_dv_is_rounded_once(size, cu):
    n = size[0] if cu is None else len(cu) - 1
    x = inputs(*size, BF, F32, n, 31)
    s = size[4] ** -0.5
    ref = R.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], s, x["init"], cu, x["do"],
                  x["dfin"])["dv"]
    d = cuda(x)
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    dv = la.gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"],
                            initial_state=d["init"], d_final_state=d["dfin"], cu_seqlens=cu_t)[2]
    off = (dv.cpu().double() - ref).abs()
    rms = float(ref.square().mean().sqrt())
    over = off - (2.0 ** -8 * ref.abs() + 4.6e-4 * rms)
    assert float(over.max()) <= 0.0, "%d of %d numbers beyond one rounding, by up to %.3g rms" % (
        int((over > 0).sum()), over.numel(), float(over.max()) / rms)


SIZES = [  # dtype, gates' dtype, (B, T, H, H_qk, D, E), cu
    (F32, F32, (1, 150, 2, 2, 40, 24), None), (F32, F32, (2, 77, 3, 1, 128, 128), None),
    (F32, F32, (1, 60, 2, 1, 33, 200), None), (F32, F32, (1, 40, 2, 2, 256, 130), None),
    (F32, F32, (1, 100, 2, 1, 32, 40), [0, 1, 2, 3, 60, 60, 100]),
    (BF, BF, (3, 1, 4, 2, 128, 128), None), (BF, F32, (2, 16, 4, 2, 64, 96), None),
    (BF, F32, (1, 70, 2, 2, 12, 20), None), (BF, F32, (1, 50, 2, 1, 130, 256), None),
    (BF, BF, (2, 63, 2, 1, 128, 128), None), (BF, F32, (2, 256, 4, 2, 128, 128), None),
    (BF, F32, (1, 333, 2, 2, 96, 120), None), (BF, F32, (1, 200, 1, 1, 8, 16), None),
    (BF, F32, (1, 300, 2, 1, 32, 40), [0, 20, 21, 21, 300]),
    (BF, F32, (1, 2100, 1, 1, 128, 128), None), (BF, F32, (2, 1601, 2, 1, 64, 40), None),
    (BF, F32, (1, 1764, 1, 1, 32, 24), [0, 0, 30, 1700, 1700, 1764])]


@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("state", [True, False])
def test_every_output_within_its_bound(case, state):
    dt, gt, size, cu = SIZES[case]
    n = size[0] if cu is None else len(cu) - 1
    x = inputs(*size, dt, gt, n, 41 + case, state)
    ref = R.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], size[4] ** -0.5, x["init"], cu,
                  x["do"], x["dfin"])
    longest = max(hi - lo for _, lo, hi in R.spans(size[0], size[1], cu))
    tc = chunked(dt, size[4], size[5], longest)
    d = cuda(x)
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    a = (d["q"], d["k"], d["v"], d["g"], d["beta"])
    kw = dict(initial_state=d["init"], cu_seqlens=cu_t)
    o, fin, saved = la.gated_delta_fwd(*a, keep=True, **kw)
    assert (saved is not None) == tc
    got = dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"),
                   la.gated_delta_bwd(*a, d["do"], d_final_state=d["dfin"], saved=saved, **kw)))
    got.update(o=o, final=fin)
    terms = DB.terms_of(x["v"], ref["dv"])
    bad = [t for name, y in got.items()
           for t in DB.faults(name, y, ref[name], dt, tc, longest, terms)]
    assert not bad, bad


@pytest.mark.parametrize("cu", [None, [0, 70, 70, 201]])
def test_dv_in_a_place_with_strides_of_its_own(cu):
    # heads before tokens, rows with room behind them: what lies between stays
    B, T, H, E = (2, 201, 3, 40) if cu is None else (1, 201, 3, 40)
    n = B if cu is None else len(cu) - 1
    d = cuda(inputs(B, T, H, 1, 64, E, BF, F32, n, 51))
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    a = (d["q"], d["k"], d["v"], d["g"], d["beta"])
    want = la.gated_delta_bwd(*a, d["do"], initial_state=d["init"], d_final_state=d["dfin"],
                              cu_seqlens=cu_t)
    c = delta._Call(*a, None, d["init"], cu_t, cu_t, True)
    room = torch.full((B, H, T + 1, E + 8), 7.0, dtype=BF, device="cuda")
    dv = room.transpose(1, 2)[:, :T, :, :E]
    dq, dk = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    dg, db = (torch.empty(B, T, H, dtype=BF, device="cuda") for _ in range(2))
    dinit = torch.empty_like(d["init"])
    dims = c.dims(do=d["do"], dq=dq, dk=dk, dv=dv)
    ws, nbytes = c.workspace(dims, 2)
    delta._call(c.device, delta.N.lib().la_gated_delta_bwd, delta._ref(dims), c.code, *c.inputs(),
                *(delta._ptr(t) if torch.is_tensor(t) else t for t in (
                    d["do"], c.scale, c.init, d["dfin"], c.cu.dev, c.cu.host, None, dq, dk, dv, dg,
                    db, dinit, ws)), nbytes)
    for x, y in zip((dq, dk, dv, dg, db, dinit), want):
        assert torch.equal(x, y)
    room.transpose(1, 2)[:, :T, :, :E] = 7.0
    assert (room == 7.0).all()
