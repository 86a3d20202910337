"""The gated delta rule's outputs number by number against fp64, at bounds near their errors.

dv of the chunked backward is rounded once: a number is off by half a step, 2^-8 of it at most,
and by what R, made of operands held as two bf16, is off.  Such an operand is off by 2^-18 of
itself and the product left out is as much; a sum of random signs is off by that much of its
terms' root sum of squares.  R takes P^T dO, K K', B^T W, and K' as many again for every chunk:
below 20 such errors over four chunks, at 6 sigma 20 * 6 * 2^-18 = 4.6e-4 of the outputs' rms.
(Rounded twice, as R and as beta R, it would be off by up to 2^-7 of a number.)"""
import pytest
import torch

import delta_reference as R
import linear_attention_head_gb300 as la
from test_gpu_delta import BF, F32, cuda, inputs

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
    assert float(over.max()) <= 0.0, "%d of %d numbers beyond one rounding, the worst by %.3g rms" % (
        int((over > 0).sum()), over.numel(), float(over.max()) / rms)
