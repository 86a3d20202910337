"""Gates of the delta rule that leave large sums in a chunk: strong decays and resets (-inf) before
slow ones.  The final state against fp64.

Tolerance: an operand held as two bf16 is off by 2^-18 of it at most, the product left out by as
much; the writes that reach the final state come through X, B, Eps, the operand of the state and K
(exact): below 5 * 2^-18 = 1.9e-5 of their norm in one chunk if every one were the largest and of
one sign.  Decays within 4e-6 where they count (test_delta_gate_sums.py) leave 2e-5 standing, as
neither is near its largest everywhere.  Sums in one float were off by up to 2.4e-4."""
import math

import pytest
import torch

import delta_reference as R
import linear_attention_head_gb300 as la
from test_gpu_delta import BF, F32, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["strong", 1, 4, 16, 32])
@pytest.mark.parametrize("T", [64, 128, 100])
def test_slow_gates_after_strong_ones(kind, T):
    x = inputs(2, T, 4, 2, 128, 128, BF, F32, 2, 21)
    gen = torch.Generator().manual_seed(T)
    last = (T - 1) // 64 * 64       # the last chunk's first token
    x["g"][:, last:] *= 0.1
    early = max(1, min(40, T - last - 4))
    if kind == "strong":
        x["g"][:, last:last + early] = -3.0 - 5.0 * torch.rand(early, generator=gen)[:, None]
    else:
        x["g"][:, last + torch.randperm(early, generator=gen)[:kind]] = -math.inf
    ref = R.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], 128 ** -0.5, x["init"])
    d = cuda(x)
    o, fin = la.gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["init"])
    off = (fin.cpu().double() - ref["final"]).flatten(2).norm(dim=2)
    off /= ref["final"].flatten(2).norm(dim=2)
    assert float(off.max()) <= 2e-5, float(off.max())
    assert float((o.cpu().double() - ref["o"]).norm()) <= 2.0 ** -8 * float(ref["o"].norm())
