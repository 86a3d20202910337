"""What autograd hands to the delta rule's backward: no gradient for an output that went unused."""
import pytest
import torch

import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import delta
from test_gpu_delta import BF, F32, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,T", [(BF, 90), (F32, 20)])
def test_an_unused_output_has_no_gradient(dt, T, monkeypatch):
    x = cuda(inputs(2, T, 2, 1, 32, 32, dt, F32, 2, 15))
    seen = []
    bwd = delta.gated_delta_bwd

    def watched(*a, **kw):
        seen.append(a)
        return bwd(*a, **kw)
    monkeypatch.setattr(delta, "gated_delta_bwd", watched)
    names = ("q", "k", "v", "g", "beta")
    for part in ("o", "final"):
        leaves = [x[n].clone().requires_grad_() for n in names]
        init = x["init"].clone().requires_grad_()
        o, fin = la.gated_delta(*leaves, initial_state=init)
        w = x["do"] if part == "o" else x["dfin"]
        ((o if part == "o" else fin) * w).sum().backward()
        do, dfin = seen[-1][5], seen[-1][8]
        assert (dfin is None) == (part == "o")
        # as with zeros in its place
        want = bwd(*(x[n] for n in names), x["do"] if part == "o" else torch.zeros_like(x["do"]),
                   initial_state=x["init"],
                   d_final_state=torch.zeros_like(x["dfin"]) if part == "o" else x["dfin"])
        for n, t, r in zip(names + ("init",), leaves + [init], want):
            assert torch.equal(t.grad, r.to(t.dtype)), (part, n)
    assert len(seen) == 2
