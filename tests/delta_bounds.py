"""Bounds near the errors of the gated delta rule's kernels, for every output number by number.

With u = 2^-24, L tokens, C chunks of 64, rms that of the whole output:

Token by token (fp32 states): a token adds below 25 u of what it meets (its sums over D, the
write, the decay), with signs of its own, so L of them sqrt(L) as much: an output is within
e = 25 u sqrt(L) in the norm, and a number within 6 e of the rms beside e of itself.  dg is
four times that off: it is a running sum, and of differences q.dq - v.dv, so what is off goes by
those terms (one token without a state: they are equal, dg is 0 and comes out as 2^-24 of them);
terms: the rms of v.dv.  bf16 outputs are rounded once: 2^-8 of a number.

Chunks: o and dv are made of operands held as two bf16 (2^-18 of a term and as much left out, with
signs of their own), below 20 such errors over four chunks and sqrt(C / 4) times that over more,
at 6 sigma 20 * 6 * 2^-18 = 4.6e-4 of the rms, and rounded once.  The states (final, and back): the
same operands, 5 of them a chunk, a chunk's error decaying with what it is of: 5 * 2^-18 = 1.9e-5
in the norm, four times that for a number beside the largest.  dq, dk, dg, dbeta: products of
numbers rounded to bf16 once, up to six in a sum: 1e-2 in the norm, 2e-2 of the largest."""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def terms_of(v, dv):
    """The rms of v.dv: what dg is a difference of."""
    return float((v.double() * dv).sum(-1).square().mean().sqrt()) if v.numel() else 0.0


def faults(name, got, ref, dtype, tc, L, terms):
    """What of got is beyond its bounds: texts, none where it is not."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not ref.numel():
        return []
    if not torch.isfinite(got).all():
        return [name + ": not finite"]
    off = (got - ref).abs()
    norm, rms, big = float(ref.norm()), float(ref.square().mean().sqrt()), float(ref.abs().max())
    state = name in ("final", "dinit")
    half = HALF_STEP[torch.float32 if state else dtype]
    if not tc:
        e = 25 * U * math.sqrt(max(L, 1)) * (4 if name == "dg" else 1)
        rms, norm = (rms + terms, norm + terms * math.sqrt(ref.numel())) if name == "dg" else \
            (rms, norm)
        most = (half + e) * ref.abs() + 6 * e * rms
        far = (half + e) * norm
    elif state:
        most, far = 4 * 2e-5 * big, 2e-5 * norm
    elif name in ("o", "dv"):
        e = 4.6e-4 * max(1.0, math.sqrt(L / 256))
        most = half * ref.abs() + e * rms
        far = (half + e) * norm
    else:
        most, far = 2e-2 * big, 1e-2 * norm
    bad = []
    over = off - most
    if float(over.max()) > 1e-30:
        bad.append("%s: a value beyond its bound by %.3g, rms %.3g"
                   % (name, float(over.max()), rms))
    if float(off.norm()) > far + 1e-30:
        bad.append("%s: off by %.3g, %.3g allowed" % (name, float(off.norm()), far))
    return bad
