"""The gated delta rule on the GPU against its fp64 definition (delta_reference.py), forward and
backward, token by token and in chunks on the tensor cores.

Tolerances, with u = 2^-24.  Keys have length one and 0 <= beta <= 1, so a step carries an error
of S (and back, of K = dL/dS) on without growing it, and errors add up in the Frobenius norm.
Token by token in fp32 a token adds: its sum over D (16 products, at most 4 joins: 20 u), the
write (3 u), the decay (2 u): below 25 u of the largest ||S||.  In chunks, an operand held as two
bf16 is off by 2^-18 and the product left out by 2^-18; three such products a chunk and the
state's own 2^-18: below 8 * 2^-17 a chunk with the fp32 sums.  So with L tokens, C = L / 64
chunks a state is within r = 25 u L, or 8 * 2^-17 C (or their like for K), of its largest norm,
an output made from it (o, dv) within r times the norm of the vector it meets, and a rounding to
the tokens' type adds half a step.  dq, dk, dg, dbeta of the chunked backward are products of
numbers rounded to bf16 once (2^-9 rms a factor): up to 6 roundings in a sum, and the result's,
stay below 1e-2 in the norm; largest single errors below 2e-2 of the largest value, the
library's bound for bf16.
"""
import math

import pytest
import torch

import delta_reference as R
import linear_attention_head_gb300 as la

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF_STEP = {BF: 2.0 ** -8, F32: U}


def inputs(B, T, H, HK, D, E, dt, gt, n, seed, state=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt)
    x = {"q": unit(rnd(B, T, HK, D)), "k": unit(rnd(B, T, HK, D)), "v": rnd(B, T, H, E).to(dt),
         "g": (-torch.exp(rnd(B, T, H) * 1.5 - 3.0)).to(gt),
         "beta": torch.sigmoid(rnd(B, T, H)).to(gt), "do": rnd(B, T, H, E).to(dt),
         "init": rnd(n, H, D, E) * 0.2 if state else None,
         "dfin": rnd(n, H, D, E) * 0.2 if state else None}
    return x


def cuda(x):
    return {n: t.cuda() if t is not None else None for n, t in x.items()}


def chunked(dt, D, E, longest):
    return dt == BF and D % 8 == 0 and E % 8 == 0 and D <= 128 and E <= 128 and longest > 16


def near(got, ref, rel, extra, dtype, label, most=None):
    """||got - ref|| <= rel ||ref|| + half a step + extra, and single values within most."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert torch.isfinite(got).all(), label + ": not finite"
    if not got.numel():
        return
    off, tol = float((got - ref).norm()), (rel + HALF_STEP[dtype]) * float(ref.norm()) + extra
    assert off <= tol + 1e-30, "%s: off by %.3g, %.3g allowed" % (label, off, tol)
    if most is not None:
        big = float((got - ref).abs().max())
        assert big <= most * float(ref.abs().max()) + 1e-30, "%s: a value off by %.3g of %.3g" % (
            label, big, float(ref.abs().max()))


def check(x, cu=None, scale=None, label="", dev=None):
    """Forward, backward (from what the forward kept, and without it) against the definition."""
    q, v = x["q"], x["v"]
    B, T, HK, D = q.shape
    H, E = v.shape[2:]
    dt = q.dtype
    s = D ** -0.5 if scale is None else scale
    ref = R.delta(x["q"], x["k"], v, x["g"], x["beta"], s, x["init"], cu, x["do"], x["dfin"])
    spans = R.spans(B, T, cu)
    longest = max([hi - lo for _, lo, hi in spans], default=0)
    tc = chunked(dt, D, E, longest)
    L = max(longest, 1)
    r = 8 * 2.0 ** -17 * (1 + math.ceil(L / 64)) if tc else 25 * U * L
    d = dev if dev is not None else cuda(x)
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    kw = dict(scale=scale, initial_state=d["init"],
              cu_seqlens=cu_t.cuda() if cu is not None else None, cu_seqlens_host=cu_t)
    a = (d["q"], d["k"], d["v"], d["g"], d["beta"])
    o, fin, saved = la.gated_delta_fwd(*a, keep=True, **kw)
    assert (saved is not None) == (tc and T > 0)
    S, K = ref["scale_S"].max() if len(spans) else 0.0, ref["scale_K"].max() if len(spans) else 0.0
    S, K = float(S), float(K)
    root = math.sqrt(max(1, v.shape[0] * T * H))
    near(o, ref["o"], 0.0, s * r * S * root, dt, label + " o")
    near(fin, ref["final"], 0.0, r * S * math.sqrt(len(spans) * H), F32, label + " final_state")
    plain = la.gated_delta_fwd(*a, **kw)
    assert torch.equal(plain[0], o) and torch.equal(plain[1], fin), label + ": keep changes o"
    got = la.gated_delta_bwd(*a, d["do"], d_final_state=d["dfin"], saved=saved, **kw)
    names = ("dq", "dk", "dv", "dg", "dbeta", "dinit")
    beyond = r * (S * K + S + K) * root * 4
    for name, t in zip(names, got):
        dtype = F32 if name == "dinit" else dt
        if not tc:
            near(t, ref[name], 0.0, beyond, dtype, label + " " + name)
        elif name == "dv":
            near(t, ref[name], 0.0, 4 * r * K * root, dtype, label + " " + name)
        elif name == "dinit":
            near(t, ref[name], 0.0, 4 * r * K * math.sqrt(len(spans) * H), F32, label + " dinit")
        else:
            near(t, ref[name], 1e-2, 0.0, dtype, label + " " + name, most=2e-2)
    again = la.gated_delta_bwd(*a, d["do"], d_final_state=d["dfin"], **kw)
    for name, t, w in zip(names, got, again):
        assert torch.equal(t, w), label + ": computed again, %s differs" % name
    torch.cuda.synchronize()
    la.get_device_error()
    return ref


TYPES = [(BF, BF), (BF, F32), (F32, F32)]
# batch, tokens, value heads, query/key heads, D, E
TOKEN_SIZES = [(1, 1, 1, 1, 1, 1), (3, 1, 4, 2, 128, 128), (2, 5, 2, 1, 64, 96), (1, 16, 3, 3, 33, 7),
               (2, 9, 2, 2, 256, 256), (1, 17, 2, 2, 12, 20), (1, 40, 1, 1, 130, 66)]


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("size", TOKEN_SIZES)
def test_token_by_token(size, dt, gt):
    for state in (True, False):
        x = inputs(*size, dt, gt, size[0], 7 * size[1] + size[4], state)
        check(x, label="%s state %d" % (size, state))


CHUNK_SIZES = [(1, 17, 1, 1, 128, 128), (2, 63, 2, 1, 128, 128), (1, 64, 2, 2, 128, 128),
               (1, 65, 1, 1, 64, 64), (2, 128, 2, 2, 64, 128), (1, 130, 4, 2, 128, 64),
               (1, 200, 1, 1, 8, 16), (1, 333, 2, 2, 96, 120), (3, 256, 1, 1, 128, 128)]


@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("size", CHUNK_SIZES)
def test_chunks(size, gt):
    for state in (True, False):
        x = inputs(*size, BF, gt, size[0], size[1] + size[4], state)
        check(x, label="%s state %d" % (size, state))


@pytest.mark.parametrize("size", [(1, 150, 2, 2, 40, 24), (2, 77, 3, 1, 128, 128)])
def test_fp32(size):
    check(inputs(*size, F32, F32, size[0], 5), label=str(size))


PACKS = [[0, 5], [0, 0, 0, 7, 7, 8, 30, 30], [0, 64, 128, 129, 193], [0, 20, 21, 21, 300],
         [0, 1, 2, 3, 100, 101, 260], list(range(0, 33)) + [100], []]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("pack", range(len(PACKS)))
def test_packed(pack, dt):
    cu = PACKS[pack] or [0]
    x = inputs(1, cu[-1], 2, 1, 32, 40, dt, F32, len(cu) - 1, pack)
    check(x, cu=cu, label="pack %s" % cu)


@pytest.mark.parametrize("size", [(1, 2100, 1, 1, 128, 128), (2, 1601, 2, 1, 64, 40)])
def test_segments(size):
    # few heads, long sequences: segments at once, joined by a scan over their states
    for state in (True, False):
        x = inputs(*size, BF, F32, size[0], 9, state)
        check(x, label="%s state %d" % (size, state))


def test_segments_packed():
    # one long sequence among short and empty ones: segments past a sequence's end
    cu = [0, 0, 30, 1700, 1700, 1764]
    check(inputs(1, cu[-1], 1, 1, 32, 24, BF, F32, len(cu) - 1, 4), cu=cu)


def test_scale():
    check(inputs(1, 100, 2, 1, 64, 64, BF, F32, 1, 3), scale=1.0)
    check(inputs(1, 10, 2, 1, 64, 64, BF, F32, 1, 3), scale=0.0)
