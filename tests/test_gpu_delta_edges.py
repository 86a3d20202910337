"""The gated delta rule on the GPU where it can go wrong: neighbours that are not finite, gates
that forget all, keys that repeat, layouts, places given by the caller, streams, graphs, autograd,
offsets beyond 32 bits, a hand-off that never comes; and a run of it with the norms around it.
Tolerances as test_gpu_delta.py."""
import math
import time

import pytest
import torch

import block_norm_reference as RN
import delta_reference as R
import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import _native as N
from test_gpu_delta import BF, F32, check, cuda, inputs

pytestmark = pytest.mark.gpu


def args(d):
    return d["q"], d["k"], d["v"], d["g"], d["beta"]


def run(d, cu=None, **kw):
    """(o, final, dq, dk, dv, dg, dbeta, dinit)"""
    cu_t = torch.tensor(cu, dtype=torch.int32) if cu is not None else None
    kw.update(initial_state=d["init"], cu_seqlens=cu_t.cuda() if cu is not None else None,
              cu_seqlens_host=cu_t)
    o, fin, saved = la.gated_delta_fwd(*args(d), keep=True, **kw)
    return (o, fin) + tuple(la.gated_delta_bwd(*args(d), d["do"], d_final_state=d["dfin"],
                                               saved=saved, **kw))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_neighbours_that_are_not_finite(dt, bad):
    # sequence 1's tokens and states are all `bad`: the others come out as beside zeros
    cu = [0, 30, 75, 76, 200]
    x = cuda(inputs(1, cu[-1], 2, 1, 40, 48, dt, F32, len(cu) - 1, 3))
    outs = []
    for fill in (0.0, bad):
        d = {n: t.clone() for n, t in x.items()}
        for n in ("q", "k", "v", "g", "beta", "do"):
            d[n][:, cu[1]:cu[2]] = fill
        for n in ("init", "dfin"):
            d[n][1] = fill
        outs.append(run(d, cu))
    keep = torch.ones(cu[-1], dtype=torch.bool, device="cuda")
    keep[cu[1]:cu[2]] = False
    seqs = torch.tensor([0, 2, 3], device="cuda")
    for i, (a, b) in enumerate(zip(*outs)):
        a, b = (a[seqs], b[seqs]) if i in (1, 7) else (a[:, keep], b[:, keep])
        assert torch.isfinite(a).all() and torch.equal(a, b), i


@pytest.mark.parametrize("dt,T", [(BF, 200), (F32, 60)])
def test_gates_that_forget_all(dt, T):
    x = inputs(1, T, 2, 2, 64, 64, dt, F32, 1, 5)
    for t in {0, 17, 18, min(63, T - 2), min(64, T - 2), T - 1}:
        x["g"][:, t] = -math.inf
    x["g"][:, 40] = -1e4
    check(x, label="resets")
    x["g"].zero_()
    check(x, label="nothing forgotten")


@pytest.mark.parametrize("dt,T", [(BF, 190), (F32, 50)])
def test_repeated_keys_and_strengths(dt, T):
    x = inputs(1, T, 2, 1, 32, 32, dt, F32, 1, 6)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:, :, 0] = 1.0
    x["beta"][:, ::3, 1] = 0.0
    x["g"].mul_(0.1)
    check(x, label="one key")
    x["beta"].zero_()
    check(x, label="nothing written")
    x["k"].zero_()
    x["beta"].fill_(1.0)
    check(x, label="zero keys")


def test_layouts():
    B, T, H, D = 2, 150, 2, 64
    x = inputs(B, T, H, H, D, D, BF, BF, B, 8)
    # q, k, v as slices of one projection
    d = cuda(x)
    wide = torch.cat((d["q"], d["k"], d["v"]), 3).contiguous()
    d["q"], d["k"], d["v"] = wide[..., :D], wide[..., D:2 * D], wide[..., 2 * D:]
    check(x, label="slices", dev=d)
    # heads before tokens, gates channel-last of a wider projection
    d = cuda(x)
    for n in ("q", "k", "v", "do"):
        d[n] = d[n].transpose(1, 2).contiguous().transpose(1, 2)
    gates = torch.stack((d["g"], d["beta"]), 3).contiguous()
    d["g"], d["beta"] = gates[..., 0], gates[..., 1]
    check(x, label="heads first", dev=d)
    # rows off 16 bytes: copied for the backward; the forward alone goes token by token
    d = cuda(x)
    for n in ("q", "k", "v", "do"):
        w = torch.zeros(B, T, H, D + 1, dtype=BF, device="cuda")
        w[..., 1:] = d[n]
        d[n] = w[..., 1:]
    want = run(cuda(x))
    for a, b in zip(want, run(d)):
        assert torch.equal(a, b)
    o, fin = la.gated_delta_fwd(*args(d), initial_state=d["init"])
    assert float((fin - want[1]).norm()) <= 1e-4 * float(want[1].norm())
    assert float((o.float() - want[0].float()).norm()) <= 2.0 ** -7 * float(want[0].float().norm())


@pytest.mark.parametrize("T", [1, 100, 1300])
def test_places_of_the_caller(T):
    x = cuda(inputs(1, T, 2, 2, 64, 64, BF, BF, 1, 9))
    o, fin = la.gated_delta_fwd(*args(x), initial_state=x["init"])
    state = x["init"].clone()
    out = torch.full((1, T, 2, 96), 7.0, dtype=BF, device="cuda")
    got = la.gated_delta_fwd(*args(x), initial_state=state, final_state=state,
                             out=out[..., :64])
    assert got[1] is state and torch.equal(state, fin) and torch.equal(out[..., :64], o)
    assert (out[..., 64:] == 7.0).all()
    assert la.gated_delta_fwd(*args(x), want_final_state=False)[1] is None


def test_nothing_to_do():
    for B, T in ((0, 50), (2, 0), (0, 0)):
        x = cuda(inputs(B, T, 2, 1, 64, 64, BF, BF, B, 1))
        out = run(x)
        assert out[0].shape == (B, T, 2, 64)
        assert torch.equal(out[1], x["init"]) and torch.equal(out[7], x["dfin"])


@pytest.mark.parametrize("T,H", [(1, 2), (130, 2), (1500, 1)])
def test_captured(T, H):
    x = cuda(inputs(2, T, H, 1, 64, 64, BF, F32, 2, 10))
    want = run(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(x)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x)
    y = cuda(inputs(2, T, H, 1, 64, 64, BF, F32, 2, 11))
    for values, ref in ((x, want), (y, run(y))):
        for n in x:
            x[n].copy_(values[n].clone())
        graph.replay()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_streams_at_once():
    # the same sizes on two streams, each with workspaces of its own
    xs = [cuda(inputs(2, 400, 4, 2, 128, 128, BF, F32, 2, s)) for s in (1, 2)]
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(xs[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dt,T", [(BF, 90), (F32, 20)])
def test_autograd(dt, T):
    cu = [0, 7, T]
    x = cuda(inputs(1, T, 4, 2, 32, 32, dt, F32, 2, 12))
    cu_t = torch.tensor(cu, dtype=torch.int32)
    want = run(x, cu)
    leaves = {n: x[n][0].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    init = x["init"].clone().requires_grad_()
    o, fin = la.gated_delta(*leaves.values(), initial_state=init, cu_seqlens=cu_t.cuda())
    assert torch.equal(o, want[0][0]) and torch.equal(fin, want[1])
    (o * x["do"][0]).sum().add((fin * x["dfin"]).sum()).backward()
    for (n, t), w in zip(leaves.items(), want[2:7]):
        assert t.grad.dtype == t.dtype
        assert torch.equal(t.grad, w[0].to(t.dtype)), n
    assert torch.equal(init.grad, want[7])
    # the state alone is differentiated, and nothing is
    fin = la.gated_delta(*leaves.values(), cu_seqlens=cu_t.cuda())[1]
    fin.sum().backward()
    with torch.no_grad():
        la.gated_delta(*leaves.values(), cu_seqlens=cu_t.cuda())


def test_states_beyond_32_bits():
    # 272 x 512 states of 128 x 128: 2.28e9 numbers
    n, H, D = 272, 512, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    state = torch.empty(n, H, D, D, device="cuda").normal_(generator=gen)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)
    q, k, v = rnd(n, 1, H, D), rnd(n, 1, H, D) * D ** -0.5, rnd(n, 1, H, D)
    g = -torch.rand(n, 1, H, generator=gen, device="cuda")
    beta = torch.rand(n, 1, H, generator=gen, device="cuda")
    tail = slice(n - 2, n)
    part = state[tail].clone()
    want = la.gated_delta_fwd(q[tail], k[tail], v[tail], g[tail], beta[tail], initial_state=part)
    o, fin = la.gated_delta_fwd(q, k, v, g, beta, initial_state=state, final_state=state)
    assert torch.equal(o[tail], want[0]) and torch.equal(fin[tail], want[1])


def test_tokens_beyond_32_bits():
    # 2 x 33000 tokens of 256 heads of 128: 2.16e9 numbers; the last heads alone are the same
    B, T, H, D, part = 2, 33000, 256, 128, 80
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rows(unit):
        t = torch.empty(B, T, H, D, dtype=BF, device="cuda")
        for b in range(B):
            for h in range(0, H, 32):
                x = torch.randn(T, 32, D, generator=gen, device="cuda")
                t[b, :, h:h + 32] = x / x.norm(dim=-1, keepdim=True) if unit else x
        return t
    q, k, v = rows(True), rows(True), rows(False)
    g = -0.1 * torch.rand(B, T, H, generator=gen, device="cuda")
    beta = torch.rand(B, T, H, generator=gen, device="cuda")
    o, fin = la.gated_delta_fwd(q, k, v, g, beta)
    cut = [t[:, :, -part:] for t in (q, k, v, g, beta)]
    o2, fin2 = la.gated_delta_fwd(*cut)
    assert torch.equal(o[:, :, -part:], o2) and torch.equal(fin[:, -part:], fin2)


@pytest.mark.parametrize("T", [300, 2000])
def test_withheld_handoff(T):
    # one warp leaves out a hand-off: the waits for it run out, the error reaches the host, the
    # context goes on
    x = cuda(inputs(1, T, 2, 2, 64, 64, BF, F32, 1, 13))
    la.get_device_error()
    for backward in (False, True):
        want = run(x)
        saved = la.gated_delta_fwd(*args(x), initial_state=x["init"], keep=True)[2]
        N.check(N.lib().la_debug_withhold_next_handoff(1))
        t0 = time.time()
        if backward:
            la.gated_delta_bwd(*args(x), x["do"], initial_state=x["init"],
                               d_final_state=x["dfin"], saved=saved)
        else:
            la.gated_delta_fwd(*args(x), initial_state=x["init"])
        with pytest.raises(N.LaError) as err:
            la.get_device_error()
        assert err.value.status == N.LA_ERR_TIMEOUT
        assert time.time() - t0 < 60
        la.get_device_error()
        for a, b in zip(run(x), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,at", [(12, 5), (300, 100)])
def test_a_gate_that_is_not_a_number(T, at):
    # it shows: in every output of its head from its token on, and in no other head
    x = cuda(inputs(1, T, 2, 2, 64, 64, BF, F32, 1, 17))
    want = la.gated_delta_fwd(*args(x), initial_state=x["init"])
    x["g"][0, at, 1] = math.nan
    o, fin = la.gated_delta_fwd(*args(x), initial_state=x["init"])
    assert torch.equal(o[:, :, 0], want[0][:, :, 0]) and torch.equal(fin[:, 0], want[1][:, 0])
    assert o[:, at:, 1].isnan().all() and fin[:, 1].isnan().all()
    before = at // 64 * 64 if T > 16 else at
    assert torch.equal(o[:, :before, 1], want[0][:, :before, 1])


def test_refused_tensors():
    x = cuda(inputs(1, 20, 4, 2, 64, 64, BF, F32, 1, 1))
    with pytest.raises(ValueError, match="divide"):
        la.gated_delta_fwd(x["q"][:, :, :1].expand(1, 20, 3, 64), x["k"][:, :, :1].expand(
            1, 20, 3, 64), x["v"], x["g"], x["beta"])
    with pytest.raises(ValueError, match="g must be"):
        la.gated_delta_fwd(x["q"], x["k"], x["v"], x["g"][:, :, :2], x["beta"])
    with pytest.raises(TypeError, match="share one dtype"):
        la.gated_delta_fwd(x["q"], x["k"], x["v"], x["g"].to(BF), x["beta"])
    with pytest.raises(TypeError, match="float32"):
        la.gated_delta_fwd(x["q"], x["k"], x["v"], x["g"].double(), x["beta"].double())
    with pytest.raises(TypeError):
        la.gated_delta_fwd(x["q"].float(), x["k"], x["v"], x["g"], x["beta"])
    with pytest.raises(ValueError, match="saved"):
        la.gated_delta_bwd(*args(x), x["do"], saved=torch.empty(8, dtype=torch.uint8,
                                                                device="cuda"))
    with pytest.raises(N.LaError):
        la.gated_delta_fwd(*args(x), cu_seqlens=[0, 5, 19])
    with pytest.raises(ValueError, match="final_state"):
        la.gated_delta_fwd(*args(x), final_state=torch.empty(1, 4, 64, 32, device="cuda"))


def test_a_block_of_them_together():
    # norm of the stream, queries and keys of length one, the rule, its heads normalised and
    # gated, the stream again: forward and gradients against fp64
    B, T, H, D = 1, 40, 2, 8
    C = H * D
    gen = torch.Generator().manual_seed(14)
    rnd = lambda *s: torch.randn(s, generator=gen)
    p = {"stream": rnd(B, T, C), "pre": 1 + 0.1 * rnd(C), "wq": 0.3 * rnd(C, C),
         "wk": 0.3 * rnd(C, C), "wv": 0.3 * rnd(C, C), "wz": 0.3 * rnd(C, C),
         "wg": 0.3 * rnd(C, H), "wb": 0.3 * rnd(C, H), "post": 1 + 0.1 * rnd(D),
         "next": 1 + 0.1 * rnd(C)}
    dh, dy = rnd(B, T, C), rnd(B, T, C)
    heads = lambda t: t.unflatten(-1, (H, D))

    def block(p, own):
        x = p["stream"]
        if own:
            n = la.block_norm(x, post_weight=p["pre"])[0]
        else:
            n = RN.block_norm(x, post=p["pre"])["h"]
        q, k, v, z = (heads(n @ p[w]) for w in ("wq", "wk", "wv", "wz"))
        g = -torch.nn.functional.softplus(n @ p["wg"])
        beta = torch.sigmoid(n @ p["wb"])
        if own:
            unit = torch.full((D,), D ** -0.5, device=x.device)
            q, k = la.qk_norm_rope(q, k, la.QkNorm(unit, unit, 1e-6))
            o, _ = la.gated_delta(q, k, v, g, beta)
            o = la.block_norm(o, z, post_weight=p["post"])[0]
            return la.block_norm(o.flatten(2), residual=x, pre_weight=p["next"], scale=0.5)
        q, k = (t * D ** -0.5 / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
        S = torch.zeros(B, H, D, D, dtype=torch.float64)
        o = []
        for t in range(T):
            S = g[:, t].exp()[..., None, None] * S
            e = v[:, t] - torch.einsum("bhde,bhd->bhe", S, k[:, t])
            S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
            o.append(D ** -0.5 * torch.einsum("bhde,bhd->bhe", S, q[:, t]))
        o = RN.block_norm(torch.stack(o, 1), z, post=p["post"])["h"]
        r = RN.block_norm(o.flatten(2), residual=x, pre=p["next"], scale=0.5)
        return r["h"], r["y"]

    grads = []
    for own in (False, True):
        q = {n: (t.cuda() if own else t.double()).requires_grad_() for n, t in p.items()}
        h, y = block(q, own)
        dev = (dh.cuda(), dy.cuda()) if own else (dh.double(), dy.double())
        ((h * dev[0]).sum() + (y * dev[1]).sum()).backward()
        grads.append([t.detach().cpu().double() for t in (h, y)] +
                     [t.grad.cpu().double() for t in q.values()])
    # fp32 throughout: a few hundred roundings of 2^-24 in a row, sums over 40 tokens
    for a, b, name in zip(*grads, ["h", "y"] + list(p)):
        assert float((a - b).norm()) <= 2e-4 * float(a.norm()) + 1e-6, name
