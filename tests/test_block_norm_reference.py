"""The fp64 references of the new operators' tests against differences of their own forward, on
the CPU: a formula that the GPU tests hold kernels to is itself held to the definition."""
import pytest
import torch

import block_norm_reference as RN
import delta_reference as RD


def _differences(loss, x, got, steps=8, seed=0):
    """Central differences of loss along random directions of x against <got, direction>."""
    gen = torch.Generator().manual_seed(seed)
    for _ in range(steps):
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        num = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
        want = float((got * d).sum())
        assert abs(float(num) - want) <= 1e-6 * (1 + abs(want)) + 1e-7, (float(num), want)


@pytest.mark.parametrize("activation", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("use", ["all", "post", "pre", "stream"])
def test_block_norm(use, activation):
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    t = {"x": rnd(3, 5, 12), "gate": rnd(3, 5, 12), "residual": rnd(3, 5, 12), "post": rnd(12),
         "pre": rnd(12)}
    drop = {"all": (), "post": ("pre", "residual"), "pre": ("post", "gate"),
            "stream": ("pre", "post")}[use]
    for n in drop:
        t[n] = None
    dh = rnd(3, 5, 12)
    dy = rnd(3, 5, 12) if t["pre"] is not None else None
    kw = dict(activation=activation, scale=0.7)
    ref = RN.block_norm(**t, **kw, dh=dh, dy=dy)

    def loss(name):
        def f(v):
            o = RN.block_norm(**{**t, name: v}, **kw)
            return (o["h"] * dh).sum() + ((o["y"] * dy).sum() if dy is not None else 0)
        return f

    names = {"x": "dx", "gate": "dgate", "residual": "dres", "post": "dpost", "pre": "dpre"}
    for name, grad in names.items():
        if t[name] is not None:
            _differences(loss(name), t[name], ref[grad])


@pytest.mark.parametrize("cu", [None, [0, 0, 3, 7]])
def test_delta(cu):
    gen = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    B, T, H, HK, D, E = 1, 7, 4, 2, 3, 5
    N = B if cu is None else len(cu) - 1
    k = rnd(B, T, HK, D)
    t = {"q": rnd(B, T, HK, D), "k": k / k.norm(dim=-1, keepdim=True), "v": rnd(B, T, H, E),
         "g": -rnd(B, T, H).abs(), "beta": torch.sigmoid(rnd(B, T, H)), "init": rnd(N, H, D, E)}
    do, dfin = rnd(B, T, H, E), rnd(N, H, D, E)
    ref = RD.delta(**t, scale=0.6, cu=cu, do=do, dfin=dfin)

    def loss(name):
        def f(v):
            o = RD.delta(**{**t, name: v}, scale=0.6, cu=cu)
            return (o["o"] * do).sum() + (o["final"] * dfin).sum()
        return f

    for name in t:
        _differences(loss(name), t[name], ref["d" + name], steps=4)
    # dg as a running sum, the form the kernels use
    o = ref["o"]
    c = (do * o).sum(-1) - (t["v"] * ref["dv"]).sum(-1)
    for n, (b, lo, hi) in enumerate(RD.spans(B, T, cu)):
        if hi > lo:
            end = (ref["final"][n] * dfin[n]).sum((1, 2))
            want = c[b, lo:hi].flip(0).cumsum(0).flip(0) + end
            assert torch.allclose(want, ref["dg"][b, lo:hi], atol=1e-10)
