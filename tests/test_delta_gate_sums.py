"""The running sums of a chunk's gates as csrc/la_delta_tc.cu keeps them, restated on the CPU in
fp32: sums of two floats over 64 tokens, times log2 e, and the decays M_ij = e^(G_i - G_j) and
kappa_j = e^(G_C - G_j) made of their differences.  Strong gates (a reset is taken as -100) leave
sums of thousands before slow gates of a thousandth; one float a sum loses those."""
import numpy as np
import pytest

F = np.float32
C = 64
L2E_HI = F(1.4426950408889634)
L2E_LO = F(1.4426950408889634 - float(L2E_HI))


def gates(kind, seed):
    rng = np.random.default_rng(seed)
    g = -np.exp(rng.standard_normal(C) * 1.5 - 3.0)
    if kind == "strong":
        g[:32] = -rng.uniform(3.0, 8.0, 32)
    elif kind != "slow":
        g[rng.permutation(40)[:kind]] = -100.0
    return g.astype(F)


def add_one(a, b):
    return (a[0] + b[0], F(0))


def add_two(a, b):
    s = F(a[0] + b[0])
    t = F(s - a[0])
    e = F(F(a[0] - F(s - t)) + F(b[0] - t))
    e = F(e + F(a[1] + b[1]))
    hi = F(s + e)
    return hi, F(e - F(hi - s))


def fma(a, b, c):
    return F(float(a) * float(b) + float(c))    # exact in 64 bits but for the last sum


def to_log2(x, two):
    if not two:
        return F(x[0] * L2E_HI), F(0)
    p = F(x[0] * L2E_HI)
    e = fma(x[0], L2E_HI, -p)
    e = fma(x[0], L2E_LO, fma(x[1], L2E_HI, e))
    hi = F(p + e)
    return hi, F(e - F(hi - p))


def running(g, two):
    """Inclusive sums over two warps of 32, the second's after the first's last."""
    add = add_two if two else add_one
    x = [(v, F(0)) for v in g]
    for m in (1, 2, 4, 8, 16):
        x = [add(x[i], x[i - m]) if i % 32 >= m else x[i] for i in range(C)]
    return [x[i] if i < 32 else add(x[i], x[31]) for i in range(C)]


def worst(g, two):
    """Largest relative errors of M and kappa where they are above 2^-30, beside |d| (in powers
    of two), and whether both stay within two roundings of a difference."""
    exact = np.concatenate(([0.0], np.cumsum(g.astype(np.longdouble))))[1:]
    G = running(g, two)
    P = [to_log2(x, two) for x in G]
    most_m = most_k = 0.0
    fine = True
    for i in range(C):
        for j in range(i + 1):
            d = float(F(F(P[i][0] - P[j][0]) + F(P[i][1] - P[j][1])))
            want = float(exact[i] - exact[j]) * 1.4426950408889634
            if want > -30:
                off = abs(np.expm1((d - want) * np.log(2)))
                most_m = max(most_m, off)
                fine = fine and off <= 2.0 ** -23 * abs(want) + 1e-9
        d = float(F(F(G[C - 1][0] - G[i][0]) + F(G[C - 1][1] - G[i][1])))
        want = float(exact[C - 1] - exact[i])
        if want > -20:
            off = abs(np.expm1(d - want))
            most_k = max(most_k, off)
            fine = fine and off <= 2.0 ** -23 * abs(want) + 1e-9
    return most_m, most_k, fine


@pytest.mark.parametrize("kind", ["slow", "strong", 1, 4, 16, 32])
def test_two_floats_keep_the_decays(kind):
    for seed in range(4):
        m, k, fine = worst(gates(kind, seed), True)
        assert fine and m < 4e-6 and k < 4e-6, (kind, seed, m, k)


def test_one_float_does_not():
    # what the sums were: decays off by more than the states' bound of 1e-5
    for kind in ("strong", 16, 32):
        assert max(max(worst(gates(kind, seed), False)[:2]) for seed in range(4)) > 2e-5, kind
