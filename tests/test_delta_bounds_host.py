"""The bounds of delta_bounds.py on the CPU: the definition's outputs, rounded, are within them,
and mistakes planted in them are not, in every output."""
import pytest
import torch

import delta_bounds as DB
import delta_reference as R

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("o", "final", "dq", "dk", "dv", "dg", "dbeta", "dinit")


def outputs(B, T, H, HK, D, E, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    v = rnd(B, T, H, E)
    return v, R.delta(unit(rnd(B, T, HK, D)), unit(rnd(B, T, HK, D)), v,
                      -torch.exp(rnd(B, T, H) * 1.5 - 3.0), torch.sigmoid(rnd(B, T, H)), D ** -0.5,
                      rnd(B, H, D, E) * 0.2, None, rnd(B, T, H, E), rnd(B, H, D, E) * 0.2)


def plants(name, x):
    """Copies of x with a mistake each."""
    yield "zero", torch.zeros_like(x)
    yield "half", 0.5 * x
    if name in ("final", "dinit"):
        y = x.clone()
        y[:, -1] = 0
        yield "a head lost", y
        y = x.clone()
        y[..., -8:] = y[..., :8]
        yield "columns in another's place", y
        return
    y = x.clone()
    y[:, -1] = 0
    yield "the last token lost", y
    y = x.clone()
    y[:, :, 0] = y[:, :, -1] if x.shape[2] > 1 else -y[:, :, 0]
    yield "a head in another's place", y
    y = x.clone()
    y[:, x.shape[1] // 2:] *= 1.05
    yield "half of the tokens 5% off", y


@pytest.mark.parametrize("dt,tc,size", [
    (F32, False, (1, 150, 2, 2, 40, 24)), (F32, False, (2, 77, 3, 1, 128, 128)),
    (BF, False, (3, 2, 4, 2, 64, 64)), (BF, True, (2, 256, 2, 1, 64, 64)),
    (BF, True, (1, 1600, 1, 1, 64, 40))])
def test_planted_mistakes_are_beyond_the_bounds(dt, tc, size):
    v, ref = outputs(*size, 3)
    terms = DB.terms_of(v, ref["dv"])
    for name in NAMES:
        x = ref[name]
        held = x.to(F32 if name in ("final", "dinit") else dt).double()
        assert not DB.faults(name, held, x, dt, tc, size[1], terms), name
        for what, wrong in plants(name, x):
            assert DB.faults(name, wrong, x, dt, tc, size[1], terms), (name, what)
