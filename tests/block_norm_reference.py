"""The norms around a block in fp64 from their definition, their gradients by the formulas, and
for each the magnitude of the terms that fp32 arithmetic rounds.  CPU tensors in and out."""
import torch


def act(z, kind):
    """The gate's factor and its slope."""
    if kind == "none":
        return z, torch.ones_like(z)
    s = torch.sigmoid(z)
    if kind == "sigmoid":
        return s, s * (1 - s)
    return z * s, s * (1 + z * (1 - s))


def block_norm(x, gate=None, residual=None, post=None, pre=None, activation="silu", scale=1.0,
               eps=1e-6, dh=None, dy=None):
    """{"h", "y"} and, with dh or dy, {"dx", "dgate", "dres", "dpost", "dpre"}; "*_s": the sum of
    the magnitudes of what each value is made of."""
    up = lambda t: None if t is None else t.double()
    x, gate, residual, post, pre, dh, dy = map(up, (x, gate, residual, post, pre, dh, dy))
    out = {}
    rx, n = torch.ones(()).double(), x
    if post is not None:
        rx = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        n = x * rx * post
    f, slope = act(gate, activation) if gate is not None else (torch.ones_like(x),) * 2
    m = scale * n * f
    h = m + residual if residual is not None else m
    out["h"], out["h_s"] = h, m.abs() + (residual.abs() if residual is not None else 0)
    if pre is not None:
        rh = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
        out["y"], out["y_s"] = h * rh * pre, out["h_s"] * rh * pre.abs()
    if dh is None and dy is None:
        return out
    lead = tuple(range(x.ndim - 1))
    d = dh if dh is not None else torch.zeros_like(x)
    s = d.abs()
    if dy is not None:
        u = dy * pre
        d = d + rh * (u - h * rh.square() * (u * h).mean(-1, keepdim=True))
        s = s + rh * (u.abs() + out["h_s"] * rh.square() *
                      (u.abs() * out["h_s"]).mean(-1, keepdim=True))
        out["dpre"] = (dy * h * rh).sum(lead)
        out["dpre_s"] = (dy.abs() * out["h_s"] * rh).sum(lead)
    out["dres"], out["dres_s"] = d, s
    d, s = scale * d, abs(scale) * s
    out["dgate"], out["dgate_s"] = d * n * slope, s * n.abs() * (slope.abs() + f.abs())
    d, s = d * f, s * f.abs()
    if post is not None:
        out["dpost"], out["dpost_s"] = (d * x * rx).sum(lead), (s * x.abs() * rx).sum(lead)
        u, us = d * post, s * post.abs()
        d = rx * (u - x * rx.square() * (u * x).mean(-1, keepdim=True))
        s = rx * (us + x.abs() * rx.square() * (us * x.abs()).mean(-1, keepdim=True))
    out["dx"], out["dx_s"] = d, s
    return out
