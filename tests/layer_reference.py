"""fp64 restatements of the operators beside the attention, written from their definitions
(token by token, no tiles, no code of the package), with bounds on the fp32 rounding of any
evaluation order.  CPU tensors in and out."""
import torch

U = 2.0 ** -24            # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def spans(B, T, cu):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = [int(v) for v in cu]
    return [(0, c[n], c[n + 1]) for n in range(len(c) - 1)]


def scan(x, g, init=None, reverse=False, cu=None, do=None, dfin=None):
    """The gated recurrence and, with do, its gradients, with an error scale for each output:
    every evaluation in fp32 of the recurrence stays within (a few) U times the scale,
    E_t = a_t E_{t-1} + S_t with S the recurrence of |x|: one relative rounding of the
    running magnitude a token, carried on as the recurrence carries errors."""
    x, g = x.double(), g.double()
    B, T, H, D = x.shape
    seqs = spans(B, T, cu)
    out = {n: torch.zeros_like(x) for n in ("o", "o_e", "prev", "prev_e")}
    fin = torch.zeros(len(seqs), H, D, dtype=torch.float64)
    fin_e = torch.zeros_like(fin)
    a = g.exp()
    for n, (b, lo, hi) in enumerate(seqs):
        s = init[n].double() if init is not None else torch.zeros(H, D, dtype=torch.float64)
        m, e = s.abs(), torch.zeros_like(s)
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            out["prev"][b, t], out["prev_e"][b, t] = s, e
            s = a[b, t] * s + x[b, t]
            m = a[b, t] * m + x[b, t].abs()
            e = a[b, t] * e + m
            out["o"][b, t], out["o_e"][b, t] = s, e
        fin[n], fin_e[n] = s, e
    out["final"], out["final_e"] = fin, fin_e
    if do is None:
        return out
    do = do.double()
    for name in ("dx", "dx_e", "dg", "dg_e"):
        out[name] = torch.zeros_like(x)
    dinit, dinit_e = torch.zeros_like(fin), torch.zeros_like(fin)
    for n, (b, lo, hi) in enumerate(seqs):
        K = dfin[n].double() if dfin is not None else torch.zeros(H, D, dtype=torch.float64)
        m, e = K.abs(), torch.zeros_like(K)
        for t in (range(lo, hi) if reverse else range(hi - 1, lo - 1, -1)):
            G = do[b, t] + K
            mg = do[b, t].abs() + m
            out["dx"][b, t], out["dx_e"][b, t] = G, e + mg
            K, m, e = a[b, t] * G, a[b, t] * mg, a[b, t] * (e + 2 * mg)
            p, pe = out["prev"][b, t], out["prev_e"][b, t]
            out["dg"][b, t] = K * p
            out["dg_e"][b, t] = e * p.abs() + K.abs() * pe + (K * p).abs()
        dinit[n], dinit_e[n] = K, e
    out["dinit"], out["dinit_e"] = dinit, dinit_e
    return out


def positions_of(B, T, cu, offset=None):
    """The default positions [1, B, T]: the index in the sequence, plus its offset."""
    p = torch.zeros(1, B, T, dtype=torch.int64)
    for n, (b, lo, hi) in enumerate(spans(B, T, cu)):
        p[0, b, lo:hi] = torch.arange(hi - lo) + (int(offset[n]) if offset is not None else 0)
    return p


def norm_rope(x, w=None, eps=1e-6, normalize=True, inv_freq=None, axes=None, positions=None,
              interleaved=False):
    """y for x [B,T,H,D] (fp64, differentiable); positions [axes, B, T]."""
    y = x
    if normalize:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w
    if inv_freq is None:
        return y
    pairs = len(inv_freq)
    parts = [y[..., c] for c in range(x.shape[-1])]
    for j in range(pairs):
        ax = axes[j] if axes is not None else 0
        th = (positions[ax].double() * float(inv_freq[j]))[..., None]
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        u, v = parts[i], parts[k]
        parts[i], parts[k] = u * th.cos() - v * th.sin(), u * th.sin() + v * th.cos()
    return torch.stack(parts, -1)
