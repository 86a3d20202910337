"""The gated delta rule in fp64, token by token, with its chain rule back: written from the
definition, no chunks, no code of the package.  CPU tensors in and out."""
import torch


def spans(B, T, cu):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = [int(v) for v in cu]
    return [(0, c[n], c[n + 1]) for n in range(len(c) - 1)]


def delta(q, k, v, g, beta, scale, init=None, cu=None, do=None, dfin=None):
    """{"o", "final"} and, with do, the gradients {"dq", "dk", "dv", "dg", "dbeta", "dinit"};
    "scale_S", "scale_K" [N, H]: the largest norm of the state and of its gradient on the way."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    B, T, H, E = v.shape
    HK, D = q.shape[2:]
    group = H // HK
    seqs = spans(B, T, cu)
    N = len(seqs)
    out = {"o": torch.zeros_like(v), "final": torch.zeros(N, H, D, E, dtype=torch.float64),
           "scale_S": torch.zeros(N, H, dtype=torch.float64),
           "scale_K": torch.zeros(N, H, dtype=torch.float64)}
    if do is not None:
        do = do.double()
        for name, like in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            out[name] = torch.zeros_like(like)
        out["dinit"] = torch.zeros_like(out["final"])
    for n, (b, lo, hi) in enumerate(seqs):
        S = init[n].double() if init is not None else torch.zeros(H, D, E, dtype=torch.float64)
        out["scale_S"][n] = S.flatten(1).norm(dim=1)
        kept = []
        for t in range(lo, hi):
            kt, qt = (x[b, t].repeat_interleave(group, 0) for x in (k, q))
            Sp = g[b, t].exp()[:, None, None] * S
            e = v[b, t] - torch.einsum("hde,hd->he", Sp, kt)
            S = Sp + kt[:, :, None] * (beta[b, t][:, None] * e)[:, None]
            out["o"][b, t] = scale * torch.einsum("hde,hd->he", S, qt)
            out["scale_S"][n] = torch.maximum(out["scale_S"][n], S.flatten(1).norm(dim=1))
            kept.append((kt, qt, Sp, e, S))
        out["final"][n] = S
        if do is None:
            continue
        K = dfin[n].double() if dfin is not None else torch.zeros_like(S)
        out["scale_K"][n] = K.flatten(1).norm(dim=1)
        for t in range(hi - 1, lo - 1, -1):
            kt, qt, Sp, e, S = kept[t - lo]
            d = do[b, t]
            out["dq"][b, t] += (scale * torch.einsum("hde,he->hd", S, d)).reshape(
                HK, group, D).sum(1)
            K = K + scale * qt[:, :, None] * d[:, None]
            out["scale_K"][n] = torch.maximum(out["scale_K"][n], K.flatten(1).norm(dim=1))
            w = torch.einsum("hde,hd->he", K, kt)
            dv = beta[b, t][:, None] * w
            out["dv"][b, t] = dv
            out["dbeta"][b, t] = (w * e).sum(-1)
            dk = torch.einsum("hde,he->hd", K, beta[b, t][:, None] * e) - \
                torch.einsum("hde,he->hd", Sp, dv)
            out["dk"][b, t] += dk.reshape(HK, group, D).sum(1)
            K = K - kt[:, :, None] * dv[:, None]
            out["dg"][b, t] = (K * Sp).sum((1, 2))
            K = g[b, t].exp()[:, None, None] * K
        out["dinit"][n] = K
    return out
