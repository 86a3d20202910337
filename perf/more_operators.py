"""Cases of the gated delta rule (chunked over whole sequences, token by token with a carried
state) and of the norms around a block, fused with its gate and its residual scale.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once at
the end) or, with `own` set, by the calls that a user makes of this framework.  `exact` gives
the same outputs in fp64 from the definitions.
"""
import math

import torch

own = False

# bytes that a drawn case's tensors hold at most, and the tokens of its longest sequence
_MOST_BYTES = 1 << 29
_MOST_TOKENS = 16384


# ---------------------------------------------------------------------------
# cases

def _delta(name, **kw):
    c = {"op": "delta", "direction": "forward", "batch": 1, "tokens": 1, "heads": 32,
         "qk_heads": 32, "dim_qk": 128, "dim_v": 128, "dtype": "bf16", "gate": "fp32",
         "packed": 0, "low": 64, "high": 8192, "state": True}
    c.update(kw)
    c["name"] = name
    return c


def _norm(name, **kw):
    c = {"op": "norm", "direction": "forward", "batch": 1, "tokens": 1, "heads": 1, "dim": 4096,
         "dtype": "bf16", "weights": "same", "activation": "silu", "gate": True, "post": True,
         "pre": True, "residual": True, "scale": 1.0}
    c.update(kw)
    c["name"] = name
    return c


def listed():
    return [
        # one new token of each of 4 running sequences, the states in and out: latency
        _delta("delta_decode_b4", batch=4, gate="bf16"),
        # a full batch of running sequences, 16 query and key heads for 32 value heads: the
        # states' bytes
        _delta("delta_decode_b64", batch=64, qk_heads=16),
        # five proposed tokens of 24 sequences checked at once
        _delta("delta_verify_b24_n5", batch=24, tokens=5, gate="bf16"),
        # 16 prompts of 64 to 8192 tokens packed in one row, shared query and key heads
        _delta("delta_prompt_packed16", packed=16, heads=16, qk_heads=8),
        # one long document with few heads
        _delta("delta_long_n65536_h8", tokens=65536, heads=8, qk_heads=8),
        # a training step's forward and backward, the gated benchmark's shape
        _delta("delta_train_b4_n8192", batch=4, tokens=8192, direction="both", state=False),
        # narrow heads, an odd length, shared heads, with states
        _delta("delta_train_b2_n2047_d64", batch=2, tokens=2047, heads=8, qk_heads=4, dim_qk=64,
               dim_v=64, direction="both"),
        # fp32, odd sizes
        _delta("delta_train_fp32_n257_d33", batch=1, tokens=257, heads=2, qk_heads=2, dim_qk=33,
               dim_v=40, dtype="fp32", direction="both"),
        # one token of 64 sequences through a residual stream of 4096 channels: latency
        _norm("norm_residual_decode_b64", batch=64, gate=False, post=False),
        # the heads' outputs normalised and gated, forward and backward of a training step
        _norm("norm_gate_train_b4_n8192", batch=4, tokens=8192, heads=32, dim=128, pre=False,
              residual=False, direction="both"),
        # norms on both sides, gate and residual scale over the stream in training, odd length
        _norm("norm_block_train_b4_n4095", batch=4, tokens=4095, activation="sigmoid", scale=0.25,
              direction="both"),
        # fp32, odd channels: nothing is aligned
        _norm("norm_block_train_fp32_c1001", batch=3, tokens=1025, dim=1001, dtype="fp32",
              scale=0.5, direction="both"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw_norm(rng):
    dtype = "fp32" if rng.random() < 0.3 else "bf16"
    heads = rng.choice([1, 1, _log_int(rng, 2, 40)])
    dim = 8 * _log_int(rng, 1, 1024) if heads == 1 else rng.choice([64, 96, 128, 128, 192, 256])
    if rng.random() < 0.2:
        dim += rng.choice([-1, 1, 2])
    pre = rng.random() < 0.6
    post = not pre or rng.random() < 0.6
    rows = _log_int(rng, 1, max(2, _MOST_BYTES // (heads * dim * (4 if dtype == "fp32" else 2))
                                // 2))
    rows = min(rows, 1 << 17)
    batch = min(rows, _log_int(rng, 1, 16))
    return _norm("", batch=batch, tokens=max(1, rows // batch), heads=heads, dim=dim, dtype=dtype,
                 weights=rng.choice(["same", "fp32"]), pre=pre, post=post,
                 activation=rng.choice(["silu", "sigmoid", "none"]), gate=rng.random() < 0.6,
                 residual=pre or rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.3]),
                 direction=rng.choice(["forward", "both"]))


def draw(rng):
    if rng.random() < 0.35:
        c = _draw_norm(rng)
        del c["name"]
        return c
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    heads = _log_int(rng, 1, 40)
    qk = rng.choice([h for h in range(1, heads + 1) if heads % h == 0 and heads // h <= 4])
    width = rng.choice(["same", "same", "free"])
    D = rng.choice([64, 96, 128, 128, 8 * rng.randint(2, 16), rng.randint(1, 160)])
    E = D if width == "same" else rng.choice([64, 128, 8 * rng.randint(2, 16)])
    c = dict(heads=heads, qk_heads=qk, dim_qk=D, dim_v=E, dtype=dtype,
             gate="fp32" if dtype == "fp32" or rng.random() < 0.5 else "bf16",
             state=rng.random() < 0.7, direction=rng.choice(["forward", "both"]))
    most = max(2, _MOST_BYTES // (heads * max(D, E) * (4 if dtype == "fp32" else 2)))
    if dtype == "fp32" or D % 8 or E % 8 or D > 128:
        most = min(most, 4096)
    shape = rng.choice(["step", "dense", "dense", "packed"])
    if shape == "step":
        c.update(batch=min(_log_int(rng, 1, 96), most), tokens=rng.choice([1, 1, 2, 4, 7]),
                 direction="forward", state=True)
    elif shape == "packed":
        n = _log_int(rng, 1, 32)
        high = max(2, min(_MOST_TOKENS // 2, most // n))
        c.update(packed=n, low=rng.randint(1, max(1, high // 4)), high=high)
    else:
        b = min(_log_int(rng, 1, 8), max(1, most // 2))
        c.update(batch=b, tokens=_log_int(rng, 2, max(2, min(_MOST_TOKENS, most // b))))
    case = _delta("", **c)
    del case["name"]
    return case


def _lengths(case):
    """The sequences' lengths: when packed fixed by the case, spread over [low, high]."""
    if not case.get("packed"):
        return [case["tokens"]] * case["batch"]
    gen = torch.Generator().manual_seed(1000 * case["packed"] + case["low"] + case["high"])
    return torch.randint(case["low"], case["high"] + 1, (case["packed"],), generator=gen).tolist()


def _rows(case):
    """(batch rows, tokens a row)"""
    if case.get("packed"):
        return 1, sum(_lengths(case))
    return case["batch"], case["tokens"]


# ---------------------------------------------------------------------------
# inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    B, T = _rows(case)
    both = case["direction"] == "both"

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=gen, device="cuda")
        return x.mul_(std).add_(mean).to(dtype)

    def uniform(*shape, low, high):
        return torch.rand(shape, generator=gen, device="cuda").mul_(high - low).add_(low)

    st = {"case": case}
    if case["op"] == "norm":
        shape = (B, T, case["heads"], case["dim"]) if case["heads"] > 1 else (B, T, case["dim"])
        wt = torch.float32 if case["weights"] == "fp32" else dt
        st["x"] = normal(*shape)
        st["gate"] = normal(*shape) if case["gate"] else None
        # the stream is wider than what a block adds to it
        st["residual"] = normal(*shape, std=3.0) if case["residual"] else None
        st["post"] = normal(case["dim"], dtype=wt, std=0.1, mean=1.0) if case["post"] else None
        st["pre"] = normal(case["dim"], dtype=wt, std=0.1, mean=1.0) if case["pre"] else None
        if both:
            st["dh"] = normal(*shape)
            st["dy"] = normal(*shape) if case["pre"] else None
        return st
    H, Hk, D, E = case["heads"], case["qk_heads"], case["dim_qk"], case["dim_v"]
    N = case["packed"] or B
    st["cu_host"] = st["cu"] = None
    if case["packed"]:
        cu = torch.zeros(case["packed"] + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(_lengths(case)), 0)
        st["cu_host"], st["cu"] = cu, cu.cuda()
    # queries and keys of length one, as the rule takes them
    for name in ("q", "k"):
        x = normal(B, T, Hk, D, dtype=torch.float32)
        st[name] = (x / (x.square().sum(-1, keepdim=True) + _EPS).sqrt()).to(dt)
    st["v"] = normal(B, T, H, E)
    # strength of each write, and the forget gate: every head with its own memory, from a few
    # tokens to thousands
    gt = _TYPES[case["gate"]]
    st["beta"] = torch.sigmoid(normal(B, T, H, dtype=torch.float32)).to(gt)
    rate = uniform(H, low=1.0, high=16.0)
    step = torch.exp(uniform(H, low=math.log(1e-3), high=math.log(1e-1)))
    a = normal(B, T, H, dtype=torch.float32, std=0.5) + step + torch.log(-torch.expm1(-step))
    st["g"] = (-rate * torch.nn.functional.softplus(a)).to(gt)
    st["init"] = normal(N, H, D, E, dtype=torch.float32, std=0.1) if case["state"] else None
    if both:
        st["do"] = normal(B, T, H, E)
        st["dfin"] = normal(N, H, D, E, dtype=torch.float32, std=0.1) if case["state"] else None
    return st


# ---------------------------------------------------------------------------
# one pass

def run(state):
    if state["case"]["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _delta_own(state) if own else _delta_plain(state)


def _norm_own(st):
    import linear_attention_head_gb300 as la
    case = st["case"]
    kw = dict(gate=st["gate"], residual=st["residual"], post_weight=st["post"],
              pre_weight=st["pre"], activation=case["activation"], scale=case["scale"], eps=_EPS)
    h, y = la.block_norm_fwd(st["x"], **kw)
    if case["direction"] == "forward":
        return (h, y) if y is not None else h
    g = la.block_norm_bwd(st["x"], st["dh"], st["dy"], **kw)
    return tuple(t for t in (h, y) + tuple(g) if t is not None)


def _delta_own(st):
    import linear_attention_head_gb300 as la
    case = st["case"]
    kw = dict(initial_state=st["init"], cu_seqlens=st["cu"], cu_seqlens_host=st["cu_host"])
    a = (st["q"], st["k"], st["v"], st["g"], st["beta"])
    if case["direction"] == "forward":
        return la.gated_delta_fwd(*a, **kw)
    o, fin, saved = la.gated_delta_fwd(*a, keep=True, **kw)
    g = la.gated_delta_bwd(*a, st["do"], d_final_state=st["dfin"], saved=saved,
                           want_d_initial_state=case["state"], **kw)
    return (o, fin) + tuple(t for t in g if t is not None)


def _act(z, kind):
    """The gate's factor and its slope."""
    if kind == "none":
        return z, torch.ones_like(z)
    s = 1.0 / (1.0 + torch.exp(-z))
    if kind == "sigmoid":
        return s, s * (1.0 - s)
    return z * s, s * (1.0 + z * (1.0 - s))


def _norm_plain(st):
    case = st["case"]
    x, dt = st["x"].float(), st["x"].dtype
    c = case["scale"]
    n = x
    if case["post"]:
        rx = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        w = st["post"].float()
        n = x * rx * w
    m = n
    if case["gate"]:
        f, slope = _act(st["gate"].float(), case["activation"])
        m = n * f
    h = c * m
    if case["residual"]:
        h = h + st["residual"].float()
    out = [h.to(dt)]
    if case["pre"]:
        rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
        v = st["pre"].float()
        out.append((h * rh * v).to(dt))
    if case["direction"] == "forward":
        return tuple(out) if len(out) > 1 else out[0]
    lead = tuple(range(x.ndim - 1))
    dh = st["dh"].float()
    dpre = dpost = None
    if case["pre"]:
        dy = st["dy"].float()
        dpre = (dy * (h * rh)).sum(lead, dtype=torch.float64).to(st["pre"].dtype)
        u = dy * v
        dh = dh + rh * (u - h * (rh * rh) * (u * h).mean(-1, keepdim=True))
    dm = c * dh
    dgate = None
    if case["gate"]:
        dgate = (dm * n * slope).to(dt)
        dm = dm * f
    dx = dm
    if case["post"]:
        dpost = (dm * (x * rx)).sum(lead, dtype=torch.float64).to(st["post"].dtype)
        u = dm * w
        dx = rx * (u - x * (rx * rx) * (u * x).mean(-1, keepdim=True))
    dres = dh.to(dt) if case["residual"] else None
    grads = (dx.to(dt), dgate, dres, dpost, dpre)
    return tuple(out) + tuple(t for t in grads if t is not None)


_CHUNK = 64


def _padded(st, x, L):
    """[B, T, H, ...] -> [N, H, L, ...] fp32, zeros past the end of a sequence."""
    case = st["case"]
    if not case["packed"]:
        y = x.transpose(1, 2).float()
        pad = [0, 0] * (x.ndim - 3) + [0, L - x.shape[1]]
        return torch.nn.functional.pad(y, pad)
    y = x.new_zeros((case["packed"], x.shape[2], L) + x.shape[3:], dtype=torch.float32)
    at = 0
    for n, length in enumerate(_lengths(case)):
        y[n, :, :length] = x[0, at:at + length].transpose(0, 1).float()
        at += length
    return y


def _unpadded(st, y, dtype):
    """[N, H, L, ...] -> [B, T, H, ...]"""
    lens = _lengths(st["case"])
    if not st["case"]["packed"]:
        return y[:, :, :lens[0]].transpose(1, 2).to(dtype).contiguous()
    return torch.cat([y[n, :, :m].transpose(0, 1) for n, m in enumerate(lens)])[None].to(dtype)


def _delta_plain(st):
    """Chunks of 64 tokens.  With G the running sums of g in a chunk, S its entering state,
        A_ij = beta_i e^(G_i - G_j) k_i.k_j  (j < i),    T = (I + A)^-1,
        Z = T beta (V - e^G K S)      (each token's write, beta times what it got wrong)
        O = scale (e^G Q S + P Z),    P_ij = e^(G_i - G_j) q_i.k_j  (j <= i)
        S' = e^G_C S + sum_j e^(G_C - G_j) k_j z_j^T."""
    case = st["case"]
    H, D, E, C = case["heads"], case["dim_qk"], case["dim_v"], _CHUNK
    group = H // case["qk_heads"]
    scale = D ** -0.5
    L = -(-max(_lengths(case)) // C) * C
    nc = L // C
    q, k = (_padded(st, st[n], L).repeat_interleave(group, 1) for n in ("q", "k"))
    v, beta = _padded(st, st["v"], L), _padded(st, st["beta"], L)
    N = v.shape[0]
    cut = lambda x: x.unflatten(2, (nc, C))
    q, k, v, beta = cut(q), cut(k), cut(v), cut(beta)[..., None]
    G = cut(_padded(st, st["g"], L)).double().cumsum(-1)
    low = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    M = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -1e30)).float()
    eG, eC = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    gC = G[..., -1].exp().float()[..., None, None]
    kk = (k @ k.transpose(-1, -2)) * M
    A0 = kk.tril(-1)
    A = beta * A0
    inv = torch.eye(C, device="cuda").expand_as(A).clone()
    for i in range(1, C):
        inv[..., i, :i] = -(A[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    P = scale * (q @ k.transpose(-1, -2)) * M
    U, W = inv @ (beta * v), inv @ (beta * eG * k)
    S = st["init"] if case["state"] else torch.zeros((N, H, D, E), device="cuda")
    both = case["direction"] == "both"
    kC = k * eC
    outs, states, writes = [], [], []
    for c in range(nc):
        if both:
            states.append(S)
        Z = U[:, :, c] - W[:, :, c] @ S
        outs.append(scale * eG[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ Z)
        S = gC[:, :, c] * S + kC[:, :, c].transpose(-1, -2) @ Z
        writes.append(Z)
    dt = st["q"].dtype
    out = (_unpadded(st, torch.cat(outs, 2), dt), S)
    if not both:
        return out
    del U, W, outs
    do = cut(_padded(st, st["do"], L))
    K = st["dfin"] if case["state"] else torch.zeros_like(S)
    grads = {n: [None] * nc for n in ("q", "k", "v", "g", "beta")}
    tr = lambda x: x.transpose(-1, -2)
    for c in range(nc - 1, -1, -1):
        at = lambda x: x[:, :, c]
        S, Z, qc, kc, vc, dc = states[c], writes[c], at(q), at(k), at(v), at(do)
        dZ = tr(at(P)) @ dc + at(kC) @ K
        dR = tr(at(inv)) @ dZ
        dX = at(beta) * dR
        wrong = vc - at(eG) * (kc @ S) - at(A0) @ Z
        dP = scale * (dc @ tr(Z)) * at(M)
        dA = (-(dX @ tr(Z)) * at(M)).tril(-1)
        grads["q"][c] = scale * at(eG) * (dc @ tr(S)) + dP @ kc
        row = -at(eG) * (dX @ tr(S)) + dA @ kc
        col = tr(dP) @ qc + tr(dA) @ kc + at(eC) * (Z @ tr(K))
        grads["k"][c] = row + col
        grads["v"][c] = dX
        grads["beta"][c] = (dR * wrong).sum(-1)
        # each token's share in the running sums, and the state's that leaves the chunk
        each = (qc * grads["q"][c]).sum(-1) + (kc * (row - col)).sum(-1)
        end = (at(gC) * S + tr(at(kC)) @ Z).mul_(K).sum((-1, -2))[..., None]
        grads["g"][c] = each.flip(-1).cumsum(-1).flip(-1) + end
        K = at(gC) * K + tr(scale * at(eG) * qc) @ dc - tr(at(eG) * kc) @ dX
    g = {n: torch.cat(x, 2) for n, x in grads.items()}
    for n in ("q", "k"):
        g[n] = g[n].unflatten(1, (case["qk_heads"], group)).sum(2)
    # the gates' gradients come in the tokens' type, whatever the gates' own
    out += tuple(_unpadded(st, g[n], dt) for n in ("q", "k", "v", "g", "beta"))
    return out + ((K,) if case["state"] else ())


# ---------------------------------------------------------------------------
# work and exact results

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = _rows(case)
    both = case["direction"] == "both"
    if case["op"] == "norm":
        n = B * T * case["heads"] * case["dim"]
        given = 1 + case["gate"] + case["residual"]
        if both:    # inputs, the outputs' gradients; outputs, the inputs' gradients
            return {"bytes": e * n * (2 * given + 2 * (1 + case["pre"])), "flops": 30 * n}
        return {"bytes": e * n * (given + 1 + case["pre"]), "flops": 12 * n}
    f = 2 if case["gate"] == "bf16" else 4
    H, Hk, D, E = case["heads"], case["qk_heads"], case["dim_qk"], case["dim_v"]
    states = (case["packed"] or B) * H * D * E * 4
    qk, v, gates = 2 * B * T * Hk * D * e, B * T * H * E * e, 2 * B * T * H * f
    if both:    # q, k, v, do, gates, states in; o, gradients out
        return {"bytes": 2 * (qk + 2 * v) + gates + 2 * B * T * H * e + states * (4 if case["state"] else 1),
                "flops": 20 * B * T * H * D * E}
    return {"bytes": qk + 2 * v + gates + states * (2 if case["state"] else 1),
            "flops": 6 * B * T * H * D * E}


def exact(case, seed):
    st = prepare(case, seed)
    return _norm_exact(st) if case["op"] == "norm" else _delta_exact(st)


def _norm_exact(st):
    """By differentiating the definition, some rows at a time."""
    case = st["case"]
    dim, both = case["dim"], case["direction"] == "both"
    flat = {n: st[n].reshape(-1, dim) for n in ("x", "gate", "residual", "dh", "dy")
            if st.get(n) is not None}
    ws = [st[n].double().requires_grad_(both) if st[n] is not None else None
          for n in ("post", "pre")]
    rows = max(1, (1 << 24) // dim)
    pieces, dws = [], [0.0, 0.0]
    norm = lambda z: z / torch.sqrt(z.square().sum(-1, keepdim=True) / dim + _EPS)
    for at in range(0, flat["x"].shape[0], rows):
        part = {n: t[at:at + rows].double() for n, t in flat.items()}
        leaves = [part[n].requires_grad_(both) for n in ("x", "gate", "residual") if n in part]
        with torch.set_grad_enabled(both):
            h = part["x"]
            if ws[0] is not None:
                h = norm(h) * ws[0]
            if "gate" in part:
                s = torch.sigmoid(part["gate"])
                h = h * {"none": part["gate"], "sigmoid": s,
                         "silu": part["gate"] * s}[case["activation"]]
            h = h * case["scale"]
            if "residual" in part:
                h = h + part["residual"]
            ys = [h] + ([norm(h) * ws[1]] if ws[1] is not None else [])
            got = []
            if both:
                on = [w for w in ws if w is not None]
                dys = [part["dh"]] + ([part["dy"]] if ws[1] is not None else [])
                got = list(torch.autograd.grad(ys, leaves + on, dys))
        tail = got[len(leaves):]
        for i in (0, 1):
            if both and ws[i] is not None:
                dws[i] = dws[i] + tail.pop(0)
        pieces.append([y.detach() for y in ys] + got[:len(leaves)])
    out = [torch.cat(p).reshape(st["x"].shape) for p in zip(*pieces)]
    if both:
        out += [dws[i] for i in (0, 1) if ws[i] is not None]
    return tuple(out) if len(out) > 1 else out[0]


def _delta_exact(st):
    """The rule token by token over every sequence at once, and its chain rule back from
    states kept every 64 tokens."""
    case = st["case"]
    H, Hk, D, E = case["heads"], case["qk_heads"], case["dim_qk"], case["dim_v"]
    lens = _lengths(case)
    N, L = len(lens), max(lens)
    scale = 1.0 / math.sqrt(D)
    if L > 70000:
        return None

    def steps(x, fill=0.0):     # [L, N * H, ...]; past a sequence's end nothing is written
        x = x.double()
        if x.shape[2] != H:
            x = x.repeat_interleave(H // x.shape[2], 2)
        parts = list(x) if not case["packed"] else list(x[0].split(lens))
        y = torch.nn.utils.rnn.pad_sequence(parts, padding_value=fill)
        return y.flatten(1, 2)

    def back(y, heads=H):       # [L, N * H, ...] -> [B, T, heads, ...]
        y = y.unflatten(1, (N, H))
        if heads != H:
            y = y.unflatten(2, (heads, H // heads)).sum(3)
        if case["packed"]:
            return torch.cat([y[:m, n] for n, m in enumerate(lens)])[None]
        return y.transpose(0, 1)

    q, k, v = (steps(st[n]) for n in "qkv")
    a, beta = steps(st["g"]).exp(), steps(st["beta"])
    S = st["init"].double().flatten(0, 1) if case["state"] else \
        torch.zeros((N * H, D, E), dtype=torch.float64, device="cuda")
    both = case["direction"] == "both"
    o = torch.empty_like(v)
    keep = []

    def step(S, t):
        S = S * a[t][:, None, None]
        wrong = v[t] - (k[t][:, None] @ S)[:, 0]
        return S, wrong, torch.baddbmm(S, k[t][..., None], (beta[t][:, None] * wrong)[:, None])

    for t in range(L):
        if both and t % 64 == 0:
            keep.append(S)
        S = step(S, t)[2]
        o[t] = scale * (q[t][:, None] @ S)[:, 0]
    out = (back(o), S.unflatten(0, (N, H)))
    if not both:
        return out
    do = steps(st["do"])
    dS = st["dfin"].double().flatten(0, 1) if case["state"] else torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(a), torch.empty_like(a)
    for first in range((L - 1) // 64 * 64, -1, -64):
        S, run_ = keep.pop(), []
        for t in range(first, min(first + 64, L)):
            run_.append(step(S, t))
            S = run_[-1][2]
        for t in range(min(first + 64, L) - 1, first - 1, -1):
            decayed, wrong, S = run_.pop()
            dq[t] = scale * (S @ do[t][..., None])[..., 0]
            dS = torch.baddbmm(dS, q[t][..., None], do[t][:, None], alpha=scale)
            into = (k[t][:, None] @ dS)[:, 0]           # gradient of this token's write
            dbeta[t] = (into * wrong).sum(-1)
            dv[t] = beta[t][:, None] * into
            dk[t] = (dS @ (beta[t][:, None] * wrong)[..., None] -
                     decayed @ dv[t][..., None])[..., 0]
            dS = torch.baddbmm(dS, k[t][..., None], dv[t][:, None], alpha=-1.0)
            dg[t] = (dS * decayed).sum((-1, -2))
            dS = dS * a[t][:, None, None]
    out += (back(dq, Hk), back(dk, Hk), back(dv), back(dg), back(dbeta))
    return out + ((dS.unflatten(0, (N, H)),) if case["state"] else ())
