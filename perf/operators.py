"""Cases of the operators that stand beside the linear-attention kernels: the
per-head norms of queries and keys with the position rotation, the rotation
alone with several position axes, and the gated linear recurrence.

`run` computes a case in its plain form (elementary torch operations in fp32,
rounded once at the end) or, with `own` set, by the calls that a user makes of
this framework.  `exact` gives the same outputs in fp64 from the definitions.
"""
import math

import torch

own = False

# bytes that a drawn case's pass moves at most
_MOST_BYTES = 1 << 30


# ---------------------------------------------------------------------------
# cases

def _norm_rope(name, **kw):
    c = {"op": "norm_rope", "direction": "forward", "batch": 1, "tokens": 1, "q_heads": 32,
         "k_heads": 8, "dim": 128, "rotary": 128, "axes": 1, "interleaved": False, "base": 10000.0,
         "dtype": "bf16", "packed": 0, "low": 64, "high": 8192, "normalize": True, "far": 0}
    c.update(kw)
    c["name"] = name
    return c


def _scan(name, **kw):
    c = {"op": "scan", "direction": "forward", "batch": 1, "tokens": 1, "heads": 32, "dim": 128,
         "dtype": "bf16", "gate": "bf16", "packed": 0, "low": 64, "high": 8192, "reverse": False,
         "state": True}
    c.update(kw)
    c["name"] = name
    return c


def listed():
    return [
        # one new token of each of 32 running sequences, 32 query and 8 key heads, each row
        # at its own far position: latency
        _norm_rope("norm_rope_decode_b32", batch=32, far=131072),
        # 16 prompts of 64 to 8192 tokens packed in one row: positions count inside each
        _norm_rope("norm_rope_prompt_packed16", packed=16),
        # a training step's forward and backward, the benchmark's batch and heads
        _norm_rope("norm_rope_train_b4_n8192", batch=4, tokens=8192, direction="both"),
        # fp32, wide heads, a rotation of part of the channels in neighbouring pairs, odd length
        _norm_rope("norm_rope_train_fp32_n2047_d192", batch=2, tokens=2047, q_heads=12,
                   k_heads=12, dim=192, rotary=96, interleaved=True, dtype="fp32",
                   direction="both"),
        # a clip of 21 frames of 30 x 52 patches: time, height, width
        _norm_rope("rotary_video_n32760", tokens=32760, q_heads=16, k_heads=16, axes=3,
                   normalize=False),
        # a batch of images of 32 x 32 patches in training: height, width
        _norm_rope("rotary_image_train_b8_n1024_d64", batch=8, tokens=1024, q_heads=12,
                   k_heads=12, dim=64, rotary=64, axes=2, normalize=False, direction="both"),
        # one new token a sequence after images and text: three axes a row
        _norm_rope("rotary_decode_b64", batch=64, axes=3, normalize=False, far=32768),
        # one new token of 64 sequences with the carried state in and out
        _scan("scan_decode_b64", batch=64),
        # 16 packed prompts with initial states, the gate in fp32
        _scan("scan_prompt_packed16", packed=16, heads=16, gate="fp32"),
        # one long sequence with few heads: the scan has to be split over the tokens
        _scan("scan_long_n262144_h8", tokens=262144, heads=8),
        # a training step's forward and backward, the gated benchmark's shape
        _scan("scan_train_b4_n8192", batch=4, tokens=8192, direction="both"),
        # fp32, few odd channels, odd length, from last to first
        _scan("scan_train_fp32_n1025_d33", batch=3, tokens=1025, heads=5, dim=33, dtype="fp32",
              gate="fp32", reverse=True, direction="both"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    dtype = "fp32" if rng.random() < 0.3 else "bf16"
    e = 4 if dtype == "fp32" else 2
    direction = rng.choice(["forward", "both"])
    kind = rng.choice(["norm_rope", "rotary", "scan"])
    shape = rng.choice(["step", "dense", "dense", "packed"])
    if kind == "scan":
        heads, dim = _log_int(rng, 1, 40), rng.choice([rng.randint(1, 256), 64, 128, 128, 192, 256])
        gate = "fp32" if dtype == "fp32" or rng.random() < 0.4 else "bf16"
        most = max(2, _MOST_BYTES // (heads * dim * (4 * e + (8 if gate == "fp32" else 4))))
        c = dict(heads=heads, dim=dim, dtype=dtype, gate=gate, direction=direction,
                 reverse=rng.random() < 0.3, state=rng.random() < 0.7)
    else:
        q_heads = _log_int(rng, 1, 40)
        k_heads = rng.choice([h for h in range(1, q_heads + 1) if q_heads % h == 0])
        dim = rng.choice([2 * rng.randint(1, 128), 64, 96, 128, 128, 192, 256])
        rotary = rng.choice([dim, dim, 2 * rng.randint(1, dim // 2)])
        axes = 1 if kind == "norm_rope" or shape == "packed" else rng.choice([1, 2, 3])
        axes = min(axes, rotary // 2)
        most = max(2, _MOST_BYTES // ((q_heads + k_heads) * dim * 4 * e))
        c = dict(q_heads=q_heads, k_heads=k_heads, dim=dim, rotary=rotary, axes=axes,
                 interleaved=rng.random() < 0.3, base=rng.choice([1e4, 5e5]), dtype=dtype,
                 direction=direction, normalize=kind == "norm_rope",
                 far=rng.choice([0, 1 << 17, 1 << 24]) if shape != "packed" else 0)
    if shape == "step":
        c.update(batch=min(_log_int(rng, 1, 512), most), tokens=1)
    elif shape == "packed":
        n = _log_int(rng, 1, 64)
        high = max(2, min(8192, most // n))
        c.update(packed=n, low=rng.randint(1, max(1, high // 4)), high=high)
    else:
        b = min(_log_int(rng, 1, 16), max(1, most // 2))
        tokens = _log_int(rng, 2, max(2, min(262144 if kind == "scan" else 65536, most // b)))
        c.update(batch=b, tokens=tokens)
    case = (_scan if kind == "scan" else _norm_rope)("", **c)
    del case["name"]
    return case


def _lengths(case):
    """The packed sequences' lengths: fixed by the case, spread over [low, high]."""
    gen = torch.Generator().manual_seed(1000 * case["packed"] + case["low"] + case["high"])
    return torch.randint(case["low"], case["high"] + 1, (case["packed"],), generator=gen).tolist()


def _rows(case):
    """(batch rows, tokens a row)"""
    return (1, sum(_lengths(case))) if case["packed"] else (case["batch"], case["tokens"])


# ---------------------------------------------------------------------------
# inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _sections(pairs, axes):
    """Frequency pairs of each axis: the first axis takes the smaller part, the rest share."""
    if axes == 1:
        return (pairs,)
    if axes == 2:
        return (pairs // 2, pairs - pairs // 2)
    first = max(1, pairs // 4)
    second = (pairs - first) // 2
    return (first, second, pairs - first - second)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    B, T = _rows(case)

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=gen, device="cuda")
        return x.mul_(std).add_(mean).to(dtype)

    st = {"case": case}
    if case["packed"]:
        cu = torch.zeros(case["packed"] + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(_lengths(case)), 0)
        st["cu_host"], st["cu"] = cu, cu.cuda()
    else:
        st["cu_host"] = st["cu"] = None
    both = case["direction"] == "both"
    if case["op"] == "scan":
        H, D = case["heads"], case["dim"]
        N = case["packed"] or B
        st["x"] = normal(B, T, H, D)
        # log of a forget gate: each channel with its own memory, a few to thousands of tokens
        bias = torch.rand((H, D), generator=gen, device="cuda").mul_(7.0).add_(1.0)
        z = torch.randn((B, T, H, D), generator=gen, device="cuda").add_(bias)
        st["g"] = torch.nn.functional.logsigmoid(z).to(_TYPES[case["gate"]])
        del z
        st["init"] = normal(N, H, D, dtype=torch.float32) if case["state"] else None
        if both:
            st["do"] = normal(B, T, H, D)
            st["dfin"] = normal(N, H, D, dtype=torch.float32) if case["state"] else None
        return st
    Hq, Hk, D, R = case["q_heads"], case["k_heads"], case["dim"], case["rotary"]
    st["q"], st["k"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
    st["qw"] = st["kw"] = None
    if case["normalize"]:
        st["qw"], st["kw"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1, mean=1.0)
    if both:
        st["dq_out"], st["dk_out"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
    pairs = R // 2
    st["inv_freq"] = case["base"] ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    st["inv_freq"] = st["inv_freq"].cuda()
    st["sections"] = _sections(pairs, case["axes"])
    axis = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
    st["axis"] = torch.tensor(axis, device="cuda")
    st["positions"] = None
    if not case["packed"] and (case["axes"] > 1 or case["far"]):
        if case["far"]:     # each row at a place of its own, up to `far`
            start = torch.randint(0, case["far"], (case["axes"], B, 1), generator=gen,
                                  device="cuda")
            st["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        else:               # a grid walked row by row, time the slowest
            w = max(1, int(math.sqrt(T / case["axes"])))
            t = torch.arange(T, device="cuda")
            grid = [t % w, t // w % w, t // (w * w)] if case["axes"] == 3 else [t % w, t // w]
            grid = torch.stack(grid[::-1]) if case["axes"] > 1 else t[None]
            st["positions"] = grid[:, None, :].expand(-1, B, -1).contiguous().to(torch.int32)
    if own:
        import linear_attention_head_gb300 as la
        # the plan of the rotation, which a model keeps
        st["rope"] = la.Rope(st["inv_freq"], sections=st["sections"],
                             interleaved=case["interleaved"])
    return st


# ---------------------------------------------------------------------------
# one pass

_EPS = 1e-6


def run(state):
    case = state["case"]
    if case["op"] == "scan":
        return _scan_own(state) if own else _scan_plain(state)
    return _norm_rope_own(state) if own else _norm_rope_plain(state)


def _norm_rope_own(st):
    import linear_attention_head_gb300 as la
    case = st["case"]
    kw = dict(rope=st["rope"], positions=st["positions"], cu_seqlens=st["cu"],
              cu_seqlens_host=st["cu_host"])
    if case["normalize"]:
        kw.update(q_weight=st["qw"], k_weight=st["kw"], eps=_EPS)
        q, k = la.qk_norm_rope_fwd(st["q"], st["k"], **kw)
        if case["direction"] == "forward":
            return q, k
        return (q, k) + tuple(la.qk_norm_rope_bwd(st["q"], st["k"], st["dq_out"], st["dk_out"],
                                                  **kw))
    q, k = la.rotary_fwd(st["q"], st["k"], **kw)
    if case["direction"] == "forward":
        return q, k
    return (q, k) + tuple(la.rotary_bwd(st["dq_out"], st["dk_out"], **kw))


def _scan_own(st):
    import linear_attention_head_gb300 as la
    case = st["case"]
    kw = dict(reverse=case["reverse"], cu_seqlens=st["cu"], cu_seqlens_host=st["cu_host"])
    if case["direction"] == "forward":
        return la.gated_scan_fwd(st["x"], st["g"], st["init"], **kw)
    o, fin, states = la.gated_scan_fwd(st["x"], st["g"], st["init"], keep_states=True, **kw)
    return (o, fin) + tuple(la.gated_scan_bwd(st["x"], st["g"], st["do"], st["init"], st["dfin"],
                                              states=states, **kw))


def _turn(st):
    """cos and sin [B or 1, T, 1, pairs]: angles in fp64 (far positions), rounded to fp32."""
    case = st["case"]
    B, T = _rows(case)
    if case["packed"]:
        cu = st["cu"].long()
        t = torch.arange(T, device="cuda")
        seq = torch.searchsorted(cu, t, right=True) - 1
        pos = (t - cu[seq])[None, None]
    elif st["positions"] is None:
        pos = torch.arange(T, device="cuda")[None, None]
    else:
        pos = st["positions"]
    angle = pos[st["axis"]].permute(1, 2, 0).double() * st["inv_freq"]
    return angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _pairs(x, case):
    """First and second channels of the pairs, and the channels that are not rotated."""
    R = case["rotary"]
    if case["interleaved"]:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _join(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)
    return torch.cat((a, b, rest), -1)


def _norm_rope_plain(st):
    case = st["case"]
    cos, sin = _turn(st)
    both = case["direction"] == "both"
    ys, dxs, dws = [], [], []
    for x_in, w_in, dy_name in ((st["q"], st["qw"], "dq_out"), (st["k"], st["kw"], "dk_out")):
        x = x_in.float()
        n = x
        if case["normalize"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
            n = x * r * w_in.float()
        a, b, rest = _pairs(n, case)
        ys.append(_join(a * cos - b * sin, a * sin + b * cos, rest, case).to(x_in.dtype))
        if not both:
            continue
        a, b, rest = _pairs(st[dy_name].float(), case)
        u = _join(a * cos + b * sin, b * cos - a * sin, rest, case)
        if case["normalize"]:
            dws.append((u * (x * r)).sum((0, 1, 2), dtype=torch.float64).to(w_in.dtype))
            z = u * w_in.float()
            u = r * (z - x * (r * r) * (z * x).mean(-1, keepdim=True))
        dxs.append(u.to(x_in.dtype))
    return tuple(ys + dxs + dws)


def _edges(st):
    """Masks [B, T] of each sequence's first and last token in processing order, and the
    number of the sequence [B, T]."""
    case = st["case"]
    B, T = _rows(case)
    t = torch.arange(T, device="cuda")
    if case["packed"]:
        cu = st["cu"].long()
        seq = (torch.searchsorted(cu, t, right=True) - 1)[None]
        low, high = (t == cu[seq[0]])[None], (t == cu[seq[0] + 1] - 1)[None]
    else:
        seq = torch.arange(B, device="cuda")[:, None].expand(B, T)
        low, high = (t == 0)[None].expand(B, T), (t == T - 1)[None].expand(B, T)
    return (high, low, seq) if case["reverse"] else (low, high, seq)


def _linear_scan(a, b, length, backward):
    """s_t = a_t s_{t-1} + b_t along dim 1 (from the last token with backward), by doubling:
    after step d every s_t covers the 2 d tokens that end at t.  length: the longest run."""
    d = 1
    while d < length:
        if backward:
            s = b[:, :-d] + a[:, :-d] * b[:, d:]
            p = a[:, :-d] * a[:, d:]
            b, a = torch.cat((s, b[:, -d:]), 1), torch.cat((p, a[:, -d:]), 1)
        else:
            s = b[:, d:] + a[:, d:] * b[:, :-d]
            p = a[:, d:] * a[:, :-d]
            b, a = torch.cat((b[:, :d], s), 1), torch.cat((a[:, :d], p), 1)
        d *= 2
    return b


def _scan_plain(st):
    case = st["case"]
    dt = st["x"].dtype
    first, last, seq = _edges(st)
    length = max(_lengths(case)) if case["packed"] else case["tokens"]
    # the decays in fp64: an error of theirs that keeps its sign adds up over thousands of tokens
    a = st["g"].double().exp().float()
    cut = a.masked_fill(first[..., None, None], 0.0)
    x = st["x"].float()
    if st["init"] is not None:
        x = x + torch.where(first[..., None, None], a * st["init"][seq], 0.0)
    s = _linear_scan(cut, x, length, case["reverse"])
    fin = s[last]
    out = (s.to(dt), fin)
    if case["direction"] == "forward":
        return out
    del x, cut
    # K_t = a_t (do_t + K_{t+1}), entering with d_final after the last token
    do = st["do"].float()
    if st["dfin"] is not None:
        do = do + torch.where(last[..., None, None], st["dfin"][seq], 0.0)
    K = _linear_scan(a.masked_fill(last[..., None, None], 0.0), a * do, length,
                     not case["reverse"])
    step = -1 if case["reverse"] else 1
    after = torch.roll(K, -step, 1).masked_fill_(last[..., None, None], 0.0)
    dx = (do + after).to(dt)
    del do, after
    before = torch.roll(s, step, 1)
    start = st["init"][seq] if st["init"] is not None else torch.zeros((), device="cuda")
    before = torch.where(first[..., None, None], start, before)
    dg = (K * before).to(st["g"].dtype)
    return out + (dx, dg, K[first])


# ---------------------------------------------------------------------------
# work and exact results

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = _rows(case)
    both = case["direction"] == "both"
    if case["op"] == "scan":
        f = 2 if case["gate"] == "bf16" else 4
        n = B * T * case["heads"] * case["dim"]
        states = (case["packed"] or B) * case["heads"] * case["dim"] * 4
        given = 1 if case["state"] else 0
        if both:    # x, g, do and the states in; o, dx, dg and the states' gradients out
            return {"bytes": n * (4 * e + 2 * f) + states * (2 + 2 * given), "flops": 8 * n}
        return {"bytes": n * (2 * e + f) + states * (1 + given), "flops": 3 * n}
    n = B * T * (case["q_heads"] + case["k_heads"]) * case["dim"]
    pos = 4 * case["axes"] * B * T if not case["packed"] and (case["axes"] > 1 or case["far"]) \
        else 0
    if not both:
        return {"bytes": 2 * e * n + pos, "flops": (7 if case["normalize"] else 3) * n}
    # x and dy in, y and dx out
    return {"bytes": 4 * e * n + pos, "flops": (20 if case["normalize"] else 6) * n}


def exact(case, seed):
    st = prepare(case, seed)
    return _scan_exact(st) if case["op"] == "scan" else _norm_rope_exact(st)


def _norm_rope_exact(st):
    """The rotation as a product of complex numbers, the gradients by differentiating it."""
    case = st["case"]
    B, T = _rows(case)
    R, both = case["rotary"], case["direction"] == "both"
    if case["packed"]:
        pos = torch.cat([torch.arange(n, device="cuda") for n in _lengths(case)])
        pos = pos.expand(1, 1, T)
    elif st["positions"] is None:
        pos = torch.arange(T, device="cuda").expand(1, 1, T)
    else:
        pos = st["positions"]
    angle = torch.stack([pos[a] for a in st["axis"].tolist()], -1).double() * st["inv_freq"]
    turn = torch.polar(torch.ones_like(angle), angle)
    ys, dxs, dws = [], [], []
    for x_in, w_in, dy_name in ((st["q"], st["qw"], "dq_out"), (st["k"], st["kw"], "dk_out")):
        outs, grads, dw = [], [], 0.0
        heads = max(1, (1 << 25) // max(1, B * T * case["dim"]))    # a few heads at a time
        for h in range(0, x_in.shape[2], heads):
            x = x_in[:, :, h:h + heads].double().requires_grad_(both)
            w = w_in.double().requires_grad_(both) if w_in is not None else None
            with torch.set_grad_enabled(both):
                n = x
                if case["normalize"]:
                    n = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + _EPS) * w
                head = n[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"]
                                            else (2, R // 2))
                if not case["interleaved"]:
                    head = head.transpose(-1, -2)
                z = torch.complex(head[..., 0], head[..., 1]) * turn[:, :, None]
                z = torch.view_as_real(z)
                if not case["interleaved"]:
                    z = z.transpose(-1, -2)
                y = torch.cat((z.flatten(-2), n[..., R:]), -1)
                if both:
                    dy = st[dy_name][:, :, h:h + heads].double()
                    got = torch.autograd.grad(y, (x, w) if w is not None else (x,), dy)
                    grads.append(got[0])
                    dw = dw + got[1] if w is not None else None
            outs.append(y.detach())
        ys.append(torch.cat(outs, 2))
        if both:
            dxs.append(torch.cat(grads, 2))
            if w_in is not None:
                dws.append(dw)
    return tuple(ys + dxs + dws)


def _scan_exact(st):
    """The recurrence token by token over every sequence at once, and its chain rule back."""
    case = st["case"]
    B, T = _rows(case)
    H, D, both = case["heads"], case["dim"], case["direction"] == "both"
    lens = _lengths(case) if case["packed"] else [T] * B
    N, L = len(lens), max(lens)
    if L > 300000:
        return None
    begin = [0]
    for n in lens[:-1]:
        begin.append(begin[-1] + n)
    # where the j-th processed token of sequence n lies in the row of all tokens
    j = torch.arange(L, device="cuda")[:, None]
    n_len = torch.tensor(lens, device="cuda")
    place = torch.tensor(begin, device="cuda") + (n_len - 1 - j if case["reverse"] else j)
    inside = j < n_len
    ragged = not bool(inside.all())

    def by_step(x):     # [L, N, H * D], zero past the end of a sequence
        y = x.reshape(B * T, H * D)[place.clamp(0, B * T - 1)].double()
        return y.masked_fill_(~inside[..., None], 0.0) if ragged else y

    def back(y, like):
        z = torch.empty((B * T, H * D), dtype=torch.float64, device="cuda")
        z[place[inside]] = y[inside]
        return z.reshape(like.shape)

    a = by_step(st["g"]).exp_()     # exp(0) = 1 past the end: the state stays
    s = by_step(st["x"])
    start = st["init"].reshape(N, H * D).double() if st["init"] is not None else \
        torch.zeros((N, H * D), dtype=torch.float64, device="cuda")
    rows, decay = s.unbind(0), a.unbind(0)
    before = start
    for row, d in zip(rows, decay):
        before = row.addcmul_(d, before)
    out = (back(s, st["x"]), before.reshape(N, H, D).clone())
    if not both:
        return out
    G = by_step(st["do"])
    K = st["dfin"].reshape(N, H * D).double() if st["dfin"] is not None else \
        torch.zeros((N, H * D), dtype=torch.float64, device="cuda")
    dg = torch.empty_like(G)
    for t in range(L - 1, -1, -1):
        K = G[t].add_(K) * decay[t]
        dg[t] = K * (rows[t - 1] if t else start)
    return out + (back(G, st["x"]), back(dg, st["x"]), K.reshape(N, H, D))
