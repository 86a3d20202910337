"""The operators beside the attention without a GPU: the gradients' formulas against
differences, the refusals of the C entry points (before anything touches a device) and of the
Python layer."""
import ctypes

import pytest
import torch

import layer_reference as R
import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import _native as N
from linear_attention_head_gb300 import build as libbuild

FAKE = ctypes.c_void_p(0x1000)     # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return N.lib()


# ---- formulas ------------------------------------------------------------------

@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
def test_scan_gradients_against_differences(reverse, cu):
    gen = torch.Generator().manual_seed(1)
    B, T = (2, 9) if cu is None else (1, 9)
    n = B if cu is None else len(cu) - 1
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, g, do = r(B, T, 2, 3), -r(B, T, 2, 3).abs(), r(B, T, 2, 3)
    init, dfin = r(n, 2, 3), r(n, 2, 3)

    def loss(x, g, init):
        out = R.scan(x, g, init, reverse, cu)
        return float((out["o"] * do).sum() + (out["final"] * dfin).sum())

    out = R.scan(x, g, init, reverse, cu, do, dfin)
    h = 1e-6
    for i, name in enumerate(("dx", "dg", "dinit")):
        args = [x, g, init]
        want = torch.zeros_like(args[i])
        for k in range(want.numel()):
            d = torch.zeros_like(want)
            d.view(-1)[k] = h
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + d, args[i] - d
            want.view(-1)[k] = (loss(*up) - loss(*down)) / (2 * h)
        assert torch.allclose(out[name], want, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rotation_gradient_formula(interleaved):
    # dx = r (z - x r^2 mean(z x)), z = R^T(dy) w; dw = sum R^T(dy) x r
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, w, dy = r(1, 5, 2, 10).requires_grad_(), r(10).requires_grad_(), r(1, 5, 2, 10)
    freq, pos = [1.0, 0.3, 0.01], R.positions_of(1, 5, [0, 2, 5], [4, 100])
    y = R.norm_rope(x, w, 1e-3, True, freq, None, pos, interleaved)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    u = R.norm_rope(dy, None, 0.0, False, freq, None, -pos, interleaved)
    rr = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-3)
    z = u * w
    assert torch.allclose(dx, rr * (z - x * rr ** 2 * (z * x).mean(-1, keepdim=True)))
    assert torch.allclose(dw, (u * x * rr).sum((0, 1, 2)))


# ---- C entry points ------------------------------------------------------------------

I3 = ctypes.c_int64 * 3


def _scan_dims(B=2, T=20, H=3, D=8, n=0, gate=0):
    st = I3(T * H * D, H * D, D)
    return N.LaScanDims(B, T, H, D, n, gate, st, st, st, st, st, st)


def _scan_fwd(lib, d, dtype=0, x=FAKE, o=FAKE, cu=None, cu_host=None, ws=(FAKE, 1 << 40)):
    return lib.la_gated_scan_fwd(ctypes.byref(d) if d is not None else None, dtype, x, FAKE, None,
                                 0, cu, cu_host, o, None, None, *ws, None)


def _scan_bwd(lib, d, dtype=0, do=FAKE, dg=FAKE, ws=(FAKE, 1 << 40)):
    return lib.la_gated_scan_bwd(ctypes.byref(d), dtype, FAKE, FAKE, do, None, None, 0, None, None,
                                 None, FAKE, dg, None, *ws, None)


def _refused(status, text, kind=N.LA_ERR_INVALID_ARG):
    assert status == kind, (status, N.last_error())
    assert text in N.last_error(), N.last_error()


def _cu(vals):
    arr = (ctypes.c_int32 * len(vals))(*vals)
    return ctypes.cast(arr, ctypes.c_void_p)


def test_struct_layouts():
    assert ctypes.sizeof(N.LaScanDims) == 6 * 4 + 6 * 24
    assert N.LaScanDims.x_strides.offset == 24
    assert ctypes.sizeof(N.LaRopeDims) == 12 * 4 + 7 * 24 + 128
    assert N.LaRopeDims.q_strides.offset == 48 and N.LaRopeDims.pair_axis.offset == 216


def test_scan_refusals(lib):
    _refused(_scan_fwd(lib, None), "dims")
    _refused(_scan_fwd(lib, _scan_dims(), dtype=5), "dtype 5")
    _refused(_scan_fwd(lib, _scan_dims(gate=0), dtype=1), "gate_dtype")
    _refused(_scan_fwd(lib, _scan_dims(gate=7)), "gate_dtype")
    _refused(_scan_fwd(lib, _scan_dims(B=-1)), "negative batch")
    _refused(_scan_fwd(lib, _scan_dims(H=0)), "heads")
    _refused(_scan_fwd(lib, _scan_dims(D=257)), "dim", N.LA_ERR_UNSUPPORTED)
    _refused(_scan_fwd(lib, _scan_dims(), x=None), "x is NULL")
    _refused(_scan_fwd(lib, _scan_dims(), o=None), "o is NULL")
    d = _scan_dims()
    d.g_strides[1] = -8
    _refused(_scan_fwd(lib, d), "negative stride of g")
    d = _scan_dims()
    d.o_strides[0] = 0
    _refused(_scan_fwd(lib, d), "stride 0 of o")
    _refused(_scan_bwd(lib, _scan_dims(), do=None), "d_o is NULL")
    _refused(_scan_bwd(lib, _scan_dims(), dg=None), "dg is NULL")
    # packed sequences
    d = _scan_dims(B=1, n=3)
    _refused(_scan_fwd(lib, d, cu=FAKE, cu_host=_cu([0, 9, 5, 20])), "decreases")
    _refused(_scan_fwd(lib, d, cu=FAKE, cu_host=_cu([0, 5, 9, 19])), "seq_len")
    _refused(_scan_fwd(lib, d, cu=FAKE, cu_host=_cu([1, 5, 9, 20])), "expected 0")
    _refused(_scan_fwd(lib, d, cu_host=_cu([0, 5, 9, 20])), "without cu_seqlens")
    _refused(_scan_fwd(lib, _scan_dims(n=3), cu=FAKE, cu_host=_cu([0, 5, 9, 20])), "batch must")


def test_scan_workspace_is_checked(lib):
    d = _scan_dims(B=1, T=100000)
    ref = ctypes.byref(d)
    assert lib.la_gated_scan_states_size(ref) > 0
    assert lib.la_gated_scan_workspace_size(ref, 0, 2) >= lib.la_gated_scan_states_size(ref)
    need = lib.la_gated_scan_workspace_size(ref, 0, 2)
    _refused(_scan_bwd(lib, d, ws=(FAKE, need - 1)), "workspace")
    _refused(_scan_bwd(lib, d, ws=(None, 0)), "workspace")
    _refused(_scan_bwd(lib, d, ws=(ctypes.c_void_p(0x1010), need)), "aligned")
    assert lib.la_gated_scan_workspace_size(None, 0, 0) == 0
    assert lib.la_gated_scan_states_size(ctypes.byref(_scan_dims(D=0))) == 0


def test_scan_sizes_of_states_and_workspaces(lib):
    states = lambda d: lib.la_gated_scan_states_size(ctypes.byref(d))
    ws = lambda d, mode: lib.la_gated_scan_workspace_size(ctypes.byref(d), 0, mode)
    row = 3 * 8 * 4
    # a tile's tokens or fewer: no states; one more, two of them a row (few rows: no threads
    # of their own); many rows of some tokens: a state for every 8
    assert states(_scan_dims(B=2, T=128, H=3, D=8)) == 0
    assert states(_scan_dims(B=2, T=129, H=3, D=8)) == 2 * 2 * row
    assert states(_scan_dims(B=5000, T=9, H=3, D=8)) == 5000 * 2 * row
    assert states(_scan_dims(B=5000, T=8, H=3, D=8)) == 0
    # packed: enough for any lengths, whichever kernels they get
    for T in (5, 100, 1000, 5000):
        assert states(_scan_dims(B=1, T=T, H=3, D=8, n=6)) >= (T // 128 + 6) * row
    assert states(_scan_dims(B=1, T=700, H=3, D=8, n=6)) >= (700 // 8 + 6) * row
    # in place: a copy of every sequence's initial state besides
    d = _scan_dims(B=1, T=700, H=3, D=8, n=6)
    assert ws(d, 3) >= ws(d, 0) + 6 * row
    assert ws(d, 2) >= ws(d, 1) + states(d)
    assert ws(_scan_dims(B=4, T=128), 0) == 0


def test_empty_scans_enqueue_nothing(lib):
    assert _scan_fwd(lib, _scan_dims(B=0), x=None, o=None) == N.LA_OK
    assert _scan_fwd(lib, _scan_dims(B=1, T=0, n=0), x=None, o=None, cu=FAKE,
                     cu_host=_cu([0])) == N.LA_OK


def _rope_dims(B=2, T=20, Hq=4, Hk=2, D=16, R_=8, **kw):
    d = N.LaRopeDims()
    d.batch, d.seq_len, d.q_heads, d.k_heads, d.dim, d.rotary_dim = B, T, Hq, Hk, D, R_
    d.num_axes, d.normalize, d.position_bytes = 1, 1, 4
    for name in ("q_strides", "qo_strides", "dq_strides"):
        setattr(d, name, I3(T * Hq * D, Hq * D, D))
    for name in ("k_strides", "ko_strides", "dk_strides"):
        setattr(d, name, I3(T * Hk * D, Hk * D, D))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _rope_fwd(lib, d, dtype=0, q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, freq=FAKE, pos=None,
              off=None, cu=None, cu_host=None, qo=ctypes.c_void_p(0x2000),
              ko=ctypes.c_void_p(0x3000)):
    return lib.la_qk_norm_rope_fwd(ctypes.byref(d) if d is not None else None, dtype, q, k, qw, kw,
                                   eps, freq, pos, off, cu, cu_host, qo, ko, None)


def test_rope_refusals(lib):
    _refused(_rope_fwd(lib, None), "dims")
    _refused(_rope_fwd(lib, _rope_dims(), dtype=3), "dtype 3")
    _refused(_rope_fwd(lib, _rope_dims(weight_dtype=9)), "weight_dtype 9")
    _refused(_rope_fwd(lib, _rope_dims(Hq=0, Hk=0)), "heads")
    _refused(_rope_fwd(lib, _rope_dims(D=300)), "dim", N.LA_ERR_UNSUPPORTED)
    _refused(_rope_fwd(lib, _rope_dims(R_=7)), "rotary_dim")
    _refused(_rope_fwd(lib, _rope_dims(R_=18)), "rotary_dim")
    _refused(_rope_fwd(lib, _rope_dims(num_axes=5)), "num_axes")
    _refused(_rope_fwd(lib, _rope_dims(num_axes=2)), "needs positions")
    d = _rope_dims()
    d.pair_axis[3] = 1
    _refused(_rope_fwd(lib, d), "pair_axis[3]")
    _refused(_rope_fwd(lib, _rope_dims(), freq=None), "inv_freq")
    _refused(_rope_fwd(lib, _rope_dims(), eps=-1.0), "eps")
    _refused(_rope_fwd(lib, _rope_dims(), eps=float("nan")), "eps")
    _refused(_rope_fwd(lib, _rope_dims(normalize=0)), "without normalize")
    _refused(_rope_fwd(lib, _rope_dims(), q=None), "q is NULL")
    _refused(_rope_fwd(lib, _rope_dims(), ko=None), "ko is NULL")
    _refused(_rope_fwd(lib, _rope_dims(), pos=FAKE, off=FAKE), "position_offset")
    _refused(_rope_fwd(lib, _rope_dims(position_bytes=2), pos=FAKE), "position_bytes")
    _refused(_rope_fwd(lib, _rope_dims(position_strides=I3(0, -1, 1)), pos=FAKE),
             "negative stride of positions")
    _refused(_rope_fwd(lib, _rope_dims(qo_strides=I3(0, 64, 16))), "stride 0 of qo")
    # in place only with the same strides
    _refused(_rope_fwd(lib, _rope_dims(qo_strides=I3(9999, 64, 16)), qo=FAKE), "in place")
    d = _rope_dims(B=1, num_seqs=2)
    _refused(_rope_fwd(lib, d, cu=FAKE, cu_host=_cu([0, 25, 20])), "decreases")
    b = lambda ws, d_=None, dqw=FAKE, dq=FAKE: lib.la_qk_norm_rope_bwd(
        ctypes.byref(d_ if d_ is not None else _rope_dims()), 0, FAKE, FAKE, FAKE, FAKE, FAKE,
        FAKE, 1e-6, FAKE, None, None, None, None, dq, FAKE, dqw, None, *ws, None)
    need = lib.la_qk_norm_rope_workspace_size(ctypes.byref(_rope_dims()), 0)
    assert need > 0
    _refused(b((FAKE, need - 1)), "workspace")
    _refused(b((None, 0)), "workspace")
    _refused(b((FAKE, need), dq=None), "dq is NULL")
    assert lib.la_qk_norm_rope_workspace_size(ctypes.byref(_rope_dims(normalize=0)), 0) == 0


def test_empty_norm_rotation_enqueues_nothing(lib):
    assert _rope_fwd(lib, _rope_dims(T=0), q=None, k=None, qo=None, ko=None) == N.LA_OK


# ---- Python layer ------------------------------------------------------------------

def test_rope_plan():
    f = la.rope_inv_freq(8, 100.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([100.0 ** (-j / 4) for j in range(4)],
                                          dtype=torch.float64))
    assert la.Rope(f, sections=(1, 2, 1)).axes == (0, 1, 1, 2)
    assert la.Rope(f, axes=(0, 1, 0, 1)).num_axes == 2
    assert la.Rope(f).num_axes == 1 and la.Rope(f).rotary_dim == 8
    for bad in (dict(sections=(1, 2)), dict(axes=(0, 1)), dict(axes=(0, 0, 0, 4)),
                dict(axes=(0, 0, 0, 1), sections=(3, 1)), dict(sections=(1, 1, 1, 1, 0))):
        with pytest.raises(ValueError):
            la.Rope(f, **bad)
    with pytest.raises(ValueError):
        la.Rope(torch.zeros(129))


def test_python_refusals_on_host_tensors():
    x = torch.zeros(1, 4, 2, 8)
    rope = la.Rope(la.rope_inv_freq(8, device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        la.gated_scan_fwd(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        la.qk_norm_rope_fwd(x, x, rope=rope)
    with pytest.raises(ValueError, match="rope"):
        la.rotary_fwd(x, x)
    with pytest.raises(ValueError, match="norm, rope or both"):
        la.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="cu_seqlens"):
        la.gated_scan(x[0], x[0])
    with pytest.raises(ValueError, match=r"\[B, T, H, D\]"):
        la.gated_scan_fwd(x[0], x[0])
    with pytest.raises(ValueError, match="positions need rope"):
        la.recurrent(x, x, x, positions=torch.zeros(4))
