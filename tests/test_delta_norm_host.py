"""The gated delta rule and the norms around a block without a GPU: sizes of workspaces, refusals
of the C entry points (before anything touches a device) and of the Python layer."""
import ctypes

import pytest
import torch

import linear_attention_head_gb300 as la
from linear_attention_head_gb300 import _native as N
from linear_attention_head_gb300 import build as libbuild

FAKE = ctypes.c_void_p(0x1000)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1002)
I3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return N.lib()


def _refused(status, text, kind=N.LA_ERR_INVALID_ARG):
    assert status == kind, (status, N.last_error())
    assert text in N.last_error(), N.last_error()


def _cu(vals):
    arr = (ctypes.c_int32 * len(vals))(*vals)
    return ctypes.cast(arr, ctypes.c_void_p)


# ---- gated delta rule ----------------------------------------------------------------

def _dims(B=2, T=40, H=4, HK=2, D=64, E=64, n=0, gate=1):
    qk, v, g = I3(T * HK * D, HK * D, D), I3(T * H * E, H * E, E), I3(T * H, H, 1)
    return N.LaDeltaDims(B, T, H, HK, D, E, n, gate, qk, qk, v, g, g, v, v, qk, qk, v)


def _fwd(lib, d, dtype=0, q=FAKE, beta=FAKE, scale=1.0, cu=None, cu_host=None, o=FAKE, saved=None,
         ws=(FAKE, 1 << 40)):
    return lib.la_gated_delta_fwd(ctypes.byref(d) if d is not None else None, dtype, q, FAKE, FAKE,
                                  FAKE, beta, scale, None, cu, cu_host, o, None, saved, *ws, None)


def _bwd(lib, d, dtype=0, do=FAKE, dq=FAKE, dbeta=FAKE, saved=None, ws=(FAKE, 1 << 40)):
    return lib.la_gated_delta_bwd(ctypes.byref(d), dtype, FAKE, FAKE, FAKE, FAKE, FAKE, do, 1.0,
                                  None, None, None, None, saved, dq, FAKE, FAKE, FAKE, dbeta, None,
                                  *ws, None)


def test_struct_layouts():
    assert ctypes.sizeof(N.LaDeltaDims) == 8 * 4 + 10 * 24
    assert N.LaDeltaDims.q_strides.offset == 32
    assert ctypes.sizeof(N.LaBlockNormDims) == 6 * 4 + 10 * 24
    assert N.LaBlockNormDims.x_strides.offset == 24


def test_delta_refusals(lib):
    _refused(_fwd(lib, None), "dims")
    _refused(_fwd(lib, _dims(), dtype=9), "dtype 9")
    _refused(_fwd(lib, _dims(gate=0), dtype=1), "gate_dtype")
    _refused(_fwd(lib, _dims(H=0)), "heads")
    _refused(_fwd(lib, _dims(HK=3)), "qk_heads")
    _refused(_fwd(lib, _dims(HK=8)), "qk_heads")
    _refused(_fwd(lib, _dims(D=257)), "dim = 257", N.LA_ERR_UNSUPPORTED)
    _refused(_fwd(lib, _dims(E=257)), "dim_v = 257", N.LA_ERR_UNSUPPORTED)
    _refused(_fwd(lib, _dims(B=-1)), "negative")
    _refused(_fwd(lib, _dims(), q=None), "q is NULL")
    _refused(_fwd(lib, _dims(), beta=None), "beta is NULL")
    _refused(_fwd(lib, _dims(), o=None), "o is NULL")
    _refused(_fwd(lib, _dims(), scale=float("inf")), "scale")
    _refused(_fwd(lib, _dims(), cu_host=_cu([0, 40])), "without cu_seqlens")
    _refused(_fwd(lib, _dims(n=1), cu=FAKE, cu_host=_cu([0, 40])), "batch must be 1")
    one = _dims(B=1, n=2)
    _refused(_fwd(lib, one, cu=FAKE, cu_host=_cu([0, 50, 40])), "decreases")
    _refused(_fwd(lib, one, cu=FAKE, cu_host=_cu([0, 10, 30])), "seq_len")
    _refused(_fwd(lib, _dims(), ws=(None, 0)), "workspace")
    _refused(_fwd(lib, _dims(), ws=(ODD, 1 << 40)), "aligned")
    _refused(_fwd(lib, _dims(), saved=ODD), "saved is not")
    # what the forward keeps is laid out for aligned rows
    _refused(_fwd(lib, _dims(), q=ODD, saved=FAKE), "16-byte")
    _refused(_fwd(lib, _dims(), o=ODD, saved=FAKE), "16-byte")
    bad = _dims()
    bad.o_strides[1] = 0
    _refused(_fwd(lib, bad), "stride 0 of o")
    bad = _dims()
    bad.g_strides[2] = -1
    _refused(_fwd(lib, bad), "negative stride of g")
    _refused(_bwd(lib, _dims(), do=None), "d_o is NULL")
    _refused(_bwd(lib, _dims(), dbeta=None), "dbeta is NULL")
    _refused(_bwd(lib, _dims(), dq=ODD), "16-byte")
    _refused(_bwd(lib, _dims(), do=ODD), "16-byte")
    _refused(_bwd(lib, _dims(), ws=(FAKE, 16)), "workspace")
    bad = _dims()
    bad.dv_strides[0] = 0
    _refused(_bwd(lib, bad), "stride 0 of dv")


def test_delta_sizes(lib):
    def size(d, which, dtype=0, cu=None):
        return lib.la_gated_delta_workspace_size(ctypes.byref(d), dtype, cu, which)

    def saved(d, dtype=0, cu=None):
        return lib.la_gated_delta_saved_size(ctypes.byref(d), dtype, cu)

    d = _dims()
    assert saved(d) > 0 and size(d, 3) == 0 and size(d, 0) > 0
    assert size(d, 2) >= size(d, 1) + saved(d)
    # decoding, fp32, widths the tensor cores do not take, rows off 16 bytes: token by token
    assert size(_dims(T=16), 0) == 0 and saved(_dims(T=16)) == 0 and size(_dims(T=16), 1) > 0
    assert saved(d, dtype=1) == 0 and saved(_dims(D=60)) == 0 and saved(_dims(E=136)) == 0
    odd = _dims()
    odd.q_strides[1] += 4
    assert saved(odd) == 0
    zero = _dims()
    zero.v_strides[0] = 0
    assert saved(zero) == 0
    # packed: the longest sequence decides, and room for every sequence's own chunks
    p = _dims(B=1, T=40, n=4)
    assert saved(p, cu=_cu([0, 10, 20, 30, 40])) == 0
    assert saved(p, cu=_cu([0, 0, 20, 20, 40])) > 0
    assert saved(p, cu=_cu([0, 0, 20, 20, 41])) == 0            # not a table of 40 tokens
    assert saved(_dims(HK=3)) == 0 and size(_dims(HK=3), 1) == 0


def test_delta_chunk_slots():
    # sequence n's chunks begin at slot cu[n] / 64 + n: no two sequences share a slot, all
    # slots lie below T / 64 + N, and a search over the first slots finds each one's sequence
    gen = torch.Generator().manual_seed(0)
    for _ in range(200):
        n = int(torch.randint(1, 12, (1,), generator=gen))
        lens = torch.randint(0, 200, (n,), generator=gen) * \
            (torch.rand(n, generator=gen) < 0.8).long()
        cu = [0] + torch.cumsum(lens, 0).tolist()
        first = [cu[i] // 64 + i for i in range(n)]
        taken = {}
        for i in range(n):
            for c in range(-(-(cu[i + 1] - cu[i]) // 64)):
                assert first[i] + c not in taken
                taken[first[i] + c] = i
        assert all(s < cu[-1] // 64 + n for s in taken)
        for s, i in taken.items():
            lo, hi = 0, n - 1
            while lo < hi:
                mid = (lo + hi + 1) // 2
                if first[mid] <= s:
                    lo = mid
                else:
                    hi = mid - 1
            assert lo == i


def test_delta_python_refusals():
    x = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        la.gated_delta_fwd(x, x, x, g, g)
    with pytest.raises(ValueError, match="B, T, H, D"):
        la.gated_delta_fwd(x[0], x, x, g, g)
    with pytest.raises(ValueError, match="cu_seqlens"):
        la.gated_delta(x[0], x[0], x[0], g[0], g[0])


# ---- norms around a block ---------------------------------------------------------------

def _norm_dims(B=2, T=5, H=3, D=16, act=2, w=0):
    st = I3(T * H * D, H * D, D)
    return N.LaBlockNormDims(B, T, H, D, act, w, *([st] * 10))


def _norm_fwd(lib, d, dtype=0, x=FAKE, gate=None, residual=None, post=None, pre=None, eps=1e-6,
              scale=1.0, h=ctypes.c_void_p(0x2000), y=None):
    return lib.la_block_norm_fwd(ctypes.byref(d) if d is not None else None, dtype, x, gate,
                                 residual, post, pre, eps, scale, h, y, None)


def _norm_bwd(lib, d, gate=None, post=None, pre=None, dh=FAKE, dy=None, dx=FAKE, dgate=None,
              dpost=None, dpre=None, ws=(FAKE, 1 << 40)):
    return lib.la_block_norm_bwd(ctypes.byref(d), 0, FAKE, gate, None, post, pre, 1e-6, 1.0, dh, dy,
                                 dx, dgate, None, dpost, dpre, *ws, None)


def test_norm_refusals(lib):
    _refused(_norm_fwd(lib, None), "dims")
    _refused(_norm_fwd(lib, _norm_dims(), dtype=3), "dtype 3")
    _refused(_norm_fwd(lib, _norm_dims(w=4)), "weight_dtype")
    _refused(_norm_fwd(lib, _norm_dims(act=3)), "activation")
    _refused(_norm_fwd(lib, _norm_dims(D=0)), "dim", N.LA_ERR_UNSUPPORTED)
    _refused(_norm_fwd(lib, _norm_dims(D=16385)), "dim", N.LA_ERR_UNSUPPORTED)
    _refused(_norm_fwd(lib, _norm_dims(H=0)), "heads")
    _refused(_norm_fwd(lib, _norm_dims(T=-1)), "negative")
    _refused(_norm_fwd(lib, _norm_dims(B=1 << 20, T=1 << 20)), "rows", N.LA_ERR_UNSUPPORTED)
    _refused(_norm_fwd(lib, _norm_dims(), x=None), "x is NULL")
    _refused(_norm_fwd(lib, _norm_dims(), h=None), "h is NULL")
    _refused(_norm_fwd(lib, _norm_dims(), eps=-1.0), "eps")
    _refused(_norm_fwd(lib, _norm_dims(), eps=float("nan")), "eps")
    _refused(_norm_fwd(lib, _norm_dims(), scale=float("inf")), "scale")
    _refused(_norm_fwd(lib, _norm_dims(), y=FAKE), "pre_weight")
    _refused(_norm_fwd(lib, _norm_dims(), pre=FAKE), "y is NULL")
    _refused(_norm_fwd(lib, _norm_dims(), pre=FAKE, y=FAKE), "overlaps")
    _refused(_norm_fwd(lib, _norm_dims(), gate=FAKE, h=FAKE), "overlaps")
    bad = _norm_dims()
    bad.h_strides[1] += 8
    _refused(_norm_fwd(lib, bad, h=FAKE), "in place")
    bad = _norm_dims()
    bad.h_strides[2] = 0
    _refused(_norm_fwd(lib, bad), "stride 0 of h")
    _refused(_norm_bwd(lib, _norm_dims(), dy=FAKE), "pre_weight")
    _refused(_norm_bwd(lib, _norm_dims(), dpost=FAKE), "post_weight")
    _refused(_norm_bwd(lib, _norm_dims(), dgate=FAKE), "gate")
    _refused(_norm_bwd(lib, _norm_dims(), gate=FAKE), "d_gate is NULL")
    _refused(_norm_bwd(lib, _norm_dims(), dx=None), "dx is NULL")
    _refused(_norm_bwd(lib, _norm_dims(), dh=None), "d_h is NULL")
    _refused(_norm_bwd(lib, _norm_dims(), pre=FAKE, dh=None), "d_y is NULL")
    _refused(_norm_bwd(lib, _norm_dims(), post=FAKE, dpost=FAKE, ws=(None, 0)), "workspace")
    assert lib.la_block_norm_workspace_size(ctypes.byref(_norm_dims()), 0) > 0
    assert lib.la_block_norm_workspace_size(ctypes.byref(_norm_dims(act=5)), 0) == 0


def test_norm_python_refusals():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        la.block_norm_fwd(x)
    with pytest.raises(ValueError, match="activation"):
        la.block_norm_fwd(x, activation="tanh")
