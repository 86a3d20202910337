"""The operators that stand beside the attention in a layer, over the C ABI
(argument marshalling only, as api.py):

  * `qk_norm_rope`: norms of queries and keys for each head and the position
    rotation in one pass; `rotary`: the rotation alone.  `recurrent`,
    `recurrent_gla` and `lightning_attn` take them as qk_norm= and rope=.
  * `block_norm`: the norms before and after a block, with its gate and its
    residual scale.
  * `gated_scan`: the gated linear recurrence s_t = exp(g_t) s_{t-1} + x_t,
    elementwise, the vector-state sibling of `recurrent_gla`.

Each has its `_fwd` and `_bwd` call (the C ABI, one call each) and a
differentiable form.  A backward pass that is to be captured in a CUDA graph
calls `_fwd` and `_bwd`: they run on the current stream only.  (Autograd runs a
leaf's last step on the stream that an earlier graph of the same leaf used, and
while that graph lives a capture breaks off there.)
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .api import Tensor, _packed_batch_msg, _state, _traced

# The calls of a decoding step take a few microseconds on the GPU, so what the
# host does for one counts: structures are packed in one go, pointers are plain
# integers, the stream is asked for as one (torch.cuda.current_stream makes an
# object for it: 2 us of a call's 20).
_ref = ctypes.byref
_scan_pack = struct.Struct("=6i18q").pack
_rope_pack = struct.Struct("=12i21q128s").pack
_norm_pack = struct.Struct("=6i30q").pack
_norm_dims = N.LaBlockNormDims.from_buffer_copy
_scan_dims = N.LaScanDims.from_buffer_copy
_rope_dims = N.LaRopeDims.from_buffer_copy
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
_CODES = {torch.bfloat16: N.LA_DTYPE_BF16, torch.float32: N.LA_DTYPE_F32}
_NONE3 = (0, 0, 0)


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("token tensors must be bfloat16 or float32, got %s" % dtype)
    return code


def _ptr(t: Optional[Tensor]):
    return None if t is None else t.data_ptr()


def _strides(t: Optional[Tensor]):
    return _NONE3 if t is None else t.stride()[:3]


def _call(device, fn, *args) -> None:
    """fn(*args) with `device` current, on its current stream (the last argument)."""
    index = device.index
    if index == _current_device():
        st = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _current_stream(index))
    if st:
        N.check(st)


def _workspace(nbytes: int, device) -> Tuple[Optional[Tensor], int]:
    return (torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None), nbytes


def _token(t: Tensor, name: str, like: Optional[Tensor] = None) -> Tensor:
    """A [B, T, H, D] token tensor with contiguous channels, on `like`'s device."""
    if t.ndim != 4:
        raise ValueError("%s must be [B, T, H, D], got %s" % (name, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("token tensors must be CUDA tensors")
    if like is not None and t.device != like.device:
        raise ValueError("all tensors must be on one device")
    return t if t.is_contiguous() or t.stride(3) == 1 or t.shape[3] == 1 else t.contiguous()


def _new(like: Tensor) -> Tensor:
    """A dense tensor with the shape and the type of `like`."""
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=like.dtype, device=like.device)


def _state_of(x: Optional[Tensor], shape, device, name) -> Optional[Tensor]:
    """_state, without its conversions where x is as the call wants it."""
    if x is not None and x.dtype is torch.float32 and x.shape == shape and x.device == device \
            and x.is_contiguous():
        return x
    return _state(x, shape, device, name)


def _output(t: Optional[Tensor], like: Tensor, name: str) -> Tensor:
    """The caller's output, checked, or a dense new one with the shape of `like`."""
    if t is None:
        return _new(like)
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device or \
            (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s must be a %s tensor of shape %s with contiguous channels on %s"
                         % (name, like.dtype, tuple(like.shape), like.device))
    return t


class _Cu(NamedTuple):
    dev: Optional[Tensor]
    host: Optional[Tensor]
    n: int


def _cu(cu_seqlens, cu_seqlens_host, device, batch: int) -> _Cu:
    """cu_seqlens on the device and on the host.  With both given nothing is copied."""
    if cu_seqlens is None:
        if cu_seqlens_host is not None:
            raise ValueError("cu_seqlens_host needs cu_seqlens")
        return _Cu(None, None, batch)
    if batch != 1:
        raise ValueError(_packed_batch_msg(batch))
    cu = torch.as_tensor(cu_seqlens)
    if cu.ndim != 1 or cu.numel() < 1:
        raise ValueError("cu_seqlens must be 1-D with at least one entry")
    if cu_seqlens_host is None:
        host = cu.detach().to("cpu", torch.int32).contiguous()
    else:
        host = cu_seqlens_host
        if host.device.type != "cpu" or host.dtype != torch.int32 or \
                host.shape != cu.shape or not host.is_contiguous():
            raise ValueError("cu_seqlens_host must be a contiguous int32 CPU tensor of "
                             "cu_seqlens' shape")
    if cu.device != device or cu.dtype != torch.int32 or not cu.is_contiguous():
        cu = cu.to(device, torch.int32).contiguous()
    return _Cu(cu, host, host.numel() - 1)


# ---------------------------------------------------------------------------
# norms of queries and keys, rotation

class QkNorm(NamedTuple):
    """Norms of queries and keys for each head: x * rsqrt(mean(x^2) + eps) * weight, the
    weights [D] (None: ones)."""
    q_weight: Optional[Tensor] = None
    k_weight: Optional[Tensor] = None
    eps: float = 1e-6


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, device="cuda") -> Tensor:
    """base^(-2j / rotary_dim) for j < rotary_dim / 2, fp64: the angle of frequency pair j in
    radians per position."""
    j = torch.arange(rotary_dim // 2, dtype=torch.float64)
    return (float(base) ** (-2.0 * j / rotary_dim)).to(device)


class Rope:
    """A rotation, kept by the model: its frequencies and the axis of each.

    inv_freq   [rotary_dim / 2] radians per position (kept in fp64)
    sections   frequency pairs of each position axis, in order (their sum is the number of
               pairs), e.g. (16, 24, 24) for time, height, width; None: one axis
    axes       instead of sections: the axis of every pair, in any order
    interleaved  False: pair j is channels (j, j + rotary_dim/2); True: (2j, 2j + 1)
    """

    def __init__(self, inv_freq: Tensor, sections: Optional[Sequence[int]] = None,
                 axes: Optional[Sequence[int]] = None, interleaved: bool = False):
        self.inv_freq = torch.as_tensor(inv_freq).detach().to(torch.float64).contiguous()
        if self.inv_freq.ndim != 1 or not 1 <= self.inv_freq.numel() <= 128:
            raise ValueError("inv_freq must be 1-D with 1 to 128 frequencies")
        pairs = self.inv_freq.numel()
        if sections is not None:
            if axes is not None:
                raise ValueError("give sections or axes, not both")
            axes = [a for a, n in enumerate(sections) for _ in range(int(n))]
        axes = [0] * pairs if axes is None else [int(a) for a in axes]
        if len(axes) != pairs or min(axes) < 0 or max(axes) > 3:
            raise ValueError("%d frequencies need as many axes, each 0..3 (got %s)"
                             % (pairs, axes))
        self.num_axes = len(sections) if sections is not None else max(axes) + 1
        if self.num_axes > 4:
            raise ValueError("at most 4 position axes")
        self.axes = tuple(axes)
        self.rotary_dim = 2 * pairs
        self.interleaved = bool(interleaved)
        self._pair_axis = bytes(axes).ljust(128, b"\0")


class _RopeCall:
    """The arguments that the forward and the backward share."""

    def __init__(self, q, k, q_weight, k_weight, eps, normalize, rope, positions,
                 position_offset, cu_seqlens, cu_seqlens_host, names=("q", "k")):
        q = _token(q, names[0])
        dev = self.device = q.device
        B, T, H, D = q.shape
        heads = 0
        if k is not None:
            k = _token(k, names[1], q)
            if k.shape[:2] != q.shape[:2] or k.shape[3] != D:
                raise ValueError("%s must be [B, T, H, D] and %s [B, T, H_k, D] (got %s, %s)"
                                 % (names + (tuple(q.shape), tuple(k.shape))))
            if k.dtype != q.dtype:
                raise TypeError("all token tensors must share one dtype")
            heads = k.shape[2]
        elif k_weight is not None:
            raise ValueError("k_weight needs %s" % names[1])
        self.q, self.k = q, k
        self.dtype = w_code = _code(q.dtype)
        w_dtype = None
        for w in (q_weight, k_weight):
            if w is None:
                continue
            if w.shape != (D,) or w.device != dev:
                raise ValueError("weights must be [%d] on %s" % (D, dev))
            if w.dtype != (w_dtype or w.dtype):
                raise TypeError("the weights must share one dtype")
            w_dtype, w_code = w.dtype, _code(w.dtype)
        self.qw = q_weight.contiguous() if q_weight is not None else None
        self.kw = k_weight.contiguous() if k_weight is not None else None
        self.eps = float(eps)
        self.cu = _cu(cu_seqlens, cu_seqlens_host, dev, B)
        rotary, axes, interleaved, pair_axis, self.freq = 0, 1, 0, b"", None
        if rope is not None:
            rotary, axes, interleaved = rope.rotary_dim, rope.num_axes, int(rope.interleaved)
            pair_axis, self.freq = rope._pair_axis, rope.inv_freq
            if rotary > D:
                raise ValueError("rotary_dim %d exceeds the %d channels" % (rotary, D))
            if self.freq.device != dev:
                raise ValueError("inv_freq is on %s, the tensors on %s"
                                 % (self.freq.device, dev))
        elif positions is not None or position_offset is not None:
            raise ValueError("positions need rope")
        pos_strides, pos_bytes = _NONE3, 0
        if positions is not None:
            positions, pos_strides = self._positions(positions, axes, B, T)
            pos_bytes = positions.element_size()
        self.positions = positions
        if position_offset is not None:
            if positions is not None:
                raise ValueError("position_offset goes without positions")
            off = torch.as_tensor(position_offset)
            if tuple(off.shape) != (self.cu.n,):
                raise ValueError("position_offset must have one entry per sequence (%d), got %s"
                                 % (self.cu.n, tuple(off.shape)))
            position_offset = off.to(dev, torch.int32).contiguous()
        self.offset = position_offset
        self._head = (B, T, H, heads, D, rotary, self.cu.n, axes, 1 if normalize else 0,
                      interleaved, w_code, pos_bytes)
        self._tail = tuple(pos_strides) + (pair_axis,)

    def _positions(self, p, axes, B, T):
        """[axes, B, T] (or without the axes or the batch dimension where they are 1) and its
        strides, 0 where one row serves the whole batch."""
        if p.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64, got %s" % p.dtype)
        if p.device != self.device:
            raise ValueError("positions must be on %s" % self.device)
        shape, st = tuple(p.shape), p.stride()
        if len(shape) == 1 and axes == 1:
            shape, st = (1, 1) + shape, (0, 0) + st
        elif len(shape) == 2:
            shape, st = (((1,) + shape, (0,) + st) if axes == 1 else
                         ((shape[0], 1, shape[1]), (st[0], 0, st[1])))
        if len(shape) != 3 or shape[0] != axes or shape[1] not in (1, B) or shape[2] != T:
            raise ValueError("positions must be [%d, %d, %d] (axes, batch, tokens), got %s"
                             % (axes, B, T, tuple(p.shape)))
        return p, (st[0], st[1] if shape[1] > 1 else 0, st[2])

    def dims(self, q, k, qo, ko, dq=None, dk=None):
        return _rope_dims(_rope_pack(*self._head, *_strides(q), *_strides(k), *_strides(qo),
                                     *_strides(ko), *_strides(dq), *_strides(dk), *self._tail))

    def tail(self):
        """The argument run (weights, eps, frequencies, positions, packing) of the C ABI."""
        return (_ptr(self.qw), _ptr(self.kw), self.eps, _ptr(self.freq), _ptr(self.positions),
                _ptr(self.offset), _ptr(self.cu.dev), _ptr(self.cu.host))


def _pair_of(out, name):
    return (None, None) if out is None else out if isinstance(out, (tuple, list)) else (out, None)


@_traced
def qk_norm_rope_fwd(q: Tensor, k: Optional[Tensor] = None, q_weight: Optional[Tensor] = None,
                     k_weight: Optional[Tensor] = None, eps: float = 1e-6,
                     normalize: bool = True, rope: Optional[Rope] = None,
                     positions: Optional[Tensor] = None, position_offset=None, cu_seqlens=None,
                     cu_seqlens_host: Optional[Tensor] = None, out=None):
    """Norm and rotation of queries q [B,T,H,D] and keys k [B,T,H_k,D] (or of q alone).
    Returns (q', k'), or q' without k.

    rope: the rotation (None: norms only).  positions: [axes, B, T] int32 or int64, or with one
    axis [B, T] or [T]; None: each token's index in its sequence, plus position_offset [N]
    (decoding on).  cu_seqlens packs the sequences in one row; with cu_seqlens_host (a CPU
    copy) given too the call copies nothing.  out: (q', k') to write to; they may be q and k
    themselves."""
    c = _RopeCall(q, k, q_weight, k_weight, eps, normalize, rope, positions, position_offset,
                  cu_seqlens, cu_seqlens_host)
    qo, ko = _pair_of(out, "out")
    qo = _output(qo, c.q, "out")
    ko = _output(ko, c.k, "out") if c.k is not None else None
    d = c.dims(c.q, c.k, qo, ko)
    _call(c.device, N.lib().la_qk_norm_rope_fwd, _ref(d), c.dtype, _ptr(c.q), _ptr(c.k),
          *c.tail(), _ptr(qo), _ptr(ko))
    return (qo, ko) if c.k is not None else qo


def _rope_bwd(c: _RopeCall, x, want_weights: bool):
    """Gradients for the call c, whose q and k are the outputs' gradients; x: the inputs."""
    xq, xk = x
    dq = _new(c.q)
    dk = _new(c.k) if c.k is not None else None
    dqw = dkw = None
    if want_weights:
        dqw = torch.empty_like(c.qw) if c.qw is not None else None
        dkw = torch.empty_like(c.kw) if c.kw is not None else None
    d = c.dims(xq, xk, c.q, c.k, dq, dk)
    lib = N.lib()
    ws, nbytes = None, 0
    if dqw is not None or dkw is not None:
        ws, nbytes = _workspace(int(lib.la_qk_norm_rope_workspace_size(_ref(d), c.dtype)),
                                c.device)
    _call(c.device, lib.la_qk_norm_rope_bwd, _ref(d), c.dtype, _ptr(xq), _ptr(xk), _ptr(c.q),
          _ptr(c.k), *c.tail(), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(ws), nbytes)
    return dq, dk, dqw, dkw


@_traced
def qk_norm_rope_bwd(q: Tensor, k: Optional[Tensor], dq_out: Tensor,
                     dk_out: Optional[Tensor] = None, q_weight: Optional[Tensor] = None,
                     k_weight: Optional[Tensor] = None, eps: float = 1e-6,
                     normalize: bool = True, rope: Optional[Rope] = None,
                     positions: Optional[Tensor] = None, position_offset=None, cu_seqlens=None,
                     cu_seqlens_host: Optional[Tensor] = None):
    """Backward of qk_norm_rope_fwd on the same arguments, from the gradients of its outputs:
    (dq, dk, dq_weight, dk_weight), None for what was not given.  With normalize=False q and k
    are not read."""
    c = _RopeCall(dq_out, dk_out, q_weight, k_weight, eps, normalize, rope, positions,
                  position_offset, cu_seqlens, cu_seqlens_host, ("dq_out", "dk_out"))
    x = [None, None]
    if normalize:
        for i, (t, dy, name) in enumerate(((q, c.q, "q"), (k, c.k, "k"))):
            if (t is None) != (dy is None):
                raise ValueError("%s and its output's gradient go together" % name)
            if t is None:
                continue
            x[i] = _token(t, name, c.q)
            if t.shape != dy.shape or t.dtype != dy.dtype:
                raise ValueError("%s and its output's gradient must share shape and dtype" % name)
    return _rope_bwd(c, x, True)


@_traced
def rotary_fwd(q: Tensor, k: Optional[Tensor] = None, rope: Optional[Rope] = None,
               positions: Optional[Tensor] = None, position_offset=None, cu_seqlens=None,
               cu_seqlens_host: Optional[Tensor] = None, out=None):
    """The rotation alone (qk_norm_rope_fwd without the norms): one or several position axes."""
    if rope is None:
        raise ValueError("rotary needs rope")
    return qk_norm_rope_fwd(q, k, normalize=False, rope=rope, positions=positions,
                            position_offset=position_offset, cu_seqlens=cu_seqlens,
                            cu_seqlens_host=cu_seqlens_host, out=out)


@_traced
def rotary_bwd(dq_out: Tensor, dk_out: Optional[Tensor] = None, rope: Optional[Rope] = None,
               positions: Optional[Tensor] = None, position_offset=None, cu_seqlens=None,
               cu_seqlens_host: Optional[Tensor] = None):
    """Backward of rotary_fwd: the rotation back.  Returns (dq, dk), or dq without dk_out."""
    if rope is None:
        raise ValueError("rotary needs rope")
    c = _RopeCall(dq_out, dk_out, None, None, 0.0, False, rope, positions, position_offset,
                  cu_seqlens, cu_seqlens_host, ("dq_out", "dk_out"))
    dq, dk, _, _ = _rope_bwd(c, (None, None), False)
    return (dq, dk) if dk_out is not None else dq


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, qw, kw, positions, offset, cu, eps, normalize, rope, cu_host):
        y = qk_norm_rope_fwd(q, k, qw, kw, eps, normalize, rope, positions, offset, cu, cu_host)
        keep = (q, k) if normalize else (None, None)
        ctx.save_for_backward(*keep, qw, kw, positions, offset, cu, cu_host)
        ctx.eps, ctx.normalize, ctx.rope, ctx.dtype = eps, normalize, rope, q.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko=None):
        q, k, qw, kw, positions, offset, cu, cu_host = ctx.saved_tensors
        c = _RopeCall(dqo.to(ctx.dtype), dko.to(ctx.dtype) if dko is not None else None, qw, kw,
                      ctx.eps, ctx.normalize, ctx.rope, positions, offset, cu, cu_host)
        x = [None if t is None else _token(t, "q", c.q) for t in (q, k)]
        need = ctx.needs_input_grad
        dq, dk, dqw, dkw = _rope_bwd(c, x, need[2] or need[3])
        return (dq, dk, dqw, dkw) + (None,) * 7


def _on_device(x, device):
    """Integers given as a list or on the host, as an int32 tensor on the device."""
    return None if x is None else torch.as_tensor(x).to(device, torch.int32)


def qk_norm_rope(q: Tensor, k: Optional[Tensor] = None, norm: Optional[QkNorm] = None,
                 rope: Optional[Rope] = None, positions: Optional[Tensor] = None,
                 position_offset=None, cu_seqlens=None,
                 cu_seqlens_host: Optional[Tensor] = None):
    """Differentiable qk_norm_rope_fwd: in q, k and norm's weights.  norm None: no norms;
    rope None: no rotation.  Accepts [B,T,H,D] or packed [T_total,H,D] with cu_seqlens."""
    if norm is None and rope is None:
        raise ValueError("give norm, rope or both")
    squeeze = q.ndim == 3
    if squeeze:
        if cu_seqlens is None:
            raise ValueError("3-D inputs need cu_seqlens")
        q, k = q[None], k[None] if k is not None else None
    if cu_seqlens is not None and cu_seqlens_host is None:
        # the host copy once, for the backward too
        cu_seqlens_host = torch.as_tensor(cu_seqlens).detach().to("cpu", torch.int32).contiguous()
    qw, kw, eps = norm if norm is not None else (None, None, 0.0)
    y = _QkNormRope.apply(q, k, qw, kw, positions, _on_device(position_offset, q.device),
                          _on_device(cu_seqlens, q.device), eps, norm is not None, rope,
                          cu_seqlens_host)
    if not squeeze:
        return y
    return tuple(t[0] for t in y) if k is not None else y[0]


def rotary(q: Tensor, k: Optional[Tensor] = None, rope: Optional[Rope] = None,
           positions: Optional[Tensor] = None, position_offset=None, cu_seqlens=None,
           cu_seqlens_host: Optional[Tensor] = None):
    """Differentiable rotary_fwd."""
    if rope is None:
        raise ValueError("rotary needs rope")
    return qk_norm_rope(q, k, None, rope, positions, position_offset, cu_seqlens,
                        cu_seqlens_host)


# ---------------------------------------------------------------------------
# gated linear recurrence

def _scan_call(x, g, initial_state, cu_seqlens, cu_seqlens_host):
    x = _token(x, "x")
    if g.shape != x.shape:
        raise ValueError("g must have x's shape %s, got %s" % (tuple(x.shape), tuple(g.shape)))
    g = _token(g, "g", x)
    if g.dtype not in (x.dtype, torch.float32):
        raise TypeError("g must have x's dtype %s or float32, got %s" % (x.dtype, g.dtype))
    B, T, H, D = x.shape
    cu = _cu(cu_seqlens, cu_seqlens_host, x.device, B)
    init = _state_of(initial_state, (cu.n, H, D), x.device, "initial_state")
    head = (B, T, H, D, cu.n, _code(g.dtype)) + tuple(_strides(x)) + tuple(_strides(g))
    return x, g, init, cu, head, _code(x.dtype)


@_traced
def gated_scan_fwd(x: Tensor, g: Tensor, initial_state: Optional[Tensor] = None,
                   reverse: bool = False, cu_seqlens=None,
                   cu_seqlens_host: Optional[Tensor] = None, out: Optional[Tensor] = None,
                   final_state: Optional[Tensor] = None, want_final_state: bool = True,
                   keep_states: bool = False):
    """s_t = exp(g_t) s_{t-1} + x_t for every channel of x [B,T,H,D]; g, the log-decay, has x's
    shape and its dtype or fp32.  Returns (o, final_state [N,H,D] fp32), and with
    keep_states=True (o, final_state, states): what gated_scan_bwd starts from, 4 bytes a
    channel for every 128 tokens (every 8 where the sequences are short and many).
    final_state may be the initial_state tensor itself.  cu_seqlens, cu_seqlens_host and
    reverse as qk_norm_rope_fwd and la_fwd."""
    x, g, init, cu, head, code = _scan_call(x, g, initial_state, cu_seqlens, cu_seqlens_host)
    dev = x.device
    out = _output(out, x, "out")
    shape = (cu.n,) + tuple(x.shape[2:])
    if final_state is not None:
        if tuple(final_state.shape) != shape or final_state.dtype != torch.float32 or \
                not final_state.is_contiguous() or final_state.device != dev:
            raise ValueError("final_state must be a contiguous fp32 tensor of shape %s on %s"
                             % (shape, dev))
    elif want_final_state:
        final_state = torch.empty(shape, dtype=torch.float32, device=dev)
    d = _scan_dims(_scan_pack(*head, *_strides(out), *_NONE3, *_NONE3, *_NONE3))
    lib = N.lib()
    states = None
    if keep_states:
        states = torch.empty(int(lib.la_gated_scan_states_size(_ref(d))) // 4,
                             dtype=torch.float32, device=dev)
    in_place = init is not None and final_state is not None and \
        init.data_ptr() == final_state.data_ptr()
    ws, nbytes = _workspace(lib.la_gated_scan_workspace_size(_ref(d), code, 3 if in_place else 0),
                            dev)
    _call(dev, lib.la_gated_scan_fwd, _ref(d), code, _ptr(x), _ptr(g), _ptr(init),
          1 if reverse else 0, _ptr(cu.dev), _ptr(cu.host), _ptr(out), _ptr(final_state),
          _ptr(states), _ptr(ws), nbytes)
    return (out, final_state, states) if keep_states else (out, final_state)


@_traced
def gated_scan_bwd(x: Tensor, g: Tensor, do: Tensor, initial_state: Optional[Tensor] = None,
                   d_final_state: Optional[Tensor] = None, reverse: bool = False,
                   cu_seqlens=None, cu_seqlens_host: Optional[Tensor] = None,
                   want_d_initial_state: bool = True, states: Optional[Tensor] = None):
    """Backward of gated_scan_fwd: (dx, dg, d_initial_state) of
    sum(o * do) + sum(final_state * d_final_state); dg has g's dtype.  states: what
    gated_scan_fwd(..., keep_states=True) returned for the same arguments; without it they are
    computed again (one more pass over x and g)."""
    x, g, init, cu, head, code = _scan_call(x, g, initial_state, cu_seqlens, cu_seqlens_host)
    dev = x.device
    do = _token(do, "do", x)
    if do.shape != x.shape or do.dtype != x.dtype:
        raise ValueError("do must have x's shape and dtype")
    dfin = _state_of(d_final_state, (cu.n,) + tuple(x.shape[2:]), dev, "d_final_state")
    dx, dg = _new(x), _new(g)
    dinit = (torch.empty((cu.n,) + tuple(x.shape[2:]), dtype=torch.float32, device=dev)
             if want_d_initial_state else None)
    d = _scan_dims(_scan_pack(*head, *_NONE3, *_strides(do), *_strides(dx), *_strides(dg)))
    lib = N.lib()
    if states is not None:
        want = int(lib.la_gated_scan_states_size(_ref(d))) // 4
        if states.dtype != torch.float32 or states.device != dev or states.numel() != want or \
                not states.is_contiguous():
            raise ValueError("states are not those of a gated_scan_fwd call of these sizes")
        if want == 0:
            states = None
    ws, nbytes = _workspace(int(lib.la_gated_scan_workspace_size(
        _ref(d), code, 1 if states is not None else 2)), dev)
    _call(dev, lib.la_gated_scan_bwd, _ref(d), code, _ptr(x), _ptr(g), _ptr(do), _ptr(init),
          _ptr(dfin), 1 if reverse else 0, _ptr(cu.dev), _ptr(cu.host), _ptr(states), _ptr(dx),
          _ptr(dg), _ptr(dinit), _ptr(ws), nbytes)
    return dx, dg, dinit


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, init, cu, reverse, cu_host):
        grad = any(ctx.needs_input_grad)
        y = gated_scan_fwd(x, g, init, reverse, cu, cu_host, keep_states=grad)
        ctx.save_for_backward(x, g, init, cu, cu_host, y[2] if grad else None)
        ctx.reverse = reverse
        return y[0], y[1]

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dfin):
        x, g, init, cu, cu_host, states = ctx.saved_tensors
        dx, dg, dinit = gated_scan_bwd(x, g, do.to(x.dtype), init, dfin, ctx.reverse, cu,
                                       cu_host, want_d_initial_state=init is not None,
                                       states=states)
        return dx, dg, None if dinit is None else dinit.to(init.dtype), None, None, None


def gated_scan(x: Tensor, g: Tensor, initial_state: Optional[Tensor] = None,
               reverse: bool = False, cu_seqlens=None,
               cu_seqlens_host: Optional[Tensor] = None):
    """Differentiable gated_scan_fwd: (o, final_state), in x, g and initial_state.  Accepts
    [B,T,H,D] or packed [T_total,H,D] with cu_seqlens, as `recurrent`."""
    squeeze = x.ndim == 3
    if squeeze:
        if cu_seqlens is None:
            raise ValueError("3-D inputs need cu_seqlens")
        x, g = x[None], g[None]
    if cu_seqlens is not None and cu_seqlens_host is None:
        cu_seqlens_host = torch.as_tensor(cu_seqlens).detach().to("cpu", torch.int32).contiguous()
    o, fin = _GatedScan.apply(x, g, initial_state, _on_device(cu_seqlens, x.device),
                              bool(reverse), cu_seqlens_host)
    return (o[0] if squeeze else o), fin


# ---------------------------------------------------------------------------
# norms around a block

_ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2}


class _NormCall:
    """The arguments that the forward and the backward share; [B,T,C] as one head."""

    def __init__(self, x, gate, residual, post_weight, pre_weight, activation, scale, eps):
        kind = _ACTIVATIONS.get(activation)
        if kind is None:
            raise ValueError("activation must be one of %s, got %r"
                             % (sorted(_ACTIVATIONS), activation))
        if x.ndim not in (3, 4):
            raise ValueError("x must be [B, T, H, D] or [B, T, C], got %s" % (tuple(x.shape),))
        if not x.is_cuda:
            raise ValueError("token tensors must be CUDA tensors")
        self.x = x = self.channels(x)
        self.dtype = code = _code(x.dtype)
        self.device = x.device
        self.gate = self.like(gate, "gate")
        self.residual = self.like(residual, "residual")
        shape = x.shape
        w_dtype = None
        for w in (post_weight, pre_weight):
            if w is None:
                continue
            if w.shape != shape[-1:] or w.device != self.device:
                raise ValueError("weights must be [%d] on %s" % (shape[-1], self.device))
            if w.dtype != (w_dtype or w.dtype):
                raise TypeError("the weights must share one dtype")
            w_dtype, code = w.dtype, _code(w.dtype)
        self.post = post_weight.contiguous() if post_weight is not None else None
        self.pre = pre_weight.contiguous() if pre_weight is not None else None
        self.tail = (float(eps), float(scale))
        self._head = (tuple(shape) if len(shape) == 4 else (shape[0], shape[1], 1, shape[2])) + \
            (kind, code)

    @staticmethod
    def channels(t):
        return t if t.is_contiguous() or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()

    def like(self, t, name):
        """t with x's rows, or None."""
        if t is None:
            return None
        if t.shape != self.x.shape or t.dtype != self.x.dtype:
            raise ValueError("%s must have x's shape and dtype" % name)
        if t.device != self.device:
            raise ValueError("all tensors must be on one device")
        return self.channels(t)

    def dims(self, *outs):
        strides = []
        for t in (self.x, self.gate, self.residual) + outs:
            strides += (0, 0, 0) if t is None else t.stride()[:-1]
            if t is not None and t.ndim == 3:
                strides.append(0)
        return _norm_dims(_norm_pack(*self._head, *strides))

    def inputs(self):
        return (_ptr(self.x), _ptr(self.gate), _ptr(self.residual), _ptr(self.post),
                _ptr(self.pre)) + self.tail


@_traced
def block_norm_fwd(x: Tensor, gate: Optional[Tensor] = None, residual: Optional[Tensor] = None,
                   post_weight: Optional[Tensor] = None, pre_weight: Optional[Tensor] = None,
                   activation: str = "silu", scale: float = 1.0, eps: float = 1e-6, out=None):
    """The norms around a block over rows x [B,T,H,D] or [B,T,C], in one pass:
        n = rms(x) * post_weight   (x without post_weight),   m = n * act(gate),
        h = residual + scale * m,   y = rms(h) * pre_weight,
    rms(x) = x * rsqrt(mean(x^2) + eps).  Returns (h, y), y None without pre_weight.

    A layer's end: block_norm_fwd(block_out, residual=stream, pre_weight=next_norm) gives the
    stream and the next block's input; the heads' outputs, normalised and gated:
    block_norm_fwd(o, gate=z, post_weight=w)[0].  activation: "none", "sigmoid" or "silu" of
    the gate.  out: (h, y) to write to; h may be x or residual itself."""
    c = _NormCall(x, gate, residual, post_weight, pre_weight, activation, scale, eps)
    h, y = _pair_of(out, "out")
    h = _output(h, c.x, "out")
    y = _output(y, c.x, "out") if c.pre is not None else None
    d = c.dims(h, y, None, None, None, None, None)
    _call(c.device, N.lib().la_block_norm_fwd, _ref(d), c.dtype, *c.inputs(), _ptr(h), _ptr(y))
    return h, y


@_traced
def block_norm_bwd(x: Tensor, dh: Optional[Tensor], dy: Optional[Tensor] = None,
                   gate: Optional[Tensor] = None, residual: Optional[Tensor] = None,
                   post_weight: Optional[Tensor] = None, pre_weight: Optional[Tensor] = None,
                   activation: str = "silu", scale: float = 1.0, eps: float = 1e-6):
    """Backward of block_norm_fwd on the same arguments, from the gradients of h and y (either
    may be None, not both): (dx, dgate, dresidual, dpost_weight, dpre_weight), None for what was
    not given."""
    c = _NormCall(x, gate, residual, post_weight, pre_weight, activation, scale, eps)
    dh, dy = c.like(dh, "dh"), c.like(dy, "dy")
    if dy is not None and c.pre is None:
        raise ValueError("dy needs pre_weight")
    if dy is None and c.pre is not None:
        if dh is None:
            raise ValueError("give dh, dy or both")
        # y went unused: the same block without it
        g = block_norm_bwd(x, dh, None, gate, residual, post_weight, None, activation,
                           scale, eps)
        return g[:4] + (torch.zeros_like(c.pre),)
    if dh is None and dy is None:
        raise ValueError("give dh, dy or both")
    dx = _new(c.x)
    dgate = _new(c.x) if c.gate is not None else None
    dres = _new(c.x) if c.residual is not None else None
    dpost = torch.empty_like(c.post) if c.post is not None else None
    dpre = torch.empty_like(c.pre) if c.pre is not None else None
    d = c.dims(None, None, dh, dy, dx, dgate, dres)
    lib = N.lib()
    ws, nbytes = None, 0
    if dpost is not None or dpre is not None:
        ws, nbytes = _workspace(int(lib.la_block_norm_workspace_size(_ref(d), c.dtype)), c.device)
    _call(c.device, lib.la_block_norm_bwd, _ref(d), c.dtype, *c.inputs(), _ptr(dh), _ptr(dy),
          _ptr(dx), _ptr(dgate), _ptr(dres), _ptr(dpost), _ptr(dpre), _ptr(ws), nbytes)
    return dx, dgate, dres, dpost, dpre


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, residual, post, pre, activation, scale, eps):
        ctx.save_for_backward(x, gate, residual, post, pre)
        ctx.args = (activation, scale, eps)
        ctx.set_materialize_grads(False)
        return block_norm_fwd(x, gate, residual, post, pre, activation, scale, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy=None):
        x, gate, residual, post, pre = ctx.saved_tensors
        if dh is None and dy is None:
            return (None,) * 8
        dh, dy = (None if t is None else t.to(x.dtype) for t in (dh, dy))
        return block_norm_bwd(x, dh, dy, gate, residual, post, pre, *ctx.args) + (None,) * 3


def block_norm(x: Tensor, gate: Optional[Tensor] = None, residual: Optional[Tensor] = None,
               post_weight: Optional[Tensor] = None, pre_weight: Optional[Tensor] = None,
               activation: str = "silu", scale: float = 1.0, eps: float = 1e-6):
    """Differentiable block_norm_fwd: (h, y), in x, gate, residual and the weights."""
    return _BlockNorm.apply(x, gate, residual, post_weight, pre_weight, activation, scale, eps)
