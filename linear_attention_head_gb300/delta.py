"""The gated delta rule over the C ABI (argument marshalling only, as api.py):

    S' = exp(g_t) S,  e_t = v_t - S'^T k_t,  S = S' + beta_t k_t e_t^T,  o_t = scale S^T q_t

per sequence and value head, forward (prompts in chunks on the tensor cores, a few tokens
against a carried state), backward and differentiable.  A backward pass that is to be captured
in a CUDA graph calls gated_delta_fwd and gated_delta_bwd, as those of layer.py.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .api import Tensor, _traced
from .layer import (_call, _code, _cu, _new, _on_device, _output, _ptr, _ref, _state_of, _strides,
                    _token, _workspace, _NONE3)

_pack = struct.Struct("=8i30q").pack
_dims = N.LaDeltaDims.from_buffer_copy


def _gate(t: Tensor, name: str, like: Tensor) -> Tensor:
    if t.shape != like.shape[:3]:
        raise ValueError("%s must be [B, T, H] = %s, got %s"
                         % (name, tuple(like.shape[:3]), tuple(t.shape)))
    if t.device != like.device:
        raise ValueError("all tensors must be on one device")
    if t.dtype not in (like.dtype, torch.float32):
        raise TypeError("%s must have the tokens' dtype %s or float32, got %s"
                        % (name, like.dtype, t.dtype))
    return t


def _rows16(t: Tensor) -> Tensor:
    """bf16 t with its rows on 16-byte boundaries (the tensor-core kernels' loads): itself, or a
    dense copy.  Rows that no copy puts there (odd channels) stay as they are."""
    if t.dtype != torch.bfloat16 or t.shape[3] % 8:
        return t
    if t.data_ptr() % 16 == 0 and all(s * t.element_size() % 16 == 0 and (s > 0 or n == 1)
                                      for s, n in zip(t.stride()[:3], t.shape[:3])):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _Call:
    """The arguments that the forward and the backward share."""

    def __init__(self, q, k, v, g, beta, scale, initial_state, cu_seqlens, cu_seqlens_host,
                 aligned):
        q = _token(q, "q")
        k, v = _token(k, "k", q), _token(v, "v", q)
        B, T, HK, D = q.shape
        if k.shape != q.shape:
            raise ValueError("q and k must share their shape [B, T, H_qk, D] (got %s, %s)"
                             % (tuple(q.shape), tuple(k.shape)))
        if v.shape[:2] != q.shape[:2]:
            raise ValueError("v must be [%d, %d, H, E], got %s" % (B, T, tuple(v.shape)))
        if k.dtype != q.dtype or v.dtype != q.dtype:
            raise TypeError("all token tensors must share one dtype")
        self.code = _code(q.dtype)
        H, E = v.shape[2:]
        if HK < 1 or H % HK:
            raise ValueError("the %d query and key heads must divide the %d value heads" % (HK, H))
        g, beta = _gate(g, "g", v), _gate(beta, "beta", v)
        if g.dtype != beta.dtype:
            raise TypeError("g and beta must share one dtype")
        if aligned:
            q, k, v = _rows16(q), _rows16(k), _rows16(v)
        self.q, self.k, self.v, self.g, self.beta = q, k, v, g, beta
        self.device = q.device
        self.scale = float(D ** -0.5 if scale is None else scale)
        self.cu = _cu(cu_seqlens, cu_seqlens_host, q.device, B)
        self.state_shape = (self.cu.n, H, D, E)
        self.init = _state_of(initial_state, self.state_shape, q.device, "initial_state")
        self._head = (B, T, H, HK, D, E, self.cu.n, _code(g.dtype)) + tuple(_strides(q)) + \
            tuple(_strides(k)) + tuple(_strides(v)) + tuple(g.stride()) + tuple(beta.stride())

    def dims(self, o=None, do=None, dq=None, dk=None, dv=None):
        return _dims(_pack(*self._head, *_strides(o), *_strides(do), *_strides(dq),
                           *_strides(dk), *_strides(dv)))

    def inputs(self):
        return (_ptr(self.q), _ptr(self.k), _ptr(self.v), _ptr(self.g), _ptr(self.beta))

    def saved_size(self, d) -> int:
        return int(N.lib().la_gated_delta_saved_size(_ref(d), self.code, _ptr(self.cu.host)))

    def workspace(self, d, backward):
        if backward == 0 and self._head[1] <= 16:
            return None, 0      # a few tokens forward: token by token, which takes none
        return _workspace(int(N.lib().la_gated_delta_workspace_size(
            _ref(d), self.code, _ptr(self.cu.host), backward)), self.device)


@_traced
def gated_delta_fwd(q: Tensor, k: Tensor, v: Tensor, g: Tensor, beta: Tensor,
                    scale: Optional[float] = None, initial_state: Optional[Tensor] = None,
                    cu_seqlens=None, cu_seqlens_host: Optional[Tensor] = None,
                    out: Optional[Tensor] = None, final_state: Optional[Tensor] = None,
                    want_final_state: bool = True, keep: bool = False):
    """The gated delta rule over q, k [B,T,H_qk,D] and v [B,T,H,E] (H a multiple of H_qk), with
    the log-decay g and the write strength beta [B,T,H], both of the tokens' dtype or fp32.
    Returns (o, final_state [N,H,D,E] fp32), and with keep=True (o, final_state, saved): what
    gated_delta_bwd starts from (None where it needs nothing), 66 KB for every 64 tokens of a
    head: 1.1 GB at 4 x 8192 tokens of 32 heads.

    scale: D^-1/2 when None.  q and k come normalised (QkNorm with weights D^-1/2 does it).
    final_state may be the initial_state tensor itself.  cu_seqlens packs the sequences in one
    row; with cu_seqlens_host (a CPU copy) given too the call copies nothing."""
    c = _Call(q, k, v, g, beta, scale, initial_state, cu_seqlens, cu_seqlens_host, keep)
    dev = c.device
    out = _output(out, c.v, "out")
    if final_state is not None:
        if tuple(final_state.shape) != c.state_shape or final_state.dtype != torch.float32 or \
                not final_state.is_contiguous() or final_state.device != dev:
            raise ValueError("final_state must be a contiguous fp32 tensor of shape %s on %s"
                             % (c.state_shape, dev))
    elif want_final_state:
        final_state = torch.empty(c.state_shape, dtype=torch.float32, device=dev)
    d = c.dims(o=out)
    saved, nsaved = None, 0
    if keep:
        saved, nsaved = _workspace(c.saved_size(d), dev)
    ws, nbytes = c.workspace(d, 3 if nsaved else 0)
    _call(dev, N.lib().la_gated_delta_fwd, _ref(d), c.code, *c.inputs(), c.scale, _ptr(c.init),
          _ptr(c.cu.dev), _ptr(c.cu.host), _ptr(out), _ptr(final_state), _ptr(saved), _ptr(ws),
          nbytes)
    return (out, final_state, saved) if keep else (out, final_state)


@_traced
def gated_delta_bwd(q: Tensor, k: Tensor, v: Tensor, g: Tensor, beta: Tensor, do: Tensor,
                    scale: Optional[float] = None, initial_state: Optional[Tensor] = None,
                    d_final_state: Optional[Tensor] = None, cu_seqlens=None,
                    cu_seqlens_host: Optional[Tensor] = None,
                    want_d_initial_state: bool = True, saved: Optional[Tensor] = None):
    """Backward of gated_delta_fwd: (dq, dk, dv, dg, dbeta, d_initial_state) of
    sum(o * do) + sum(final_state * d_final_state).  dg and dbeta have the tokens' dtype.
    saved: what gated_delta_fwd(..., keep=True) returned for the same arguments; without it it
    is computed again, in a workspace that lives for the call alone."""
    c = _Call(q, k, v, g, beta, scale, initial_state, cu_seqlens, cu_seqlens_host, True)
    dev = c.device
    do = _token(do, "do", c.v)
    if do.shape != c.v.shape or do.dtype != c.v.dtype:
        raise ValueError("do must have v's shape and dtype")
    do = _rows16(do)
    dfin = _state_of(d_final_state, c.state_shape, dev, "d_final_state")
    dq, dk, dv = _new(c.q), _new(c.k), _new(c.v)
    dg = torch.empty(c.v.shape[:3], dtype=c.v.dtype, device=dev)
    dbeta = torch.empty_like(dg)
    dinit = (torch.empty(c.state_shape, dtype=torch.float32, device=dev)
             if want_d_initial_state else None)
    d = c.dims(do=do, dq=dq, dk=dk, dv=dv)
    if saved is not None:
        want = c.saved_size(d)
        if saved.dtype != torch.uint8 or saved.device != dev or saved.numel() != want or \
                not saved.is_contiguous():
            raise ValueError("saved is not that of a gated_delta_fwd call of these sizes")
        if want == 0:
            saved = None
    ws, nbytes = c.workspace(d, 1 if saved is not None else 2)
    _call(dev, N.lib().la_gated_delta_bwd, _ref(d), c.code, *c.inputs(), _ptr(do), c.scale,
          _ptr(c.init), _ptr(dfin), _ptr(c.cu.dev), _ptr(c.cu.host), _ptr(saved), _ptr(dq),
          _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dinit), _ptr(ws), nbytes)
    return dq, dk, dv, dg, dbeta, dinit


class _GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, init, cu, scale, cu_host):
        grad = any(ctx.needs_input_grad)
        y = gated_delta_fwd(q, k, v, g, beta, scale, init, cu, cu_host, keep=grad)
        ctx.save_for_backward(q, k, v, g, beta, init, cu, cu_host, y[2] if grad else None)
        ctx.scale = scale
        ctx.set_materialize_grads(False)    # a final state that went unused has no gradient
        return y[0], y[1]

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dfin):
        if do is None and dfin is None:
            return (None,) * 9
        q, k, v, g, beta, init, cu, cu_host, saved = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.to(v.dtype)
        dq, dk, dv, dg, db, dinit = gated_delta_bwd(
            q, k, v, g, beta, do, ctx.scale, init, dfin, cu, cu_host,
            want_d_initial_state=init is not None, saved=saved)
        return (dq, dk, dv, dg.to(g.dtype), db.to(beta.dtype),
                None if dinit is None else dinit.to(init.dtype), None, None, None)


def gated_delta(q: Tensor, k: Tensor, v: Tensor, g: Tensor, beta: Tensor,
                scale: Optional[float] = None, initial_state: Optional[Tensor] = None,
                cu_seqlens=None, cu_seqlens_host: Optional[Tensor] = None):
    """Differentiable gated_delta_fwd: (o, final_state), in q, k, v, g, beta and initial_state.
    Accepts [B,T,H,D] or packed [T_total,H,D] (g and beta [T_total,H]) with cu_seqlens, as
    `recurrent`.  Between forward and backward the graph holds gated_delta_fwd's `saved`; who
    would rather have it made again calls gated_delta_fwd and gated_delta_bwd."""
    squeeze = v.ndim == 3
    if squeeze:
        if cu_seqlens is None:
            raise ValueError("3-D inputs need cu_seqlens")
        q, k, v, g, beta = (t[None] for t in (q, k, v, g, beta))
    if cu_seqlens is not None and cu_seqlens_host is None:
        cu_seqlens_host = torch.as_tensor(cu_seqlens).detach().to("cpu", torch.int32).contiguous()
    o, fin = _GatedDelta.apply(q, k, v, g, beta, initial_state, _on_device(cu_seqlens, v.device),
                               scale, cu_seqlens_host)
    return (o[0] if squeeze else o), fin
