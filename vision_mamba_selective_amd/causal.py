"""Torch-facing binding of the causal mixer (include/vimscan.h, "The causal
mixer"): the short causal convolution and the causal selective scan of
prompts, their gradients, and their single-token forms on pools of states.

Activations are [batch, dim, L] (fp32 or bf16), token stride 1; batch and
channel strides are free, so the halves of a projection's output or a span of
a longer tensor go in as they are. Outputs are contiguous. lengths is an int32
tensor [batch] on the device, or None when every row has L tokens: what stands
at and past a row's length is never used, outputs there are zero.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _native as nat
from .scan import _DTYPES, _ptr

_lib = nat.lib
_F32 = torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(device):
    """The current stream's handle on a device (of a tensor, so with an index):
    as torch.cuda.current_stream(device).cuda_stream, without making an object."""
    return _raw_stream(device.index)


def _fail(name, t, shape, dtype, device):
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    raise ValueError("%s must be contiguous" % name)


def _dense(name, t, shape, dtype, device):
    """A contiguous tensor of this shape, or None."""
    if t is not None and not (t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _fail(name, t, shape, dtype, device)


def _input(name, t, shape, dtype, device):
    """An activation of this shape: contiguous along its last axis, other strides free."""
    if not (t.dtype == dtype and t.shape == shape and t.device == device):
        _fail(name, t, shape, dtype, device)
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError("%s must be contiguous along its last axis" % name)


def _need(name, t):
    if t is None:
        raise ValueError("%s is required" % name)


def _start(name, t, ndim):
    if t.dtype not in _DTYPES:
        raise TypeError("unsupported dtype %s" % t.dtype)
    if t.ndim != ndim:
        raise ValueError("%s must have %d axes, got shape %s" % (name, ndim, tuple(t.shape)))
    if t.device.type != "cuda":
        raise ValueError("%s must be on the GPU" % name)
    return t.dtype, t.device


def _strides(*tensors):
    """The ABI's stride array (batch and channel stride of each); None when all are contiguous."""
    if all(t is None or t.is_contiguous() for t in tensors):
        return None
    v = []
    for t in tensors:
        v += (0, 0) if t is None else t.stride()[:2]
    return (ctypes.c_int64 * len(v))(*v)


def _lengths(lengths, batch, device):
    _dense("lengths", lengths, (batch,), torch.int32, device)


def _out(name, out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dense(name, out, shape, dtype, device)
    return out


def s6_workspace_bytes(op: int, batch: int, dim: int, inner: int, seqlen: int) -> int:
    """Bytes of a buffer of the causal entry points (op: VS_S6_SCAN, VS_S6_SAVED,
    VS_S6_GRAD, or VS_S6_CONV_GRAD with the width in place of dstate)."""
    return int(_lib.s6_workspace_bytes(op, batch, dim, inner, seqlen))


def _buffer(name, op, batch, dim, inner, L, device, given):
    need = _lib.s6_workspace_bytes(op, batch, dim, inner, L)
    if given is None:
        return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need
    have = given.numel() * given.element_size()
    if have < need or not given.is_contiguous() or given.device != device:
        raise ValueError("%s needs %d contiguous bytes on %s" % (name, need, device))
    return given, have


# ------------------------------------------------------------- convolution
def s6_causal_conv(x, w, bias=None, window=None, lengths=None, silu=True, out=None, window_out=None):
    """Depthwise causal convolution of prompts: y[t] = silu(bias + sum_j w[j]
    line[t + j]), line = [window | x].

    x [batch, dim, L]; w [dim, width] fp32 (tap width-1 multiplies the token
    itself); bias [dim] fp32 or None; window [batch, dim, width-1] in x's dtype
    (the tokens before x) or None. Returns (y, window_out): window_out holds
    the row's last width-1 entries, the window of the text that follows.
    """
    dt, dev = _start("x", x, 3)
    batch, dim, L = x.shape
    width = w.shape[-1]
    _input("x", x, (batch, dim, L), dt, dev)
    _dense("w", w, (dim, width), _F32, dev)
    _dense("bias", bias, (dim,), _F32, dev)
    _dense("window", window, (batch, dim, width - 1), dt, dev)
    _lengths(lengths, batch, dev)
    y = _out("out", out, (batch, dim, L), dt, dev)
    wo = _out("window_out", window_out, (batch, dim, width - 1), dt, dev)
    rc = _lib.s6_causal_conv(batch, dim, width, L, _DTYPES[dt], 1 if silu else 0, x.data_ptr(), _strides(x),
                             w.data_ptr(), _ptr(bias), _ptr(window), _ptr(lengths), y.data_ptr(), wo.data_ptr(), _stream(dev))
    nat.check("s6_causal_conv", rc)
    return y, wo


def s6_causal_conv_grad(x, w, bias, dy, window=None, dwindow=None, lengths=None, silu=True, workspace=None):
    """Gradient of s6_causal_conv for dy = dL/dy [batch, dim, L] and dwindow =
    dL/d window_out (or None). Returns a dict: dx [batch, dim, L] in x's dtype;
    dw [dim, width], dbias [dim] fp32; dwindow, the gradient of the incoming
    window (None without one)."""
    dt, dev = _start("x", x, 3)
    batch, dim, L = x.shape
    width = w.shape[-1]
    _input("x", x, (batch, dim, L), dt, dev)
    _input("dy", dy, (batch, dim, L), dt, dev)
    _dense("w", w, (dim, width), _F32, dev)
    _dense("bias", bias, (dim,), _F32, dev)
    _dense("window", window, (batch, dim, width - 1), dt, dev)
    _dense("dwindow", dwindow, (batch, dim, width - 1), dt, dev)
    _lengths(lengths, batch, dev)
    ws, ws_bytes = _buffer("workspace", nat.VS_S6_CONV_GRAD, batch, dim, width, L, dev, workspace)
    dx = torch.empty((batch, dim, L), dtype=dt, device=dev)
    dw = torch.empty((dim, width), dtype=_F32, device=dev)
    db = torch.empty((dim,), dtype=_F32, device=dev)
    dwin = None if window is None else torch.empty((batch, dim, width - 1), dtype=dt, device=dev)
    rc = _lib.s6_causal_conv_grad(batch, dim, width, L, _DTYPES[dt], 1 if silu else 0, x.data_ptr(), dy.data_ptr(),
                                  _strides(x, dy), w.data_ptr(), _ptr(bias), _ptr(window), _ptr(lengths), _ptr(dwindow),
                                  dx.data_ptr(), dw.data_ptr(), db.data_ptr(), _ptr(dwin), _ptr(ws), ws_bytes, _stream(dev))
    nat.check("s6_causal_conv_grad", rc)
    return dict(dx=dx, dw=dw, dbias=db, dwindow=dwin)


def _slots(slot_in, slot_out, batch, dev):
    _dense("slot_in", slot_in, (batch,), torch.int32, dev)
    _dense("slot_out", slot_out, (batch,), torch.int32, dev)


def s6_conv_step(x, w, bias, window, slot_in=None, slot_out=None, silu=True, out=None):
    """One token of s6_causal_conv for each row: x [batch, dim] (any row
    stride); window, the pool [slots, dim, width-1] in x's dtype, is read at
    slot_in[b] and written at slot_out[b] (int32 [batch], None: slot b). A row
    whose slot is outside the pool is empty: y is zero there and no state
    changes. Rows may read one slot together (a fork); no slot that a row
    writes may be read or written by another row. Returns y [batch, dim]."""
    dt, dev = _start("x", x, 2)
    batch, dim = x.shape
    width = w.shape[-1]
    slots = window.shape[0]
    _input("x", x, (batch, dim), dt, dev)
    if batch > 1 and x.stride(0) == 0:      # one row for all: the ABI's stride 0 means dense rows
        x = x.contiguous()
    _dense("w", w, (dim, width), _F32, dev)
    _dense("bias", bias, (dim,), _F32, dev)
    _dense("window", window, (slots, dim, width - 1), dt, dev)
    _slots(slot_in, slot_out, batch, dev)
    y = _out("out", out, (batch, dim), dt, dev)
    rc = _lib.s6_conv_step(batch, dim, width, _DTYPES[dt], 1 if silu else 0, x.data_ptr(), x.stride(0) if batch > 1 else 0,
                           w.data_ptr(), _ptr(bias), window.data_ptr(), slots, _ptr(slot_in), _ptr(slot_out), y.data_ptr(),
                           _stream(dev))
    nat.check("s6_conv_step", rc)
    return y


# -------------------------------------------------------------------- scan
def _scan_inputs(u, delta, z, B, C, A, Dskip, dt_bias, lengths):
    dt, dev = _start("u", u, 3)
    act = u.shape
    batch, dim, L = act
    _need("A", A)
    dstate = A.shape[-1]
    _input("u", u, act, dt, dev)
    _input("delta", delta, act, dt, dev)
    if z is not None:
        _input("z", z, act, dt, dev)
    _input("B", B, (batch, dstate, L), dt, dev)
    _input("C", C, (batch, dstate, L), dt, dev)
    _dense("A", A, (dim, dstate), _F32, dev)
    _dense("Dskip", Dskip, (dim,), _F32, dev)
    _dense("dt_bias", dt_bias, (dim,), _F32, dev)
    _lengths(lengths, batch, dev)
    return dt, dev, batch, dim, dstate, L


def s6_causal_scan(u, delta, z, B, C, A, Dskip=None, dt_bias=None, h0=None, lengths=None, delta_softplus=True,
                   out=None, h_out=None, workspace=None):
    """Causal selective scan of prompts, gated by silu(z) (z None: no gate).

    u, delta, z [batch, dim, L]; B, C [batch, dstate, L]; A [dim, dstate],
    Dskip, dt_bias [dim] fp32; h0 [batch, dim, dstate] fp32, the state before
    token 0 (None: zeros). Returns (y, h): y [batch, dim, L] and the state
    after each row's last token.
    """
    dt, dev, batch, dim, dstate, L = _scan_inputs(u, delta, z, B, C, A, Dskip, dt_bias, lengths)
    _dense("h0", h0, (batch, dim, dstate), _F32, dev)
    y = _out("out", out, (batch, dim, L), dt, dev)
    h = _out("h_out", h_out, (batch, dim, dstate), _F32, dev)
    ws, ws_bytes = _buffer("workspace", nat.VS_S6_SCAN, batch, dim, dstate, L, dev, workspace)
    rc = _lib.s6_causal_scan(batch, dim, dstate, L, _DTYPES[dt], 1 if delta_softplus else 0, u.data_ptr(), delta.data_ptr(),
                             _ptr(z), B.data_ptr(), C.data_ptr(), _strides(u, delta, z, B, C), A.data_ptr(), _ptr(Dskip),
                             _ptr(dt_bias), _ptr(h0), _ptr(lengths), y.data_ptr(), h.data_ptr(), _ptr(ws), ws_bytes, _stream(dev))
    nat.check("s6_causal_scan", rc)
    return y, h


def s6_causal_scan_saved(u, delta, z, B, C, A, Dskip=None, dt_bias=None, h0=None, lengths=None, delta_softplus=True,
                         out=None, h_out=None, saved=None, workspace=None):
    """s6_causal_scan for training: returns (y, h, saved); saved is the opaque
    buffer that s6_causal_scan_grad reads instead of running the scan again."""
    dt, dev, batch, dim, dstate, L = _scan_inputs(u, delta, z, B, C, A, Dskip, dt_bias, lengths)
    _dense("h0", h0, (batch, dim, dstate), _F32, dev)
    y = _out("out", out, (batch, dim, L), dt, dev)
    h = _out("h_out", h_out, (batch, dim, dstate), _F32, dev)
    sv, sv_bytes = _buffer("saved", nat.VS_S6_SAVED, batch, dim, dstate, L, dev, saved)
    ws, ws_bytes = _buffer("workspace", nat.VS_S6_SCAN, batch, dim, dstate, L, dev, workspace)
    rc = _lib.s6_causal_scan_saved(batch, dim, dstate, L, _DTYPES[dt], 1 if delta_softplus else 0, u.data_ptr(),
                                   delta.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), _strides(u, delta, z, B, C),
                                   A.data_ptr(), _ptr(Dskip), _ptr(dt_bias), _ptr(h0), _ptr(lengths), y.data_ptr(),
                                   h.data_ptr(), sv.data_ptr(), sv_bytes, _ptr(ws), ws_bytes, _stream(dev))
    nat.check("s6_causal_scan_saved", rc)
    return y, h, sv


def s6_causal_scan_grad(u, delta, z, B, C, A, Dskip, dt_bias, saved, dy, dh=None, h0=None, lengths=None,
                        delta_softplus=True, workspace=None):
    """Gradient of s6_causal_scan for dy = dL/dy and dh = dL/dh (or None),
    from the saved buffer of s6_causal_scan_saved on the same inputs. Returns a
    dict: du, ddelta, dz (None without z) [batch, dim, L] in the input dtype;
    dB, dC [batch, dstate, L], dA [dim, dstate], dD, ddt_bias [dim] and dh0
    [batch, dim, dstate] (None without h0) in fp32."""
    dt, dev, batch, dim, dstate, L = _scan_inputs(u, delta, z, B, C, A, Dskip, dt_bias, lengths)
    _input("dy", dy, (batch, dim, L), dt, dev)
    _dense("dh", dh, (batch, dim, dstate), _F32, dev)
    _dense("h0", h0, (batch, dim, dstate), _F32, dev)
    _need("saved", saved)
    sv, sv_bytes = _buffer("saved", nat.VS_S6_SAVED, batch, dim, dstate, L, dev, saved)
    ws, ws_bytes = _buffer("workspace", nat.VS_S6_GRAD, batch, dim, dstate, L, dev, workspace)
    new = lambda shape, d=_F32: torch.empty(shape, dtype=d, device=dev)  # noqa: E731
    act = (batch, dim, L)
    g = dict(du=new(act, dt), ddelta=new(act, dt), dz=None if z is None else new(act, dt),
             dB=new((batch, dstate, L)), dC=new((batch, dstate, L)), dA=new((dim, dstate)), dD=new((dim,)),
             ddt_bias=new((dim,)), dh0=None if h0 is None else new((batch, dim, dstate)))
    rc = _lib.s6_causal_scan_grad(batch, dim, dstate, L, _DTYPES[dt], 1 if delta_softplus else 0, u.data_ptr(),
                                  delta.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), dy.data_ptr(),
                                  _strides(u, delta, z, B, C, dy), A.data_ptr(), _ptr(Dskip), _ptr(dt_bias), _ptr(lengths),
                                  sv.data_ptr(), sv_bytes, _ptr(dh), g["du"].data_ptr(), g["ddelta"].data_ptr(), _ptr(g["dz"]),
                                  g["dB"].data_ptr(), g["dC"].data_ptr(), g["dA"].data_ptr(), g["dD"].data_ptr(),
                                  g["ddt_bias"].data_ptr(), _ptr(g["dh0"]), _ptr(ws), ws_bytes, _stream(dev))
    nat.check("s6_causal_scan_grad", rc)
    return g


def s6_scan_step(u, delta, z, B, C, A, Dskip, dt_bias, h, slot_in=None, slot_out=None, delta_softplus=True, out=None):
    """One token of s6_causal_scan for each row: u, delta, z [batch, dim], B, C
    [batch, dstate] (any row strides); h, the pool [slots, dim, dstate] fp32,
    is read at slot_in[b] and written at slot_out[b], as in s6_conv_step.
    Returns y [batch, dim]."""
    dt, dev = _start("u", u, 2)
    batch, dim = u.shape
    dstate = A.shape[-1]
    slots = h.shape[0]
    _input("u", u, (batch, dim), dt, dev)
    _input("delta", delta, (batch, dim), dt, dev)
    if z is not None:
        _input("z", z, (batch, dim), dt, dev)
    _input("B", B, (batch, dstate), dt, dev)
    _input("C", C, (batch, dstate), dt, dev)
    _dense("A", A, (dim, dstate), _F32, dev)
    _dense("Dskip", Dskip, (dim,), _F32, dev)
    _dense("dt_bias", dt_bias, (dim,), _F32, dev)
    _dense("h", h, (slots, dim, dstate), _F32, dev)
    _slots(slot_in, slot_out, batch, dev)
    y = _out("out", out, (batch, dim), dt, dev)
    st = None
    if batch > 1 and not all(t is None or t.is_contiguous() for t in (u, delta, z, B, C)):
        st = (ctypes.c_int64 * 5)(*(0 if t is None else t.stride(0) for t in (u, delta, z, B, C)))
    rc = _lib.s6_scan_step(batch, dim, dstate, _DTYPES[dt], 1 if delta_softplus else 0, u.data_ptr(), delta.data_ptr(), _ptr(z),
                           B.data_ptr(), C.data_ptr(), st, A.data_ptr(), _ptr(Dskip), _ptr(dt_bias), h.data_ptr(), slots,
                           _ptr(slot_in), _ptr(slot_out), y.data_ptr(), _stream(dev))
    nat.check("s6_scan_step", rc)
    return y


# ---------------------------------------------------------------- autograd
def _rows(g, like):
    """An incoming gradient in the dtype of the activation, contiguous along its last axis."""
    if g is None:
        return None
    g = g.to(like.dtype)
    return g if g.stride(-1) == 1 and min(g.stride()) >= 0 else g.contiguous()


class CausalConvFunction(torch.autograd.Function):
    """s6_causal_conv for autograd; both outputs are differentiable, once: a
    gradient of the gradient is refused."""

    @staticmethod
    def forward(ctx, x, w, bias, window, lengths, silu):
        y, wo = s6_causal_conv(x, w, bias, window=window, lengths=lengths, silu=silu)
        ctx.save_for_backward(x, w, bias, window, lengths)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        return y, wo

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dwo):
        x, w, bias, window, lengths = ctx.saved_tensors
        dy = x.new_zeros(x.shape) if dy is None else _rows(dy, x)
        g = s6_causal_conv_grad(x, w, bias, dy, window=window, lengths=lengths, silu=ctx.silu,
                                dwindow=None if dwo is None else dwo.to(x.dtype).contiguous())
        return g["dx"], g["dw"], None if bias is None else g["dbias"], g["dwindow"], None, None


def s6_causal_conv_autograd(x, w, bias=None, window=None, lengths=None, silu=True):
    """s6_causal_conv as a differentiable op (CausalConvFunction)."""
    return CausalConvFunction.apply(x, w, bias, window, lengths, silu)


class CausalScanFunction(torch.autograd.Function):
    """s6_causal_scan for autograd: the forward keeps the saved buffer for the
    backward; y and h are differentiable, once: a gradient of the gradient is
    refused. The gradients of B and C come back
    in their dtype (the library sums them in fp32)."""

    @staticmethod
    def forward(ctx, u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, delta_softplus):
        y, h, saved = s6_causal_scan_saved(u, delta, z, B, C, A, Dskip, dt_bias, h0=h0, lengths=lengths,
                                           delta_softplus=delta_softplus)
        ctx.save_for_backward(u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, saved)
        ctx.delta_softplus = delta_softplus
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, saved = ctx.saved_tensors
        dy = u.new_zeros(u.shape) if dy is None else _rows(dy, u)
        g = s6_causal_scan_grad(u, delta, z, B, C, A, Dskip, dt_bias, saved, dy, h0=h0, lengths=lengths,
                                dh=None if dh is None else dh.float().contiguous(), delta_softplus=ctx.delta_softplus)
        return (g["du"], g["ddelta"], g["dz"], g["dB"].to(B.dtype), g["dC"].to(C.dtype), g["dA"],
                None if Dskip is None else g["dD"], None if dt_bias is None else g["ddt_bias"], g["dh0"], None, None)


def s6_causal_scan_autograd(u, delta, z, B, C, A, Dskip=None, dt_bias=None, h0=None, lengths=None, delta_softplus=True):
    """s6_causal_scan as a differentiable op (CausalScanFunction). Returns (y, h)."""
    return CausalScanFunction.apply(u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, delta_softplus)
