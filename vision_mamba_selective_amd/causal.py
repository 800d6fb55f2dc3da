"""Torch-facing binding of the causal mixer (include/vimscan.h, "The causal
mixer"): the short causal convolution and the causal selective scan of
prompts, their gradients, and their single-token forms on pools of states.

Activations are [batch, dim, L] (fp32 or bf16), token stride 1; batch and
channel strides are free, so the halves of a projection's output or a span of
a longer tensor go in as they are. Outputs are contiguous. lengths is an int32
tensor [batch] on the device, or None when every row has L tokens: what stands
at and past a row's length is never used, outputs there are zero.

Only s6_causal_conv_autograd and s6_causal_scan_autograd are differentiable:
what every other function returns is outside any graph, also where an input
requires a gradient. A tensor that a call writes in place (a pool, a given
output or buffer) gets a new version, as after torch's in-place operations, and
is refused if it requires a gradient while gradients are recorded.

The differentiable functions here, in gated.py, norm.py and loss.py may be captured
in a HIP graph together with their backward pass, in torch's order: a run on a
side stream first, and no eager graph alive that has leaves in common with what
is captured. Such a graph of another stream, whose backward nodes would end the
process, is refused with a RuntimeError while capturing and recording gradients,
as far as it leads to the call's inputs; what enters a captured graph by torch's
own operations alone is not seen. A forward pass by itself is captured under
torch.no_grad().
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _calls
from . import _native as nat


def s6_workspace_bytes(op: int, batch: int, dim: int, inner: int, seqlen: int) -> int:
    """Bytes of a buffer of the causal entry points (op: VS_S6_SCAN, VS_S6_SAVED,
    VS_S6_GRAD, or VS_S6_CONV_GRAD with the width in place of dstate)."""
    return int(nat.lib.s6_workspace_bytes(op, batch, dim, inner, seqlen))


# ------------------------------------------------------------- convolution
def s6_causal_conv(x, w, bias=None, window=None, lengths=None, silu=True, out=None, window_out=None):
    """Depthwise causal convolution of prompts: y[t] = silu(bias + sum_j w[j]
    line[t + j]), line = [window | x].

    x [batch, dim, L]; w [dim, width] fp32 (tap width-1 multiplies the token
    itself); bias [dim] fp32 or None; window [batch, dim, width-1] in x's dtype
    (the tokens before x) or None. Returns (y, window_out): window_out holds
    the row's last width-1 entries, the window of the text that follows.
    """
    return _calls.s6_causal_conv(x, w, bias, window, lengths, silu, out, window_out)


def s6_causal_conv_grad(x, w, bias, dy, window=None, dwindow=None, lengths=None, silu=True, workspace=None):
    """Gradient of s6_causal_conv for dy = dL/dy [batch, dim, L] and dwindow =
    dL/d window_out (or None). Returns a dict: dx [batch, dim, L] in x's dtype;
    dw [dim, width], dbias [dim] fp32; dwindow, the gradient of the incoming
    window (None without one)."""
    return _calls.s6_causal_conv_grad(x, w, bias, dy, window, dwindow, lengths, silu, workspace)


def s6_conv_step(x, w, bias, window, slot_in=None, slot_out=None, silu=True, out=None):
    """One token of s6_causal_conv for each row: x [batch, dim] (any row
    stride); window, the pool [slots, dim, width-1] in x's dtype, is read at
    slot_in[b] and written at slot_out[b] (int32 [batch], None: slot b). A row
    whose slot is outside the pool is empty: y is zero there and no state
    changes. Rows may read one slot together (a fork); no slot that a row
    writes may be read or written by another row. Returns y [batch, dim]."""
    return _calls.s6_conv_step(x, w, bias, window, slot_in, slot_out, silu, out)


# -------------------------------------------------------------------- scan
def s6_causal_scan(u, delta, z, B, C, A, Dskip=None, dt_bias=None, h0=None, lengths=None, delta_softplus=True,
                   out=None, h_out=None, workspace=None):
    """Causal selective scan of prompts, gated by silu(z) (z None: no gate).

    u, delta, z [batch, dim, L]; B, C [batch, dstate, L]; A [dim, dstate],
    Dskip, dt_bias [dim] fp32; h0 [batch, dim, dstate] fp32, the state before
    token 0 (None: zeros). Returns (y, h): y [batch, dim, L] and the state
    after each row's last token.
    """
    return _calls.s6_causal_scan(u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, delta_softplus, out, h_out, workspace)


def s6_causal_scan_saved(u, delta, z, B, C, A, Dskip=None, dt_bias=None, h0=None, lengths=None, delta_softplus=True,
                         out=None, h_out=None, saved=None, workspace=None):
    """s6_causal_scan for training: returns (y, h, saved); saved is the opaque
    buffer that s6_causal_scan_grad reads instead of running the scan again."""
    return _calls.s6_causal_scan_saved(u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, delta_softplus, out, h_out, workspace,
                                       saved)


def s6_causal_scan_grad(u, delta, z, B, C, A, Dskip, dt_bias, saved, dy, dh=None, h0=None, lengths=None,
                        delta_softplus=True, workspace=None):
    """Gradient of s6_causal_scan for dy = dL/dy and dh = dL/dh (or None),
    from the saved buffer of s6_causal_scan_saved on the same inputs. Returns a
    dict: du, ddelta, dz (None without z) [batch, dim, L] in the input dtype;
    dB, dC [batch, dstate, L], dA [dim, dstate], dD, ddt_bias [dim] and dh0
    [batch, dim, dstate] (None without h0) in fp32."""
    return _calls.s6_causal_scan_grad(u, delta, z, B, C, A, Dskip, dt_bias, saved, dy, dh, h0, lengths, delta_softplus, workspace)


def s6_scan_step(u, delta, z, B, C, A, Dskip, dt_bias, h, slot_in=None, slot_out=None, delta_softplus=True, out=None):
    """One token of s6_causal_scan for each row: u, delta, z [batch, dim], B, C
    [batch, dstate] (any row strides); h, the pool [slots, dim, dstate] fp32,
    is read at slot_in[b] and written at slot_out[b], as in s6_conv_step.
    Returns y [batch, dim]."""
    return _calls.s6_scan_step(u, delta, z, B, C, A, Dskip, dt_bias, h, slot_in, slot_out, delta_softplus, out)


# ---------------------------------------------------------------- autograd
def _rows(g, like):
    """An incoming gradient in the dtype of the activation, contiguous along its last axis."""
    if g is None:
        return None
    g = g.to(like.dtype)
    return g if g.stride(-1) == 1 and min(g.stride()) >= 0 else g.contiguous()


class CapturableFunction(torch.autograd.Function):
    """A call that may be captured in a HIP graph together with its backward
    pass: while capturing and recording gradients it refuses inputs that an eager
    graph leads to, or that were made of a leaf of one, while that graph is alive."""

    @classmethod
    def apply(cls, *args):
        _calls.capture_ready(args)
        return super().apply(*args)


class CausalConvFunction(CapturableFunction):
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


class CausalScanFunction(CapturableFunction):
    """s6_causal_scan for autograd: the forward keeps the saved buffer for the
    backward; y and h are differentiable, once: a gradient of the gradient is
    refused. The gradients of B and C come back in their dtype (the library sums
    them in fp32)."""

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
