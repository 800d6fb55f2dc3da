"""Torch-facing binding of the gated linear recurrence (include/vimscan.h, "The
gated linear recurrence"): over prompts, for training and for single tokens on
a pool of states. Layouts, strides, lengths, tensors written in place, what is
differentiable (gated_scan_autograd only) and what may be captured are as in
causal.py."""
from __future__ import annotations

from torch.autograd.function import once_differentiable

from . import _calls
from . import _native as nat
from .causal import CapturableFunction, _rows


def gated_workspace_bytes(op: int, batch: int, dim: int, seqlen: int) -> int:
    """Bytes of a buffer of these entry points (op: VS_GATED_SAVED or VS_GATED_GRAD)."""
    return int(nat.lib.gated_workspace_bytes(op, batch, dim, seqlen))


def gated_scan(x, r, i, lam, z=None, h0=None, lengths=None, rate=8.0, out=None, h_out=None):
    """Gated linear recurrence of prompts: with s = rate softplus(lam)
    sigmoid(r) and a = exp(-s), h_t = a_t h_{t-1} + sqrt(1 - a_t^2)
    sigmoid(i_t) x_t, and y = h silu(z) (z None: y = h).

    x, r, i, z [batch, dim, L]; lam [dim] fp32; h0 [batch, dim] fp32, the state
    before token 0 (None: zeros). Returns (y, h): y [batch, dim, L] and the
    state after each row's last token, [batch, dim] fp32.
    """
    return _calls.gated_scan(x, r, i, lam, z, h0, lengths, rate, out, h_out)


def gated_scan_saved(x, r, i, lam, z=None, h0=None, lengths=None, rate=8.0, out=None, h_out=None, saved=None):
    """gated_scan for training: returns (y, h, saved); saved is the opaque
    buffer that gated_scan_grad starts from."""
    return _calls.gated_scan_saved(x, r, i, lam, z, h0, lengths, rate, out, h_out, saved)


def gated_scan_grad(x, r, i, lam, saved, dy, z=None, dh=None, h0=None, lengths=None, rate=8.0, workspace=None):
    """Gradient of gated_scan for dy = dL/dy and dh = dL/dh (or None), from the
    saved buffer of gated_scan_saved on the same inputs. Returns a dict: dx,
    dr, di, dz (None without z) [batch, dim, L] in the input dtype; dlam [dim]
    and dh0 [batch, dim] (None without h0) in fp32."""
    return _calls.gated_scan_grad(x, r, i, lam, saved, dy, z, dh, h0, lengths, rate, workspace)


def gated_scan_step(x, r, i, lam, h, z=None, slot_in=None, slot_out=None, rate=8.0, out=None):
    """One token of gated_scan for each row: x, r, i, z [batch, dim] (any row
    strides); h, the pool [slots, dim] fp32, is read at slot_in[b] and written
    at slot_out[b], as in s6_conv_step. Returns y [batch, dim]."""
    return _calls.gated_scan_step(x, r, i, lam, h, z, slot_in, slot_out, rate, out)


class GatedScanFunction(CapturableFunction):
    """gated_scan for autograd; y and h are differentiable, once: a gradient of
    the gradient is refused."""

    @staticmethod
    def forward(ctx, x, r, i, lam, z, h0, lengths, rate):
        y, h, saved = gated_scan_saved(x, r, i, lam, z=z, h0=h0, lengths=lengths, rate=rate)
        ctx.save_for_backward(x, r, i, lam, z, h0, lengths, saved)
        ctx.rate = rate
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, r, i, lam, z, h0, lengths, saved = ctx.saved_tensors
        dy = x.new_zeros(x.shape) if dy is None else _rows(dy, x)
        g = gated_scan_grad(x, r, i, lam, saved, dy, z=z, h0=h0, lengths=lengths, rate=ctx.rate,
                            dh=None if dh is None else dh.float().contiguous())
        return g["dx"], g["dr"], g["di"], g["dlam"], g["dz"], g["dh0"], None, None


def gated_scan_autograd(x, r, i, lam, z=None, h0=None, lengths=None, rate=8.0):
    """gated_scan as a differentiable op (GatedScanFunction). Returns (y, h)."""
    return GatedScanFunction.apply(x, r, i, lam, z, h0, lengths, rate)
