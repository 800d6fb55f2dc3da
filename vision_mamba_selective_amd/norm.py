"""Torch-facing binding of the norm between the mixers (include/vimscan.h, "The
norm between the mixers"): prompts [batch, dim, L], normed over dim, and rows
[rows, dim]. Strides, lengths, tensors written in place, what is
differentiable (rms_norm_autograd only) and what may be captured are as in
causal.py."""
from __future__ import annotations

from torch.autograd.function import once_differentiable

from . import _calls
from . import _native as nat
from .causal import CapturableFunction, _rows


def norm_workspace_bytes(batch: int, dim: int, seqlen: int) -> int:
    """Bytes of rms_norm_grad's workspace (rows: seqlen 1)."""
    return int(nat.lib.norm_workspace_bytes(batch, dim, seqlen))


def rms_norm(x, w=None, residual=None, eps=1e-6, lengths=None, out=None, sum_out=None):
    """y = s / sqrt(mean(s^2) + eps) w over the channels of each token, s = x +
    residual in x's dtype.

    x, residual [batch, dim, L] or [rows, dim] (fp32 or bf16); w [dim] fp32 or
    None for ones; lengths [batch] int32 or None. Returns (y, s), both of x's
    shape; s is x itself without a residual. sum_out may be the residual: the
    stream is then updated in place.
    """
    y, s = _calls.rms_norm(x, w, residual, eps, lengths, out, sum_out)
    return y, x if residual is None else s


def rms_norm_grad(s, w, dy, dsum=None, eps=1e-6, lengths=None, workspace=None):
    """Gradient of rms_norm at its sum s, for dy = dL/dy and dsum, the gradient
    that reaches s from elsewhere (or None). Returns a dict: dx, of s's shape
    and dtype (the gradient of x and of the residual alike); dw [dim] fp32
    (None without w)."""
    return _calls.rms_norm_grad(s, w, dy, dsum, eps, lengths, workspace)


class RmsNormFunction(CapturableFunction):
    """rms_norm for autograd; y and s are differentiable, once: a gradient of
    the gradient is refused."""

    @staticmethod
    def forward(ctx, x, w, residual, eps, lengths):
        y, s = rms_norm(x, w, residual=residual, eps=eps, lengths=lengths)
        ctx.save_for_backward(s, w, lengths)
        ctx.eps, ctx.added = eps, residual is not None
        ctx.set_materialize_grads(False)
        return (y, s) if ctx.added else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, w, lengths = ctx.saved_tensors
        dy = s.new_zeros(s.shape) if dy is None else _rows(dy, s)
        g = rms_norm_grad(s, w, dy, dsum=None if ds is None else _rows(ds, s), eps=ctx.eps, lengths=lengths)
        return g["dx"], g["dw"], g["dx"] if ctx.added else None, None, None


def rms_norm_autograd(x, w=None, residual=None, eps=1e-6, lengths=None):
    """rms_norm as a differentiable op (RmsNormFunction). Returns (y, s)."""
    r = RmsNormFunction.apply(x, w, residual, eps, lengths)
    return r if residual is not None else (r, x)
