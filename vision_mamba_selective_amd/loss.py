"""Torch-facing binding of the loss over a vocabulary (include/vimscan.h, "The
loss over a vocabulary"): softmax cross entropy of a linear head, without
keeping the logits. Only vocab_loss_autograd is differentiable; what may be
captured is as in causal.py."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _calls
from . import _native as nat
from .causal import CapturableFunction


def vocab_workspace_bytes(op: int, tokens: int, dim: int, vocab: int, dtype: torch.dtype) -> int:
    """Bytes of a workspace of these entry points (op: VS_VOCAB_LOSS or VS_VOCAB_GRAD)."""
    code = {torch.float32: nat.VS_F32, torch.bfloat16: nat.VS_BF16}.get(dtype, -1)
    return int(nat.lib.vocab_workspace_bytes(op, tokens, dim, vocab, code))


def vocab_loss(x, W, target, workspace=None):
    """Cross entropy of every token under the head W: lse = logsumexp(W x),
    loss = lse - (W x)[target].

    x [tokens, dim] (fp32 or bf16, any row stride); W [vocab, dim] in the same
    dtype; target [tokens] int32 or int64: one outside the vocabulary (such as
    -100) leaves its token out, with a loss of zero. Returns (loss, lse), each
    [tokens] fp32; the mean over a batch is loss.sum() / (kept tokens).
    """
    return _calls.vocab_loss(x, W, target, workspace)


def vocab_loss_grad(x, W, target, lse, dloss, workspace=None):
    """Gradient of vocab_loss for dloss = dL/dloss [tokens] fp32, from its lse.
    Returns a dict: dx [tokens, dim] and dW [vocab, dim] in the input dtype. A
    token that is left out has no gradient and is no part of dW, whatever its x
    holds."""
    return _calls.vocab_loss_grad(x, W, target, lse, dloss, workspace)


class VocabLossFunction(CapturableFunction):
    """vocab_loss for autograd; the loss is differentiable once: a gradient of
    the gradient is refused."""

    @staticmethod
    def forward(ctx, x, W, target):
        loss, lse = vocab_loss(x, W, target)
        ctx.save_for_backward(x, W, target, lse)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, W, target, lse = ctx.saved_tensors
        g = vocab_loss_grad(x, W, target, lse, dloss.float().contiguous())
        return g["dx"], g["dW"], None


def vocab_loss_autograd(x, W, target):
    """vocab_loss as a differentiable op (VocabLossFunction). Returns the loss of every token."""
    return VocabLossFunction.apply(x, W, target)
