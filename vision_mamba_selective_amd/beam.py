"""Torch-facing binding of beam search (include/vimscan.h, "Beam search over
the states above")."""
from __future__ import annotations

import ctypes

import torch

from . import _native as nat
from .causal import _dense, _input, _out, _start, _stream
from .scan import _DTYPES, _ptr

_lib = nat.lib
_F32 = torch.float32


def beam_workspace_bytes(batch: int, beams: int, vocab: int) -> int:
    return int(_lib.beam_workspace_bytes(batch, beams, vocab))


def beam_select(logits, scores, done=None, eos=None, workspace=None, out=None):
    """The `beams` best continuations of each sequence.

    logits [batch, beams, vocab] (fp32 or bf16; batch and beam strides are
    free); scores [batch, beams] fp32, the beams' sums of log-probabilities;
    done [batch, beams] bool or None: a finished beam goes on with the token
    `eos` at its unchanged score. Returns (scores, parent, token), each [batch,
    beams], best first; parent is the row b * beams + k that was chosen, token
    its next token (int32). out: those three tensors, to be written in place
    of new ones.
    """
    dt, dev = _start("logits", logits, 3)
    batch, beams, vocab = logits.shape
    rows = (batch, beams)
    _input("logits", logits, (batch, beams, vocab), dt, dev)
    _dense("scores", scores, rows, _F32, dev)
    if done is not None:
        _dense("done", done, rows, torch.bool, dev)
        if eos is None:
            raise ValueError("eos is required where done is given")
    st = None
    if not logits.is_contiguous():
        st = (ctypes.c_int64 * 2)(*logits.stride()[:2])
    s, p, t = (None, None, None) if out is None else out
    s = _out("out[0]", s, rows, _F32, dev)
    p = _out("out[1]", p, rows, torch.int32, dev)
    t = _out("out[2]", t, rows, torch.int32, dev)
    need = _lib.beam_workspace_bytes(batch, beams, vocab)
    if workspace is None:
        workspace, have = torch.empty(max(need, 8), dtype=torch.uint8, device=dev), need
    else:
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError("workspace needs %d contiguous bytes on %s" % (need, dev))
    rc = _lib.beam_select(batch, beams, vocab, _DTYPES[dt], logits.data_ptr(), st, scores.data_ptr(), _ptr(done),
                          0 if eos is None else int(eos), s.data_ptr(), p.data_ptr(), t.data_ptr(), workspace.data_ptr(), have,
                          _stream(dev))
    nat.check("beam_select", rc)
    return s, p, t


def beam_reorder(state, parent, out=None):
    """Move the beams' states to the beams that go on: out[l, row] =
    state[l, parent[row]].

    state [layers, batch * beams, ...], each layer's rows contiguous (layers
    may be further apart), any dtype; parent [batch, beams] int32 as
    beam_select returns it. out: None or state itself reorders in place; or
    another tensor of state's shape and strides. Returns out.
    """
    if state.device.type != "cuda":
        raise ValueError("state must be on the GPU")
    if parent.ndim != 2 or state.ndim < 2 or state.shape[1] != parent.shape[0] * parent.shape[1]:
        raise ValueError("state must be [layers, batch * beams, ...] for a parent of [batch, beams]")
    batch, beams = parent.shape
    _dense("parent", parent, (batch, beams), torch.int32, state.device)
    layers, rows = state.shape[:2]
    if state.numel() == 0:
        raise ValueError("state is empty: %s" % (tuple(state.shape),))
    if not state[0].is_contiguous() or (layers > 1 and state.stride(0) < state[0].numel()):
        raise ValueError("each layer of state must be contiguous and apart from the others")
    es = state.element_size()
    row_bytes = state[0].numel() // rows * es
    layer_bytes = state.stride(0) * es if layers > 1 else 0
    if out is None:
        out = state
    elif out.dtype != state.dtype or out.shape != state.shape or out.stride() != state.stride() or out.device != state.device:
        raise ValueError("out must have state's dtype, shape, strides and device")
    rc = _lib.beam_reorder(layers, batch, beams, row_bytes, layer_bytes, state.data_ptr(), parent.data_ptr(), out.data_ptr(),
                           _stream(state.device))
    nat.check("beam_reorder", rc)
    return out
