"""Torch-facing binding of beam search (include/vimscan.h, "Beam search over
the states above"). Nothing here is differentiable; what a call writes in place
(the state, given outputs and buffers) is treated as in causal.py."""
from __future__ import annotations

from . import _calls
from . import _native as nat


def beam_workspace_bytes(batch: int, beams: int, vocab: int) -> int:
    return int(nat.lib.beam_workspace_bytes(batch, beams, vocab))


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
    return _calls.beam_select(logits, scores, done, eos, workspace, *((None, None, None) if out is None else out))


def beam_reorder(state, parent, out=None):
    """Move the beams' states to the beams that go on: out[l, row] =
    state[l, parent[row]].

    state [layers, batch * beams, ...], each layer's rows contiguous (layers
    may be further apart), any dtype; parent [batch, beams] int32 as
    beam_select returns it. out: None or state itself reorders in place; or
    another tensor of state's shape and strides. Returns out.
    """
    return _calls.beam_reorder(state, parent, out)
