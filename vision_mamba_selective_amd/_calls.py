"""The calls of the language model's operators (csrc/binding.cpp): each checks
its arguments, allocates its outputs and calls the library, in one step of the
host. The library's functions are those that _native loaded."""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch  # noqa: F401  (the module's tensor functions live in torch's libraries)

from . import _native as nat

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")


def _load(path: str = PATH):
    if not os.path.exists(path):
        raise nat.LibraryMissing(
            "_binding.so not found at %s; build it first with "
            "`python -c 'import __graft_entry__ as g; g.build()'` or "
            "`python vision_mamba_selective_amd/build.py`" % path)
    spec = importlib.util.spec_from_file_location("_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.bind({name: ctypes.cast(getattr(nat.lib, name), ctypes.c_void_p).value for name in nat.SIGNATURES}, nat.check)
    return module


_binding = _load()
s6_causal_conv = _binding.s6_causal_conv
s6_causal_conv_grad = _binding.s6_causal_conv_grad
s6_conv_step = _binding.s6_conv_step
s6_causal_scan = _binding.s6_causal_scan
s6_causal_scan_saved = _binding.s6_causal_scan_saved
s6_causal_scan_grad = _binding.s6_causal_scan_grad
s6_scan_step = _binding.s6_scan_step
beam_select = _binding.beam_select
beam_reorder = _binding.beam_reorder
gated_scan = _binding.gated_scan
gated_scan_saved = _binding.gated_scan_saved
gated_scan_grad = _binding.gated_scan_grad
gated_scan_step = _binding.gated_scan_step
rms_norm = _binding.rms_norm
rms_norm_grad = _binding.rms_norm_grad
vocab_loss = _binding.vocab_loss
vocab_loss_grad = _binding.vocab_loss_grad
capture_ready = _binding.capture_ready
