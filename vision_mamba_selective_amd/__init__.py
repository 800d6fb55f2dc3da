"""MI355X (gfx950) selective scan for Vision Mamba and VMamba, and the causal
form of it that a language model needs, with beam search over its states.

The scan itself lives in libvimscan.so (HIP kernels behind a C ABI,
include/vimscan.h). This package holds the in-tree build step, the binding
with the same entry-point names (ctypes; a compiled one for the causal mixer
and beam search), and the seeded workload generator.
The binding is imported lazily so that the generator can be used without the
library.
"""

__all__ = ["vim_scan_bidir", "vim_scan_bidir_noalloc", "vim_scan_bidir_chunked", "vim_scan_bidir_dirs", "vim_scan_bidir_conv", "vim_scan_bidir_grad",
           "vim_scan_bidir_fwd_saved", "vim_scan_bidir_grad_saved",
           "VimScanFunction", "vim_scan_bidir_autograd",
           "vmamba_cross_scan4", "s6_scan_1d", "workspace_bytes", "vim_x_proj", "vim_dt_proj",
           "vim_out_proj"]
_CAUSAL = ["s6_workspace_bytes", "s6_causal_conv", "s6_causal_conv_grad", "s6_conv_step",
           "s6_causal_scan", "s6_causal_scan_saved", "s6_causal_scan_grad", "s6_scan_step",
           "CausalConvFunction", "s6_causal_conv_autograd", "CausalScanFunction",
           "s6_causal_scan_autograd"]
_BEAM = ["beam_select", "beam_reorder", "beam_workspace_bytes"]
__all__ += _CAUSAL + _BEAM


def __getattr__(name):
    if name in _CAUSAL:
        from . import causal as module
    elif name in _BEAM:
        from . import beam as module
    elif name in __all__:
        from . import scan as module
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(module, name)     # the next use finds it here
    return value
