"""The compiled binding on the GPU: which library functions it calls, and on
which device."""
import ctypes

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


def test_a_failed_bind_changes_nothing():
    """A table that lacks only its last name, with other functions before it:
    the calls go on to the library. The other functions launch nothing."""
    from vision_mamba_selective_amd import _calls
    from vision_mamba_selective_amd import _native as nat
    import vision_mamba_selective_amd as vms
    say("case failed bind")
    x, scores = torch.randn(2, 3, 100, device="cuda"), torch.randn(2, 3, device="cuda")
    want = vms.beam_select(x, scores)
    real = {n: ctypes.cast(getattr(nat.lib, n), ctypes.c_void_p).value for n in nat.SIGNATURES}
    other = ctypes.cast(nat.lib.vs_abi_version, ctypes.c_void_p).value
    table = {n: other for n in real if n != "beam_reorder"}
    try:
        with pytest.raises(ValueError, match="no address of beam_reorder"):
            _calls._binding.bind(table, nat.check)
        got = vms.beam_select(x, scores)
    finally:
        _calls._binding.bind(real, nat.check)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
