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


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_calls_run_on_the_tensors_device():
    """Tensors of one device while another is the current one: the same bits."""
    import vision_mamba_selective_amd as vms
    say("case other device")
    g = torch.Generator().manual_seed(3)
    u, B, A = torch.randn(2, 20, 700, generator=g), torch.randn(2, 8, 700, generator=g), -torch.rand(20, 8, generator=g)
    x, s = torch.randn(2, 3, 9000, generator=g), torch.randn(2, 3, generator=g)

    def both(d):
        y, h = vms.s6_causal_scan(*(v.to(d) for v in (u, u, u, B, B, A)))
        return [v.cpu() for v in (y, h, *vms.beam_select(x.to(d), s.to(d)))]
    with torch.cuda.device(0):
        want = both("cuda:0")
        got = both("cuda:1")
    assert all(torch.equal(a, b) for a, b in zip(got, want))
