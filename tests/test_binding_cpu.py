"""The compiled calls behind the causal mixer's and beam search's Python
functions: what they refuse without a GPU, and how a missing module is
reported."""
import pytest
import torch

from vision_mamba_selective_amd import _calls
from vision_mamba_selective_amd import _native as nat
import vision_mamba_selective_amd as vms

ENTRIES = [("s6_causal_conv", 8), ("s6_causal_conv_grad", 9), ("s6_conv_step", 8), ("s6_causal_scan", 14), ("s6_causal_scan_saved", 15),
           ("s6_causal_scan_grad", 15), ("s6_scan_step", 13), ("beam_select", 8), ("beam_reorder", 3)]


@pytest.mark.parametrize("name,n", ENTRIES, ids=[e[0] for e in ENTRIES])
def test_arguments(name, n):
    call = getattr(_calls, name)
    for count in (0, n - 1, n + 1):
        with pytest.raises(TypeError, match="expected %d arguments" % n):
            call(*[None] * count)
    with pytest.raises(ValueError, match="is required"):
        call(*[None] * n)
    with pytest.raises(TypeError, match="must be a tensor"):
        call(*[3] * n)
    with pytest.raises((TypeError, ValueError)):
        call(*[torch.zeros(2, 3, 4)] * n)                     # not on the GPU
    with pytest.raises((TypeError, ValueError)):
        call(*[torch.zeros(2, 3, 4, dtype=torch.float64)] * n)


def test_first_argument_decides():
    x = torch.zeros(2, 3, 4)
    with pytest.raises(TypeError, match="torch.float16"):
        vms.s6_causal_conv(x.half(), x[0, :, :2])
    with pytest.raises(ValueError, match="3 axes"):
        vms.s6_causal_conv(x[0], x[0, :, :2])
    with pytest.raises(ValueError, match="GPU"):
        vms.s6_causal_conv(x, x[0, :, :2])


def test_missing_module_is_reported():
    with pytest.raises(nat.LibraryMissing, match="build"):
        _calls._load("/nonexistent/_binding.so")


def test_bind_wants_every_function():
    with pytest.raises(ValueError, match="no address"):
        _calls._binding.bind({}, nat.check)
    # a failed bind leaves the functions as they were
    assert nat.lib.s6_workspace_bytes(nat.VS_S6_SAVED, 1, 8, 16, 33) > 0
