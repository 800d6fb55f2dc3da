"""The norm at the edges of its sizes and values. Bounds as in test_gpu_norm.py."""
import math

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import close

pytestmark = pytest.mark.gpu


def test_stream_in_place_of_one_channel():
    """sum_out may be the residual where there is one channel, or one row, of several tokens."""
    import vision_mamba_selective_amd as vms
    for shape in ((4, 1, 70), (1, 1, 33), (1, 5, 40), (3, 1)):
        say("case norm in place %s" % (shape,))
        g = torch.Generator().manual_seed(1)
        x, res, w = (torch.randn(*v, generator=g).cuda() for v in (shape, shape, shape[1:2]))
        y, s = vms.rms_norm(x, w, residual=res)
        stream = res.clone()
        y2, _ = vms.rms_norm(x, w, residual=stream, sum_out=stream)
        assert torch.equal(y, y2) and torch.equal(s, stream)
