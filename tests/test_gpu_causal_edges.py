"""Edges of the causal mixer's and beam search's bindings: inputs that share
one row of memory, empty sizes, and logits far from zero.
"""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


def test_step_of_one_row_for_all():
    """x expanded over the batch (row stride 0): the same bits as its copy."""
    import vision_mamba_selective_amd as vms
    say("case expanded step")
    g = torch.Generator().manual_seed(5)
    x, w, bias = torch.randn(1, 40, generator=g).cuda(), torch.randn(40, 4, generator=g).cuda(), torch.randn(40, generator=g).cuda()
    pool = torch.randn(6, 40, 3, generator=g).cuda()
    one, two = pool.clone(), pool.clone()
    y = vms.s6_conv_step(x.expand(6, 40), w, bias, one)
    assert torch.equal(y, vms.s6_conv_step(x.repeat(6, 1), w, bias, two))
    assert torch.equal(one, two)
    u, d = torch.randn(1, 40, generator=g).cuda(), torch.randn(1, 40, generator=g).cuda()
    B, C = torch.randn(1, 8, generator=g).cuda(), torch.randn(1, 8, generator=g).cuda()
    A = -torch.rand(40, 8, generator=g).cuda() - 0.1
    h = torch.randn(6, 40, 8, generator=g).cuda()
    one, two = h.clone(), h.clone()
    all_ = lambda v: v.expand(6, v.shape[1])   # noqa: E731
    y = vms.s6_scan_step(all_(u), all_(d), None, all_(B), all_(C), A, None, None, one)
    assert torch.equal(y, vms.s6_scan_step(u.repeat(6, 1), d.repeat(6, 1), None, B.repeat(6, 1), C.repeat(6, 1), A, None, None, two))
    assert torch.equal(one, two)
