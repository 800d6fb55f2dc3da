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


def test_reorder_refuses_layers_that_share_memory_and_empty_states():
    import vision_mamba_selective_amd as vms
    say("case reorder refusals")
    one = torch.zeros(1, 4, 8, device="cuda")
    parent = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        vms.beam_reorder(one.expand(3, 4, 8), parent)             # layer stride 0
    with pytest.raises(ValueError):
        vms.beam_reorder(one.view(-1).as_strided((2, 4, 4), (8, 4, 1)), parent)
    for shape in ((0, 4, 8), (1, 4, 0)):
        with pytest.raises(ValueError):
            vms.beam_reorder(torch.zeros(shape, device="cuda"), parent)
    with pytest.raises(ValueError):
        vms.beam_reorder(torch.zeros(1, 0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"))


def test_select_far_from_zero():
    """A constant added to a row's logits changes no probability. The logits
    are multiples of 2^-6 below 16, so that the shifted ones are exact too and
    the results equal bit for bit; n equal logits, the lowest value among them,
    have probability 1 / n each: 2^-24 of log(n) and of the sum stay."""
    import math

    import vision_mamba_selective_amd as vms
    say("case select far from zero")
    g = torch.Generator().manual_seed(9)
    x = (torch.randint(-1000, 1000, (2, 3, 9001), generator=g) / 64.0).cuda()
    scores = -torch.rand(2, 3, generator=g).cuda()
    near = vms.beam_select(x, scores)
    for shift in (4096.0, -65536.0):
        for a, b in zip(near, vms.beam_select(x + shift, scores)):
            assert torch.equal(a, b), shift
    for value in (torch.finfo(torch.float32).min, -1e30, 1e30, 0.0):
        s, p, t = vms.beam_select(torch.full((1, 2, 9001), value, device="cuda"), torch.tensor([[0.0, -1.0]], device="cuda"))
        assert t.tolist() == [[0, 1]] and p.tolist() == [[0, 0]], value
        assert (s.double() + math.log(9001)).abs().max().item() < 8 * 2.0 ** -24 * math.log(9001), (value, s)


def test_second_derivatives_are_refused():
    import vision_mamba_selective_amd as vms
    say("case second derivatives")
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    x = rnd(1, 8, 20).requires_grad_()
    y, _ = vms.s6_causal_conv_autograd(x, rnd(8, 4))
    d, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    u = rnd(1, 8, 20).requires_grad_()
    y, _ = vms.s6_causal_scan_autograd(u, rnd(1, 8, 20), None, rnd(1, 4, 20), rnd(1, 4, 20), -torch.ones(8, 4, device="cuda"))
    d, = torch.autograd.grad(y.square().sum(), u, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


@pytest.mark.parametrize("shape", [(2, 37, 301), (1, 20, 2100)], ids=["rows", "pieces"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=["inf", "nan"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_non_finite_inputs_reach_only_what_they_are_part_of(dtype, value, shape):
    """One bad entry of u or x changes its own channel from its token on, one
    of dy its own channel up to its token; of the sums over channels and tokens
    only those that hold it. Everything else keeps its bits."""
    import vision_mamba_selective_amd as vms
    batch, dim, L = shape
    say("case non-finite %s %s %s" % (shape, value, dtype))
    g = torch.Generator().manual_seed(L)
    rnd = lambda *s, d=dtype: torch.randn(*s, generator=g).to(d).cuda()   # noqa: E731
    u, x, dy, delta, z = (rnd(batch, dim, L) for _ in range(5))
    B, C = rnd(batch, 16, L), rnd(batch, 16, L)
    A = -(torch.rand(dim, 16, generator=g) + 0.1).cuda() * 4
    bias, w = (rnd(dim, d=torch.float32) - 2), rnd(dim, 4, d=torch.float32)

    def both(u, x, dy):
        y, h, saved = vms.s6_causal_scan_saved(u, delta, z, B, C, A, None, bias)
        return (dict(y=y, h=h, c=vms.s6_causal_conv(x, w)[0], dx=vms.s6_causal_conv_grad(x, w, None, dy)["dx"]),
                vms.s6_causal_scan_grad(u, delta, z, B, C, A, None, bias, saved, dy))

    def spoilt(v):
        v = v.clone()
        v[0, 5, at] = value
        return v

    at, others = 100, torch.arange(dim) != 5
    out, grad = both(u, x, dy)
    out2, grad2 = both(spoilt(u), spoilt(x), dy)
    out3, grad3 = both(u, x, spoilt(dy))
    for k in ("y", "c"):
        assert torch.equal(out[k][0, 5, :at], out2[k][0, 5, :at]), k
        assert not torch.isfinite(out2[k][0, 5, at]), k
    assert torch.equal(grad["dB"][0, :, at + 1:], grad2["dB"][0, :, at + 1:])
    assert torch.equal(grad["dC"][0, :, :at], grad2["dC"][0, :, :at])
    assert torch.equal(grad["dB"][0, :, at + 1:], grad3["dB"][0, :, at + 1:])
    assert torch.equal(out["dx"][0, 5, at + 1:], out3["dx"][0, 5, at + 1:])
    for k in ("du", "ddelta"):
        assert torch.equal(grad[k][0, 5, at + 1:], grad3[k][0, 5, at + 1:]), k
        assert not torch.isfinite(grad3[k][0, 5, at]), k
    for o, gr in ((out2, grad2), (out3, grad3)):
        for k in ("y", "h", "c", "dx"):
            assert torch.equal(out[k][0, others], o[k][0, others]) and torch.equal(out[k][1:], o[k][1:]), k
        for k in ("du", "ddelta", "dz"):
            assert torch.equal(grad[k][0, others], gr[k][0, others]) and torch.equal(grad[k][1:], gr[k][1:]), k
        for k in ("dA", "ddt_bias"):
            assert torch.equal(grad[k][others], gr[k][others]), k
        for k in ("dB", "dC"):
            assert torch.equal(grad[k][1:], gr[k][1:]), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("beams", [1, 4, 8, 16, 20, 32])
def test_select_around_the_sizes_of_a_part(beams, dtype):
    """Vocabularies on both sides of one, two, four and eight thousand entries
    and of what one wave joins: the scores against a float64 log-softmax (the
    bound of test_gpu_beam.py) and, exactly, the logits of the chosen tokens in
    order; equal logits by the lowest token."""
    import vision_mamba_selective_amd as vms
    g = torch.Generator().manual_seed(beams)
    for vocab in (2047, 2048, 2049, 4096, 4097, 8192, 8193, 16385, 32769, 65537):
        say("case select part %d %d %s" % (beams, vocab, dtype))
        x = (torch.randn(1, beams, vocab, generator=g) * 3).to(dtype)
        x[0, 0, ::7] = x[0, 0, 0]                             # many equal ones, some masked
        x[0, 0, 5::11] = float("-inf")
        x[0, -1, vocab - 1] = 40.0
        scores = torch.zeros(1, beams)
        scores[0, 1:] = -1e4                                   # the first beam's alone, then the last one's
        for first in (0, beams - 1):
            sc = scores.roll(first, 1)
            s, p, t = (v.cpu() for v in vms.beam_select(x.cuda(), sc.cuda()))
            order = torch.sort(x[0, first].double(), descending=True, stable=True).indices[:beams]
            assert p.tolist() == [[first] * beams] and torch.equal(t[0].long(), order), (vocab, first)
            want = torch.log_softmax(x[0, first].double(), 0)[order]
            assert ((s[0].double() - want).abs() <= 32 * 2.0 ** -24 * (21 + want.abs())).all(), (vocab, first)
