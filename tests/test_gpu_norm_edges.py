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


# rows, dim, tokens, strided: launches that follow one another because the workspace holds the sums of a part of the rows
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,L", [(9000, 40, 1), (3000, 520, 1), (2100, 8192, 2)], ids=str)
def test_gradient_of_many_rows_in_parts(batch, dim, L, dtype):
    """Rows whose channels lie apart (one token of longer prompts), and short
    prompts of many channels, some of them empty; the workspace is exactly of the
    stated size and shared by the launches."""
    import vision_mamba_selective_amd as vms
    say("case norm parts %s" % ((batch, dim, L),))
    g = torch.Generator(device="cuda").manual_seed(dim)
    rnd = lambda: torch.randn(batch, dim, L + (2 if L == 1 else 0), generator=g, device="cuda").to(dtype)    # noqa: E731
    s, dy, dsum = ((v[:, :, 1:2] if L == 1 else v) for v in (rnd(), rnd(), rnd()))
    w = 1 + 0.3 * torch.randn(dim, generator=g, device="cuda")
    lengths = torch.randint(0, L + 1, (batch,), generator=g, device="cuda").to(torch.int32)
    size = vms.norm_workspace_bytes(batch, dim, L)
    whole = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = vms.rms_norm_grad(s, w, dy, dsum=dsum, eps=1e-5, lengths=lengths, workspace=whole[:size])
    again = vms.rms_norm_grad(s, w, dy, dsum=dsum, eps=1e-5, lengths=lengths)
    assert bool((whole[size:] == 0xA5).all())
    assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["dw"], again["dw"])
    live = (torch.arange(L, device="cuda") < lengths[:, None])[:, None, :].double()
    sd, yd, gd = (v.double() * live for v in (s, dy, dsum))
    q = 1 / torch.sqrt(sd.square().mean(1, keepdim=True) + 1e-5)
    wy = w.double()[:, None] * yd
    want = (gd + q * wy - sd * q ** 3 * (wy * sd).mean(1, keepdim=True)) * live
    close(got["dx"], want.cpu(), "dx")
    close(got["dw"], (yd * sd * q).sum((0, 2)).cpu(), "dw")


@pytest.mark.parametrize("shape,value", [(((1 << 22) - 1, 1, 2), 1.1), ((1 << 25, 1), 1.2)], ids=["tiles", "rows"])
def test_weight_gradient_of_many_equal_terms(shape, value):
    """Where all terms of dw agree, roundings of an fp32 sum lean to one side: 65,536
    (8,192) of them one after another are off by 7e-4 (8e-5) of the sum. In steps of 64
    and in 64 bits fewer than 400 roundings of 2^-24 are left, close()'s bound."""
    import vision_mamba_selective_amd as vms
    say("case norm many equal terms %s" % (shape,))
    s = torch.ones(shape, device="cuda")
    dy = torch.full_like(s, value)
    g = vms.rms_norm_grad(s, torch.ones(1, device="cuda"), dy, eps=0.0)
    close(g["dw"], dy.flatten()[:1].cpu().double() * s.numel(), "dw")
    assert float(g["dx"].abs().max()) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("scale", [2.0 ** -62, 2.0 ** -64, 2.0 ** -66])
@pytest.mark.parametrize("shape", [(5, 64), (3, 700), (2, 64, 40), (2, 500, 37)], ids=str)
def test_tokens_whose_mean_square_is_subnormal(shape, scale):
    """Without eps tokens of 2^-66 are normed like others. Their mean square, 2^-132, has
    17 significant bits, and sums of such squares lose half a unit of 2^-149 at each
    addition: 2^-18 sqrt(channels / 64) relative, of which q has half and its cube three
    halves; close() allows 2^-15.4. The other half of the tokens is 2^3 larger, so that some
    mean squares are normal numbers."""
    import vision_mamba_selective_amd as vms
    say("case norm subnormal squares %s %g" % (shape, scale))
    g = torch.Generator().manual_seed(9)
    rnd = lambda *v: torch.randn(*v, generator=g).cuda()                              # noqa: E731
    s, dy, w = rnd(*shape) * scale, rnd(*shape), 1 + 0.3 * rnd(shape[1])
    if len(shape) == 3:
        s[:, :, ::2] *= 8
    else:
        s[::2] *= 8
    lengths = None if len(shape) == 2 else torch.tensor([shape[2], shape[2] - 5], dtype=torch.int32).cuda()
    y, _ = vms.rms_norm(s, w, eps=0.0, lengths=lengths)
    got = vms.rms_norm_grad(s, w, dy, eps=0.0, lengths=lengths)
    wide = [v.view(shape[0], shape[1], -1) for v in (s, dy)]
    leaf, lw = ref.f64(wide[0] / scale).requires_grad_(), ref.f64(w).requires_grad_()
    keep = torch.ones(shape[0], 1, 1, dtype=torch.float64)
    if lengths is not None:                                    # ones stand at padding, where the reference would divide by zero
        keep = (torch.arange(shape[2]) < lengths.cpu()[:, None])[:, None].double()
        leaf = (leaf.detach() * keep + (1 - keep)).requires_grad_()
    want = ref.norm(leaf, lw, None, None, 0.0, torch.float32)[0] * keep
    dx, dw = ref.gradients([want], [ref.f64(wide[1])], [leaf, lw])
    close(y.view_as(wide[0]), want.detach(), "y")
    close(got["dx"].view_as(wide[0]) * scale, dx, "dx")
    close(got["dw"], dw, "dw")
