"""Workspaces of exactly the size that the library names: what stands behind
them keeps its bytes, at sizes on both sides of every part and piece."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


def guarded(n):
    """(a workspace of n bytes, the bytes behind it)"""
    whole = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole[:n], whole[n:]


def intact(guard):
    return bool((guard == 0xA5).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("beams", [1, 5, 8, 16, 32])
def test_select(beams, dtype):
    import vision_mamba_selective_amd as vms
    for vocab in (1, 31, 2048, 4096, 4097, 8191, 8192, 8193, 16384, 16385, 49999):
        say("case select workspace %d %d %s" % (beams, vocab, dtype))
        x, s = torch.randn(3, beams, vocab, device="cuda").to(dtype), torch.randn(3, beams, device="cuda")
        ws, guard = guarded(vms.beam_workspace_bytes(3, beams, vocab))
        got = vms.beam_select(x, s, workspace=ws)
        assert intact(guard)
        assert all(torch.equal(a, b) for a, b in zip(got, vms.beam_select(x, s)))


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 37, 301, 5), (1, 20, 2100, 16), (12, 192, 1500, 8), (3, 65, 1000, 16)],
                         ids=lambda s: "b%d-d%d-L%d-N%d" % s)
def test_mixer(shape):
    import vision_mamba_selective_amd as vms
    from vision_mamba_selective_amd import _native as nat
    batch, dim, L, N = shape
    say("case mixer workspaces %s" % (shape,))
    rnd = lambda *s: torch.randn(*s, device="cuda")      # noqa: E731
    u, B, C, A, w = rnd(batch, dim, L), rnd(batch, N, L), rnd(batch, N, L), -rnd(dim, N).abs(), rnd(dim, 4)
    buf = {op: guarded(vms.s6_workspace_bytes(op, batch, dim, inner, L)) for op, inner in
           ((nat.VS_S6_SCAN, N), (nat.VS_S6_SAVED, N), (nat.VS_S6_GRAD, N), (nat.VS_S6_CONV_GRAD, 4))}
    ws = {op: b[0] for op, b in buf.items()}
    vms.s6_causal_scan(u, u, u, B, C, A, workspace=ws[nat.VS_S6_SCAN])
    vms.s6_causal_scan_saved(u, u, u, B, C, A, saved=ws[nat.VS_S6_SAVED], workspace=ws[nat.VS_S6_SCAN])
    vms.s6_causal_scan_grad(u, u, u, B, C, A, None, None, ws[nat.VS_S6_SAVED], u, workspace=ws[nat.VS_S6_GRAD])
    vms.s6_causal_conv_grad(u, w, None, u, workspace=ws[nat.VS_S6_CONV_GRAD])
    for op, (_, guard) in buf.items():
        assert intact(guard), op
