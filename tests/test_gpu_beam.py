"""Beam search's selection and the reordering of states on the GPU, against a
plain sort of every candidate in float64.

Scores: a log-softmax in fp32 adds roundings of the row's log-sum (magnitude
about 10) and of the sums themselves, a few 2^-24 of their size: the bound is
32 x 2^-24 x (1 + |score| + 20). Whole numbers must be equal; the random cases
keep candidates apart by far more than that bound."""
import math

import pytest
import torch

import causal_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
INF = math.inf


def check(logits, scores, done=None, eos=None, what=""):
    import vision_mamba_selective_amd as vms
    say("case select %s %s %s" % (what, tuple(logits.shape), logits.dtype))
    s, p, t = vms.beam_select(logits, scores, done=done, eos=eos)
    rs, rp, rt = ref.select(logits.float().cpu(), scores.cpu(), None if done is None else done.cpu(), eos)
    assert torch.equal(p.cpu(), rp), (what, p, rp)
    assert torch.equal(t.cpu(), rt), (what, t, rt)
    g = s.cpu().double()
    same = torch.isinf(rs)
    assert torch.equal(g[same], rs[same]), what
    err = (g - rs)[~same].abs()
    assert (err <= 32 * 2.0 ** -24 * (21 + rs[~same].abs())).all(), (what, float(err.max()))
    assert p.dtype == torch.int32 and t.dtype == torch.int32 and s.dtype == torch.float32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 4, 1), (2, 4, 3), (3, 5, 17), (1, 8, 1000), (2, 3, 8192), (1, 2, 8193),
                                   (2, 7, 20011), (1, 32, 500), (1, 17, 9000)], ids=lambda s: "b%d-k%d-v%d" % s)
def test_random(shape, dtype):
    b, k, v = shape
    g = torch.Generator().manual_seed(sum(shape))
    logits = (torch.randn(b, k, v + 5, generator=g) * 3).to(dtype).cuda()[:, :, 2:2 + v]
    scores = (-10 * torch.rand(b, k, generator=g)).cuda()
    check(logits, scores, what="random")
    banned = torch.rand(b, k, v, generator=g).cuda() < 0.7
    logits.masked_fill_(banned, -INF)
    done = (torch.rand(b, k, generator=g) < 0.4).cuda()
    check(logits, scores, done, min(2, v - 1), what="banned and finished")


def test_ties_take_the_lowest():
    say("case ties")
    b, k, v = 2, 6, 9000
    check(torch.zeros(b, k, v).cuda(), torch.zeros(b, k).cuda(), what="all equal")
    check(torch.zeros(b, k, v).bfloat16().cuda(), torch.arange(b * k).flip(0).view(b, k).float().cuda(), what="equal rows")
    x = torch.zeros(1, 3, v)
    x[0, 1, 8999] = x[0, 1, 8192] = x[0, 1, 5] = 1.0
    x[0, 2] = -0.0
    check(x.cuda(), torch.zeros(1, 3).cuda(), what="few equal, negative zero")
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, 4, (2, 5, 12000), generator=g).float()
    check(x.bfloat16().cuda(), (-torch.arange(10.0)).view(2, 5).cuda(), what="four levels")


def test_close_logits_keep_their_order():
    """Logits that the fp32 score cannot tell apart are still ordered within a beam."""
    x = torch.zeros(1, 2, 300)
    x[0, :, 200], x[0, :, 7], x[0, :, 90] = 3e-9, 2e-9, 1e-9
    check(x.cuda(), torch.tensor([[0.0, -30.0]]).cuda(), what="close")


def test_masks_and_non_finite():
    lowest = torch.finfo(torch.float32).min
    v = 8500
    x = torch.full((1, 4, v), -INF)
    check(x.cuda(), torch.tensor([[0.0, -1.0, -2.0, -3.0]]).cuda(), what="nothing allowed")
    x[0, 2, 8400] = 1.0
    check(x.cuda(), torch.tensor([[0.0, -1.0, -2.0, -3.0]]).cuda(), what="one allowed")
    x = torch.full((1, 3, v), lowest)
    x[0, 1, 3] = 0.5
    check(x.cuda(), torch.tensor([[0.0, -1.0, -2.0]]).cuda(), what="lowest value")
    x = torch.zeros(1, 3, v)
    x[0, 0] = float("nan")
    x[0, 1, ::2] = float("nan")
    x[0, 2, [4, 8499]] = INF
    check(x.cuda(), torch.tensor([[5.0, -1.0, -2.0]]).cuda(), what="nan and inf")
    x = torch.zeros(1, 3, 10)
    check(x.cuda(), torch.tensor([[float("nan"), -INF, -2.0]]).cuda(), what="scores")
    check(x.cuda(), torch.tensor([[-INF, -INF, -INF]]).cuda(), what="first step, nothing alive")
    check(x.cuda(), torch.tensor([[0.0, -INF, -INF]]).cuda(), what="first step")


def test_finished_beams():
    x = torch.zeros(2, 4, 5)
    s = torch.tensor([[-1.0, -1.5, -2.0, -2.5]] * 2)
    done = torch.ones(2, 4, dtype=torch.bool)
    check(x.cuda(), s.cuda(), done.cuda(), 3, what="all finished")
    done[1] = torch.tensor([False, True, True, False])
    check(x.cuda(), s.cuda(), done.cuda(), 0, what="some finished")
    check(torch.zeros(1, 6, 2).cuda(), torch.tensor([[-INF] * 6]).cuda(), torch.ones(1, 6, dtype=torch.bool).cuda(), 1,
          what="finished without a score")


def test_select_repeats_and_takes_buffers():
    import vision_mamba_selective_amd as vms
    g = torch.Generator().manual_seed(9)
    logits, scores = torch.randn(3, 4, 30000, generator=g).cuda(), torch.randn(3, 4, generator=g).cuda()
    say("case select with buffers")
    a = vms.beam_select(logits, scores)
    out = tuple(torch.empty_like(x) for x in a)
    ws = torch.empty(vms.beam_workspace_bytes(3, 4, 30000), dtype=torch.uint8, device="cuda")
    b = vms.beam_select(logits, scores, out=out, workspace=ws)
    for x, y, o in zip(a, b, out):
        assert torch.equal(x, y) and y is o


# ------------------------------------------------------------- reordering
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8], ids=["f32", "bf16", "u8"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 3, 4, 7), (3, 2, 8, 300), (1, 2, 32, 64), (2, 1, 17, 1025), (4, 5, 2, 4096)],
                         ids=lambda s: "l%d-b%d-k%d-n%d" % s)
def test_reorder(shape, dtype):
    import vision_mamba_selective_amd as vms
    layers, b, k, n = shape
    g = torch.Generator().manual_seed(sum(shape))
    say("case reorder %s %s" % (shape, dtype))
    big = torch.randint(0, 250, (layers, b * k + 2, n), generator=g).to(dtype).cuda()
    for kind in ("random", "cycle", "identity"):
        if kind == "random":
            p = torch.randint(0, k, (b, k), generator=g)
        else:
            p = ((torch.arange(k) + (kind == "cycle")) % k).expand(b, k)
        rows = (p + k * torch.arange(b)[:, None]).reshape(-1)
        parent = rows.view(b, k).to(torch.int32).cuda()
        state = big.clone()[:, :b * k]                 # layers further apart than their rows
        want = state[:, rows.cuda()].clone()
        whole = torch.empty_like(big)
        whole.copy_(big)
        out = whole[:, :b * k]
        assert vms.beam_reorder(state, parent, out=out) is out
        assert torch.equal(out, want)
        assert torch.equal(whole[:, b * k:], big[:, b * k:])
        assert vms.beam_reorder(state, parent) is state
        assert torch.equal(state, want), kind


def test_reorder_strange_parents_keep_their_row():
    import vision_mamba_selective_amd as vms
    state = torch.arange(2 * 4 * 6, dtype=torch.float32, device="cuda").view(2, 4, 6)
    parent = torch.tensor([[-1, 0], [1, 99]], dtype=torch.int32, device="cuda")   # row 1 belongs to the other sequence
    say("case strange parents")
    want = state[:, [0, 0, 2, 3]].clone()
    assert torch.equal(vms.beam_reorder(state, parent), want)
