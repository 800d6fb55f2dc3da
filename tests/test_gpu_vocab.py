"""GPU parity of the loss over a vocabulary and of its gradient with float64
references.

Bounds. A logit is a sum of dim products, exact in fp32 for bf16 inputs and off
by 2^-24 of themselves for fp32 ones; each addition rounds a partial sum, which
like a random walk stays around |x| |W_v|, by 2^-24 of it: delta = 4 x 2^-24 sqrt(dim)
max |x| |W_v| (a factor of 4 for the largest of many). The loss and lse add the
roundings of a maximum, exponentials and a logarithm: 16 more, relative to
lse and to 1. P is off by (softmax) (delta + 16 x 2^-24) |dloss|, and in bf16
rounded by 2^-8 of itself; a product adds up K of its terms, with sqrt(K) x 4 x
2^-24 of the sum of their magnitudes; its bf16 result is rounded by 2^-8 of
itself."""
import math

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import DT

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def make(seed, dtype, tokens, dim, vocab, strided, ignored=True, bits=64):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, dim + (9 if strided else 0), generator=g).to(DT[dtype]).cuda()[:, 4 if strided else 0:][:, :dim]
    W = (torch.randn(vocab, dim, generator=g) * 2 * dim ** -0.5).to(DT[dtype]).cuda()
    target = torch.randint(0, vocab, (tokens,), generator=g)
    dloss = torch.randn(tokens, generator=g)
    if ignored:
        target[::3] = torch.tensor([-100, vocab, -1, vocab + 12345])[torch.arange(len(target[::3])) % 4]
        dloss[::3] = float("nan")
    return x, W, target.to(torch.int64 if bits == 64 else torch.int32).cuda(), dloss.cuda()


def bounds(x, W, target, dloss, loss_only=False):
    """Reference results and their bounds, on x's device."""
    kept = (target >= 0) & (target < W.shape[0])
    xd, Wd = x.double(), W.double()
    tokens, dim = x.shape
    delta = 4 * E * math.sqrt(dim) * float(xd.norm(dim=1).max()) * float(Wd.norm(dim=1).max())
    loss, lse = ref.vocab(xd, Wd, target)
    out = dict(loss=(loss, 2 * delta + 16 * E * (1 + lse.abs())), lse=(lse, delta + 16 * E * (1 + lse.abs())))
    if loss_only:
        return out
    g = torch.where(kept, dloss.double(), 0.0)
    p = torch.exp(xd @ Wd.T - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, torch.where(kept, target, 0).long()[:, None], 1.0)
    mag = (p + hot) * g.abs()[:, None]
    P = (p - hot) * g[:, None]
    xz = torch.where(kept[:, None], xd, 0.0)
    step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    rel = step + delta + 16 * E
    dx, dW = P @ Wd, P.T @ xz
    out["dx"] = dx, (rel + 4 * E * math.sqrt(W.shape[0])) * (mag @ Wd.abs()) + step * dx.abs()
    out["dW"] = dW, (rel + 4 * E * math.sqrt(tokens)) * (mag.T @ xz.abs()) + step * dW.abs()
    return out


def check(x, W, target, dloss, reference=None):
    import vision_mamba_selective_amd as vms
    loss, lse = vms.vocab_loss(x, W, target)
    g = vms.vocab_loss_grad(x, W, target, lse, dloss)
    again = vms.vocab_loss_grad(x, W, target, vms.vocab_loss(x, W, target)[1], dloss)
    want = reference or bounds(*(v.cpu() for v in (x, W, target, dloss)))
    for name, got in (("loss", loss), ("lse", lse), ("dx", g["dx"]), ("dW", g["dW"])):
        w, tol = want[name]
        d = got.to(w.device, torch.float64)
        assert d.shape == w.shape and bool(torch.isfinite(d).all()), name
        worst = ((d - w).abs() / (tol + 1e-300)).max()
        assert float(worst) <= 1, (name, float(worst))
    kept = (target >= 0) & (target < W.shape[0])
    assert float(loss[~kept].abs().sum()) == 0 and float(g["dx"][~kept].float().abs().sum()) == 0
    assert torch.equal(g["dx"], again["dx"]) and torch.equal(g["dW"], again["dW"])


# tokens, dim, vocab, strided: one token and entry, odd rows (packed), tails of a
# stage and of a tile, splits of both products, the larger tile
CASES = [
    (1, 1, 1, False), (1, 24, 100, False), (3, 8, 2, True), (5, 7, 33, False), (2, 63, 500, True), (33, 65, 129, False),
    (127, 64, 128, False), (128, 66, 127, True), (129, 100, 257, False), (197, 384, 1000, False), (300, 30, 2500, True),
    (1000, 130, 40, False), (40, 1536, 3001, False), (2100, 33, 700, False), (1030, 40, 12500, False), (3200, 12, 4100, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=["t%d-d%d-v%d%s" % (c[0], c[1], c[2], "-strided" if c[3] else "") for c in CASES])
def test_loss_and_gradient(case, dtype):
    say("case vocab %s %s" % (case, dtype))
    check(*make(sum(case[:3]), dtype, *case, bits=32 if case[0] % 2 else 64))


@pytest.mark.parametrize("dtype,tokens,dim,vocab", [("bf16", 5003, 136, 58001), ("f32", 2501, 68, 55003),
                                                    ("bf16", 3, 8, 9000001), ("f32", 2, 5, 4300001)])
def test_pieces_of_the_vocabulary(dtype, tokens, dim, vocab):
    """Logits of more than 512 MB, or rows of them of more than 16 MB: the
    gradient takes the vocabulary in pieces. The reference runs in float64 on the GPU."""
    import vision_mamba_selective_amd as vms
    say("case vocab pieces %s" % dtype)
    x, W, target, dloss = make(4, dtype, tokens, dim, vocab, False)
    assert vms.vocab_workspace_bytes(1, tokens, dim, vocab, x.dtype) < tokens * vocab * x.element_size()
    check(x, W, target, dloss, bounds(x, W, target, dloss))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_that_are_left_out_may_hold_anything(dtype):
    import vision_mamba_selective_amd as vms
    say("case vocab left out %s" % dtype)
    x, W, target, dloss = make(3, dtype, 300, 72, 900, False)
    loss, lse = vms.vocab_loss(x, W, target)
    g = vms.vocab_loss_grad(x, W, target, lse, dloss)
    bad = x.clone()
    bad[::3] = torch.tensor([math.nan, math.inf, -math.inf], dtype=x.dtype).cuda()[torch.arange(100) % 3][:, None]
    loss2, lse2 = vms.vocab_loss(bad, W, target)
    g2 = vms.vocab_loss_grad(bad, W, target, lse2, dloss)
    kept = (target >= 0) & (target < 900)
    assert torch.equal(loss, loss2) and torch.equal(lse[kept], lse2[kept])
    assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dW"], g2["dW"])
    none = torch.full_like(target, -100)
    loss, lse = vms.vocab_loss(bad, W, none)
    g = vms.vocab_loss_grad(bad, W, none, lse, dloss)
    assert float(loss.abs().sum()) == 0 and float(g["dx"].float().abs().sum()) == 0 and float(g["dW"].float().abs().sum()) == 0


def test_extreme_logits():
    """Logits of +-1e4 (only their differences count), a row of equal ones, a
    head with rows of -inf products that no token may choose, and a NaN token
    that touches no other."""
    import vision_mamba_selective_amd as vms
    say("case vocab extreme")
    x, W, target, dloss = make(11, "f32", 140, 16, 400, False, ignored=False)
    x[:, 0] = 1
    W[:, 0] = 0
    W[::2, 0] = 1e4
    W[1::2, 0] = -1e4
    target = target // 2 * 2
    x[5] = 0
    check(x, W, target, dloss)
    loss, lse = vms.vocab_loss(x, W, target)
    assert abs(float(lse[5]) - math.log(400)) < 1e-6
    out = W.clone()
    out[7, 0] = -math.inf
    x1 = x.abs()
    W1 = out.clone()
    W1[7, 1:] = 0
    a, _ = vms.vocab_loss(x1[6:], W1, target[6:])
    W1[7, 0] = -3e4
    b, _ = vms.vocab_loss(x1[6:], W1, target[6:])
    assert torch.equal(a, b)
    bad = x.clone()
    bad[9, 3] = math.nan
    l2, e2 = vms.vocab_loss(bad, W, target)
    others = torch.arange(140, device="cuda") != 9
    assert bool(l2[9].isnan()) and bool(e2[9].isnan()) and torch.equal(l2[others], loss[others])
    g, g2 = (vms.vocab_loss_grad(v, W, target, e, dloss) for v, e in ((x, lse), (bad, e2)))
    assert bool(g2["dx"][9].isnan().all()) and torch.equal(g2["dx"][others], g["dx"][others])


def test_gradient_against_differences():
    """Central differences of the mean loss along one direction, step 2^-6: each
    loss is off by under 1e-6, which over 2^-5 is 4e-5; the third derivative adds
    2^-12 / 6 times a few units."""
    import vision_mamba_selective_amd as vms
    say("case vocab differences")
    x, W, target, _ = make(17, "f32", 60, 40, 300, False)
    kept = (target >= 0) & (target < 300)
    g = torch.Generator().manual_seed(1)
    wx, wW = torch.randn(60, 40, generator=g).cuda() / 6, torch.randn(300, 40, generator=g).cuda() / 6

    def mean(e):
        return float(vms.vocab_loss(x + e * wx, W + e * wW, target)[0].double().sum() / kept.sum())
    _, lse = vms.vocab_loss(x, W, target)
    d = vms.vocab_loss_grad(x, W, target, lse, torch.ones(60).cuda() / kept.sum())
    along = float((d["dx"].double() * wx).sum() + (d["dW"].double() * wW).sum())
    e = 2.0 ** -6
    assert abs((mean(e) - mean(-e)) / (2 * e) - along) < 1e-3


def test_rows_of_any_stride():
    """One row for all tokens, overlapping rows, far rows: the bits of a dense copy."""
    import vision_mamba_selective_amd as vms
    say("case vocab strides")
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.Generator().manual_seed(2)
        base = torch.randn(3000, generator=g).to(dtype).cuda()
        W = torch.randn(90, 24, generator=g).to(dtype).cuda()
        far = torch.randn(30, 70001, generator=g).to(dtype).cuda()
        target = torch.arange(30).cuda()
        for x in (base[:24].expand(30, 24), base.as_strided((30, 24), (7, 1)), base[1:].as_strided((30, 24), (25, 1)), far[:, 3:27],
                  base[:24].expand(1, 24)):
            t = target[:x.shape[0]]
            got, want = vms.vocab_loss(x, W, t), vms.vocab_loss(x.contiguous(), W, t)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            ones = torch.ones(x.shape[0]).cuda()
            a, b = (vms.vocab_loss_grad(v, W, t, want[1], ones) for v in (x, x.contiguous()))
            assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dW"], b["dW"])


def test_autograd_matches_the_calls():
    import vision_mamba_selective_amd as vms
    say("case vocab autograd")
    x, W, target, _ = make(8, "bf16", 70, 48, 333, False)
    kept = int(((target >= 0) & (target < 333)).sum())
    lx, lW = x.clone().requires_grad_(), W.clone().requires_grad_()
    loss = vms.vocab_loss_autograd(lx, lW, target)
    (loss.sum() / kept).backward()
    want, lse = vms.vocab_loss(x, W, target)
    g = vms.vocab_loss_grad(x, W, target, lse, torch.full((70,), 1.0 / kept).cuda())
    assert torch.equal(loss, want) and torch.equal(lx.grad, g["dx"]) and torch.equal(lW.grad, g["dW"])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(vms.vocab_loss_autograd(lx, lW, target).sum(), lx, create_graph=True)[0].float().sum(), lW)
