"""The loss over a vocabulary at the edges of its layouts and values. Bounds as in
test_gpu_vocab.py, unless a test derives its own."""
import math

import pytest
import torch

from gpu_util import say
from test_gpu_vocab import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,stride", [(25, 26), (1, 2), (63, 70)], ids=str)
def test_rows_of_odd_length_at_even_strides(dim, stride):
    """bf16 rows that end between words, the last one at the end of its memory."""
    say("case vocab odd rows %d %d" % (dim, stride))
    x, W, target, dloss = make(dim, "bf16", 133, dim, 300, False)
    memory = torch.full((132 * stride + dim,), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows = memory.as_strided((133, dim), (stride, 1))
    rows.copy_(x)
    check(rows, W, target, dloss)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [64, 700, 40000])
@pytest.mark.parametrize("base", [64.0, -64.0, 8.0])
def test_loss_far_from_zero(base, vocab, dtype):
    """Logits around +-4,096 (and 64) that fp32 holds exactly: 64 x base, and steps of
    1/512 up to 1/2 added. The loss goes by their differences, so what bounds it is a
    maximum's distance (exact), an exponential, sums of positive terms and a logarithm:
    32 roundings of 2^-24, relative to 1 + the loss. lse itself is rounded at
    its size."""
    import vision_mamba_selective_amd as vms
    say("case vocab far from zero %s %d %s" % (base, vocab, dtype))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(vocab)
    tokens = 200
    x = torch.zeros(tokens, 8)
    x[:, 0], x[:, 3] = 64, 2.0 ** torch.randint(-1, 2, (tokens,), generator=g)
    W = torch.zeros(vocab, 8)
    W[:, 0], W[:, 3] = base, torch.randint(0, 128, (vocab,), generator=g) / 256.0
    target = torch.randint(0, vocab, (tokens,), generator=g)
    loss, lse = vms.vocab_loss(x.to(dt).cuda(), W.to(dt).cuda(), target.cuda())
    l = x.double() @ W.double().T
    assert torch.equal(l, l.float().double()) and torch.equal(x, x.to(dt).float()) and torch.equal(W, W.to(dt).float())
    ref = torch.logsumexp(l, dim=1)
    want = torch.logsumexp(l - l.gather(1, target[:, None]), dim=1)
    assert bool(((loss.cpu().double() - want).abs() <= 32 * 2.0 ** -24 * (1 + want)).all()), float((loss.cpu().double() - want).abs().max())
    assert bool(((lse.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 32 * 2.0 ** -24 * (1 + want)).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [8, 131])
def test_gradient_far_from_zero(dim, dtype):
    """Logits of up to 7,936, of which one is 2,112 or more above the others: lse is that
    one, exactly, its entry of P is 0 or dloss and the target's 0 or -dloss. An
    exponential of zero and the products: 8 roundings of 2^-24 and those of a sum (bf16
    adds P's and the result's). What rounding lse log2(e) takes off the exponent would be 3e-4 here."""
    import vision_mamba_selective_amd as vms
    say("case vocab gradient far from zero %d %s" % (dim, dtype))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    tokens, vocab = 150, 300
    g = torch.Generator().manual_seed(dim)
    x = torch.zeros(tokens, dim)
    x[:, 0] = torch.arange(tokens) % 30 + 33.0
    W = torch.randn(vocab, dim, generator=g).to(dt).float()
    W[:, 0] = 64.0
    W[7, 0] = 128.0
    target = torch.where(torch.arange(tokens) % 3 == 0, torch.arange(tokens) + 8, torch.tensor(7))
    dloss = torch.randn(tokens, generator=g)
    x, W, target, dloss = x.to(dt).cuda(), W.to(dt).cuda(), target.cuda(), dloss.cuda()
    _, lse = vms.vocab_loss(x, W, target)
    assert torch.equal(lse, 128.0 * x[:, 0].float())
    got = vms.vocab_loss_grad(x, W, target, lse, dloss)
    P, size = (torch.zeros(tokens, vocab, dtype=torch.float64, device="cuda") for _ in range(2))
    rows = torch.arange(tokens, device="cuda")
    P[:, 7] += dloss
    P[rows, target] -= dloss
    size[:, 7] = size[rows, target] = dloss.abs().double()
    E = 2.0 ** -24
    half = 2.0 ** -8 if dtype == "bf16" else 0.0              # P's rounding, and the result's
    for name, want, big in (("dx", P @ W.double(), size @ W.double().abs()), ("dW", P.T @ x.double(), size.T @ x.double().abs())):
        exact = P.abs() @ W.double().abs() if name == "dx" else P.abs().T @ x.double().abs()
        tol = (8 + 4 * math.sqrt(tokens)) * E * big + half * (exact + want.abs())
        off = (got[name].double() - want).abs()
        assert bool((off <= tol).all()), (name, float((off / (tol + 1e-300)).max()))


# one tile, a product cut into parts, pieces of the vocabulary
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,dim,vocab", [(300, 72, 900), (40, 300, 30001), (3, 8, 9000001)], ids=str)
def test_left_out_tokens_have_zero_gradients_whatever_the_head_holds(tokens, dim, vocab, dtype):
    """Entries of the head with a -inf (no token's logit there is above -inf) or a NaN
    and a +inf: the left-out tokens' loss and dx are zero all the same. With the -inf, dW
    of every other entry keeps its bits: that entry's part of P is zero."""
    import vision_mamba_selective_amd as vms
    say("case vocab left out, head %s %s" % ((tokens, dim, vocab), dtype))
    x, W, target, dloss = make(5, dtype, tokens, dim, vocab, False)
    x = x.abs()
    left = (target < 0) | (target >= vocab)
    bad = vocab // 2
    target = torch.where(target == bad, bad + 1, target)
    W[bad] = 0
    W[bad, 0] = -1e30
    _, lse = vms.vocab_loss(x, W, target)
    clean = vms.vocab_loss_grad(x, W, target, lse, dloss)
    W[bad, 0] = -math.inf
    loss, lse2 = vms.vocab_loss(x, W, target)
    got = vms.vocab_loss_grad(x, W, target, lse2, dloss)
    assert torch.equal(lse, lse2) and float(loss[left].abs().sum()) == 0
    assert float(got["dx"][left].float().abs().sum()) == 0
    same = torch.arange(vocab, device="cuda") != bad
    assert torch.equal(got["dW"][same], clean["dW"][same]) and float(got["dW"][bad].float().abs().sum()) == 0
    W[bad, 0], W[bad, dim - 1] = math.nan, math.inf
    loss, lse2 = vms.vocab_loss(x, W, target)
    got = vms.vocab_loss_grad(x, W, target, lse2, dloss)
    assert float(loss[left].abs().sum()) == 0 and float(got["dx"][left].float().abs().sum()) == 0


def tight(x, W, target, dloss):
    """dx and dW in float64 with the bounds of test_gpu_vocab.py, but of the target's entry of
    P only what its two parts in bf16 leave: 2^-16 of itself (each is off by at most 2^-8
    of what it stands for)."""
    kept = (target >= 0) & (target < W.shape[0])
    E, xd, Wd = 2.0 ** -24, torch.where(kept[:, None], x, 0).double(), W.double()
    l = xd @ Wd.T
    g = torch.where(kept, dloss.double(), 0.0)[:, None]
    p = torch.softmax(l, dim=1)
    hot = torch.zeros_like(p).scatter_(1, torch.where(kept, target, 0).long()[:, None], 1.0)
    P = (p - hot) * g
    delta = 4 * E * math.sqrt(x.shape[1]) * float(xd.norm(dim=1).max()) * float(Wd.norm(dim=1).max()) + 16 * E
    off = torch.where(hot > 0, 2.0 ** -16 * P.abs(), 2.0 ** -8 * P.abs()) + delta * p * g.abs()
    mag, out = (p + hot) * g.abs(), {}
    for name, left, right, size, terms in (("dx", P, Wd, (off, mag), W.shape[0]), ("dW", P.T, xd, (off.T, mag.T), x.shape[0])):
        want = left @ right
        out[name] = want, size[0] @ right.abs() + (16 + 4 * math.sqrt(terms)) * E * (size[1] @ right.abs()) + 2.0 ** -8 * want.abs()
    return out


# tokens, dim, vocab, distinct targets (0: any): few and many tokens for a tile of dW, both tile sizes, tails, products cut
# into parts, rows of odd length, one target for all (more than a pass's list), pieces of the vocabulary
@pytest.mark.parametrize("tokens,dim,vocab,targets", [
    (1, 1, 1, 0), (5, 7, 33, 0), (129, 100, 257, 0), (300, 30, 2500, 0), (1000, 130, 40, 0), (2100, 33, 700, 1), (40, 1536, 3001, 0),
    (9000, 24, 5000, 1), (9000, 264, 5000, 3), (4097, 520, 9000, 0), (3, 8, 9000001, 2), (5003, 136, 58001, 0), (20000, 8, 300, 2)], ids=str)
def test_rounding_of_the_targets_entries(tokens, dim, vocab, targets):
    import vision_mamba_selective_amd as vms
    say("case vocab targets' entries %s" % ((tokens, dim, vocab, targets),))
    x, W, target, dloss = make(7, "bf16", tokens, dim, vocab, False, bits=32 if tokens % 2 else 64)
    W = (W.float() / 4).bfloat16()                             # other entries stay small
    if targets:
        kept = (target >= 0) & (target < vocab)
        target = torch.where(kept, (target % targets) * (vocab // 2) % vocab, target)
    _, lse = vms.vocab_loss(x, W, target)
    got = vms.vocab_loss_grad(x, W, target, lse, dloss)
    again = vms.vocab_loss_grad(x, W, target, lse, dloss)
    for name, (want, tol) in tight(x, W, target, dloss).items():
        off = (got[name].double() - want).abs() / (tol + 1e-300)
        assert bool(torch.isfinite(off).all()) and float(off.max()) <= 1, (name, float(off.max()))
        assert torch.equal(got[name], again[name])


def test_bf16_gradients_are_as_good_as_their_last_rounding():
    """With the softmax spread over 5,000 entries the root of its squares' sum is about
    0.1, so that rounding its entries adds less than 1 % (in squares) to the
    results' own rounding; the target's entry, rounded once, would add as much as that."""
    import vision_mamba_selective_amd as vms
    say("case vocab bf16 gradients")
    x, W, target, _ = make(12, "bf16", 1500, 256, 5000, False)
    dloss = 0.5 + torch.rand(1500, generator=torch.Generator().manual_seed(3)).cuda()
    _, lse = vms.vocab_loss(x, W, target)
    got = vms.vocab_loss_grad(x, W, target, lse, dloss)
    for name, (want, _) in tight(x, W, target, dloss).items():
        least = float((want.bfloat16().double() - want).norm())
        assert float((got[name].double() - want).norm()) <= 1.05 * least, (name, float((got[name].double() - want).norm()) / least)
