"""The example model with gated recurrences: it trains (its gradients are those
of the same model written with torch's own operations), and decoding from
states gives the log-probabilities of the whole-sequence forward pass."""
import importlib.util
import os

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("causal_lm", os.path.join(ROOT, "examples", "causal_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_loss(lm, p, t):
    """The model in float64 torch on the CPU, with autograd."""
    def norm(x, w):
        return x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w[:, None]
    x = p["embed"][t[:, :-1]].transpose(1, 2)
    silu = torch.nn.functional.silu
    for i in range(lm.LAYERS):
        xz = p["in%d" % i] @ norm(x, p["norm%d" % i])
        u, z = xz[:, :lm.INNER], xz[:, lm.INNER:]
        width = p["w%d" % i].shape[1]
        u = silu(torch.nn.functional.conv1d(torch.nn.functional.pad(u, (width - 1, 0)), p["w%d" % i][:, None], p["b%d" % i], groups=lm.INNER))
        r, g = (p["gates%d" % i] @ u).split(lm.INNER, dim=1)
        s = 8 * torch.nn.functional.softplus(p["lam%d" % i])[:, None] * torch.sigmoid(r)
        a, v = torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s)) * torch.sigmoid(g) * u
        h, hs = torch.zeros_like(v[:, :, 0]), []
        for k in range(v.shape[2]):
            h = a[:, :, k] * h + v[:, :, k]
            hs.append(h)
        x = x + p["out%d" % i] @ (torch.stack(hs, dim=2) * silu(z))
    logits = norm(x, p["norm%d" % lm.LAYERS]).transpose(1, 2) @ p["head"].T
    return torch.nn.functional.cross_entropy(logits.reshape(-1, lm.VOCAB), t[:, 1:].reshape(-1))


def test_gradients(lm):
    """fp32 against float64 through two layers: a few thousand roundings of
    2^-24 of the values that a weight's gradient adds up, 2^-11 of its largest."""
    import vision_mamba_selective_amd as vms
    say("case example gated gradients")
    p = lm.init(seed=2, mixer="gated")
    t = lm.progressions(6, 25, torch.Generator().manual_seed(3))
    h = lm.hidden(p, t[:, :-1]).transpose(1, 2).reshape(-1, lm.MODEL)
    loss = vms.vocab_loss_autograd(h, p["head"], t[:, 1:].reshape(-1)).mean()
    loss.backward()
    q = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    want = plain_loss(lm, q, t.cpu())
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-5
    for k in p:
        d = (p[k].grad.cpu().double() - q[k].grad).abs().max()
        assert float(d) <= 2.0 ** -11 * float(q[k].grad.abs().max()), (k, float(d))


def test_training_runs(lm):
    say("case example gated training")
    losses = lm.train(lm.init(mixer="gated"), 3)
    assert len(losses) == 3 and all(0 < v < 20 for v in losses)


@pytest.mark.parametrize("move", [False, True])
def test_beam_search_scores_are_the_sequences_log_probabilities(lm, move):
    """As for the S6 mixer: fp32 sums of 6 log-probabilities of magnitude up to
    10 through a few hundred roundings on either side: 2e-4."""
    say("case example gated beam search %s" % move)
    p = lm.init(seed=3, mixer="gated")
    t = lm.progressions(4, 16, torch.Generator().manual_seed(5))
    lengths = torch.tensor([3, 16, 1, 7], dtype=torch.int32).cuda()
    out, scores = lm.beam_search(p, t, lengths, 3, 6, move=move)
    for i in range(4):
        n = int(lengths[i])
        for k in range(3):
            seq = torch.cat([t[i, :n], out[i, k].long()])[None]
            with torch.no_grad():
                logp = torch.log_softmax(lm.forward(p, seq)[0].double(), dim=1)
            want = sum(float(logp[n - 1 + j, seq[0, n + j]]) for j in range(6))
            assert abs(float(scores[i, k]) - want) < 2e-4, (i, k, float(scores[i, k]), want)
