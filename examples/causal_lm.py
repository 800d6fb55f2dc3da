"""A small causal language model of S6 mixers (or of gated recurrences), trained
and decoded with the library's entry points for language models.

    python examples/causal_lm.py [--steps N] [--beams K] [--move] [--mixer s6|gated]

It learns arithmetic progressions modulo the vocabulary (the first two tokens
give the step), then continues prompts of different lengths by beam search:

  training   s6_causal_conv_autograd, s6_causal_scan_autograd (or
             gated_scan_autograd), rms_norm_autograd with each residual, and
             vocab_loss_autograd, which keeps no logits
  prompts    s6_causal_conv and s6_causal_scan (gated_scan) on a ragged batch,
             keeping states
  decoding   s6_conv_step and s6_scan_step (gated_scan_step) on pools of two sets of states:
             a step reads one set, at the parents that beam_select chose, and
             writes the other, so no state is moved between tokens; or, with
             --move, on one set, half the memory, which beam_reorder brings
             into the beams' order after each token

Random weights and synthetic sequences; the linear maps are torch's own.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vision_mamba_selective_amd as vms  # noqa: E402

VOCAB, MODEL, INNER, STATE, WIDTH, LAYERS = 32, 64, 128, 16, 4, 2


def init(seed=0, device="cuda", mixer="s6"):
    """The model's weights: a dict of leaf tensors. mixer: "s6", or "gated" for
    the gated recurrence, whose two gates are projections of its input."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, scale: (torch.randn(*s, generator=g) * scale).to(device).requires_grad_()   # noqa: E731
    p = dict(embed=rnd(VOCAB, MODEL, scale=0.5), head=rnd(VOCAB, MODEL, scale=MODEL ** -0.5))
    for i in range(LAYERS):
        dt = torch.exp(torch.rand(INNER, generator=g) * math.log(100.0) + math.log(1e-3))
        p["in%d" % i] = rnd(2 * INNER, MODEL, scale=MODEL ** -0.5)
        p["out%d" % i] = rnd(MODEL, INNER, scale=INNER ** -0.5)
        p["norm%d" % i] = torch.ones(MODEL, device=device, requires_grad=True)
        if mixer == "gated":
            p["gates%d" % i] = rnd(2 * INNER, INNER, scale=INNER ** -0.5)
            top = 0.9 + 0.099 * torch.rand(INNER, generator=g)      # decays at a full gate
            p["lam%d" % i] = torch.log(torch.expm1(-torch.log(top) / 8)).to(device).requires_grad_()
        else:
            p["x%d" % i] = rnd(2 * STATE + 1, INNER, scale=INNER ** -0.5)
            p["dt%d" % i] = rnd(INNER, scale=0.1)
            p["bias%d" % i] = torch.log(torch.expm1(dt)).to(device).requires_grad_()
            p["A%d" % i] = (-(torch.arange(STATE) + 1.0)).repeat(INNER, 1).to(device).requires_grad_()
            p["D%d" % i] = torch.ones(INNER, device=device, requires_grad=True)
        p["w%d" % i] = rnd(INNER, WIDTH, scale=WIDTH ** -0.5)
        p["b%d" % i] = rnd(INNER, scale=0.0)
    p["norm%d" % LAYERS] = torch.ones(MODEL, device=device, requires_grad=True)
    return p


def projections(p, i, u):
    """delta, B and C of the scan from its input u [rows, INNER, L]."""
    r = p["x%d" % i] @ u
    return p["dt%d" % i][:, None] * r[:, 2 * STATE:], r[:, :STATE], r[:, STATE:2 * STATE]


def gates(p, i, u):
    """Both gates of the recurrence from its input u [rows, INNER, L]."""
    return (p["gates%d" % i] @ u).split(INNER, dim=1)


def hidden(p, tokens):
    """What the head reads of whole sequences, [rows, MODEL, L], differentiable."""
    branch, x = p["embed"][tokens].transpose(1, 2).contiguous(), None      # channel-major: [rows, MODEL, L]
    for i in range(LAYERS):
        y, x = vms.rms_norm_autograd(branch, p["norm%d" % i], residual=x)
        xz = p["in%d" % i] @ y
        u, _ = vms.s6_causal_conv_autograd(xz[:, :INNER], p["w%d" % i], p["b%d" % i])
        if "lam%d" % i in p:
            y, _ = vms.gated_scan_autograd(u, *gates(p, i, u), p["lam%d" % i], z=xz[:, INNER:])
        else:
            delta, B, C = projections(p, i, u)
            y, _ = vms.s6_causal_scan_autograd(u, delta.contiguous(), xz[:, INNER:], B.contiguous(), C.contiguous(), p["A%d" % i],
                                               p["D%d" % i], p["bias%d" % i])
        branch = p["out%d" % i] @ y
    return vms.rms_norm_autograd(branch, p["norm%d" % LAYERS], residual=x)[0]


def forward(p, tokens):
    """Logits [rows, L, VOCAB] of whole sequences, differentiable."""
    return hidden(p, tokens).transpose(1, 2) @ p["head"].T


def progressions(rows, length, g, device="cuda"):
    start = torch.randint(0, VOCAB, (rows, 1), generator=g)
    step = torch.randint(1, 6, (rows, 1), generator=g)
    return ((start + step * torch.arange(length)) % VOCAB).to(device)


def train(p, steps, seed=1, rows=64, length=24, lr=3e-3):
    """Losses of `steps` optimizer steps."""
    g = torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(p.values(), lr=lr)
    losses = []
    for _ in range(steps):
        t = progressions(rows, length + 1, g)
        h = hidden(p, t[:, :-1]).transpose(1, 2).reshape(-1, MODEL)
        loss = vms.vocab_loss_autograd(h, p["head"], t[:, 1:].reshape(-1)).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


@torch.no_grad()
def prompt(p, tokens, lengths):
    """The last token's logits [rows, VOCAB] of a ragged batch, and each layer's (window, h)."""
    branch, x = p["embed"][tokens].transpose(1, 2).contiguous(), None
    states = []
    for i in range(LAYERS):
        y, x = vms.rms_norm(branch, p["norm%d" % i], residual=x, lengths=lengths)
        xz = p["in%d" % i] @ y
        u, window = vms.s6_causal_conv(xz[:, :INNER], p["w%d" % i], p["b%d" % i], lengths=lengths)
        if "lam%d" % i in p:
            y, h = vms.gated_scan(u, *gates(p, i, u), p["lam%d" % i], z=xz[:, INNER:], lengths=lengths)
        else:
            delta, B, C = projections(p, i, u)
            y, h = vms.s6_causal_scan(u, delta.contiguous(), xz[:, INNER:], B, C, p["A%d" % i], p["D%d" % i], p["bias%d" % i],
                                      lengths=lengths)
        states.append((window, h))
        branch = p["out%d" % i] @ y
    at = (lengths.long() - 1)[:, None, None].expand(-1, MODEL, 1)
    last, _ = vms.rms_norm(branch.gather(2, at).squeeze(2), p["norm%d" % LAYERS], residual=x.gather(2, at).squeeze(2))
    return last @ p["head"].T, states


@torch.no_grad()
def step(p, token, pools, slot_in, slot_out):
    """One token of every row: logits [rows, VOCAB]; pools hold each layer's (window, h)."""
    branch, x = p["embed"][token.long()], None
    for i, (window, h) in enumerate(pools):
        y, x = vms.rms_norm(branch, p["norm%d" % i], residual=x)
        xz = y @ p["in%d" % i].T
        u = vms.s6_conv_step(xz[:, :INNER], p["w%d" % i], p["b%d" % i], window, slot_in=slot_in, slot_out=slot_out)
        if "lam%d" % i in p:
            r, gate = (u @ p["gates%d" % i].T).split(INNER, dim=1)
            y = vms.gated_scan_step(u, r, gate, p["lam%d" % i], h, z=xz[:, INNER:], slot_in=slot_in, slot_out=slot_out)
        else:
            r = u @ p["x%d" % i].T
            y = vms.s6_scan_step(u, r[:, 2 * STATE:] * p["dt%d" % i], xz[:, INNER:], r[:, :STATE], r[:, STATE:2 * STATE],
                                 p["A%d" % i], p["D%d" % i], p["bias%d" % i], h, slot_in=slot_in, slot_out=slot_out)
        branch = y @ p["out%d" % i].T
    y, _ = vms.rms_norm(branch, p["norm%d" % LAYERS], residual=x)
    return y @ p["head"].T


@torch.no_grad()
def beam_search(p, tokens, lengths, beams, count, eos=None, move=False):
    """Continue each prompt by `count` tokens. Returns (sequences [rows, beams, count], scores [rows, beams]).

    move: keep one set of states and move them to the beams that go on, instead
    of two sets that are read and written in turn. Both give the same."""
    rows, dev = tokens.shape[0], tokens.device
    n = rows * beams
    logits, states = prompt(p, tokens, lengths)
    # one or two sets of n slots, all layers in one tensor; every beam of a prompt
    # starts from the state at its first slot
    total = n if move else 2 * n
    windows, hs = (v[0].new_zeros(LAYERS, total, *v[0].shape[1:]) for v in zip(*states))
    for i, (window, h) in enumerate(states):
        windows[i, :n:beams], hs[i, :n:beams] = window, h
    pools = list(zip(windows, hs))
    slots = torch.arange(n, dtype=torch.int32, device=dev)
    scores = torch.full((rows, beams), -math.inf, device=dev)
    scores[:, 0] = 0
    done = torch.zeros(rows, beams, dtype=torch.bool, device=dev)
    picked = torch.empty(rows, beams, 0, dtype=torch.int32, device=dev)
    logits = logits[:, None].expand(rows, beams, VOCAB)
    for k in range(count):
        scores, parent, token = vms.beam_select(logits, scores, done=None if eos is None else done, eos=eos)
        flat = parent.flatten()
        picked = torch.cat([picked.view(n, k)[flat.long()].view(rows, beams, k), token[..., None]], dim=2)
        if eos is not None:
            done = done.flatten()[flat.long()].view(rows, beams) | (token == eos)
        if k + 1 == count:
            break
        source = flat // beams * beams if k == 0 else flat          # at first all beams share their prompt's state
        if move:
            for state in (windows, hs):
                vms.beam_reorder(state, source.view(rows, beams))
            logits = step(p, token.flatten(), pools, slots, slots).view(rows, beams, VOCAB)
            continue
        # read the set that the last token wrote, at the parents; write the other
        read, write = (0, n) if k % 2 == 0 else (n, 0)
        logits = step(p, token.flatten(), pools, source + read, slots + write).view(rows, beams, VOCAB)
    return picked, scores


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300, help="training steps")
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--move", action="store_true", help="one set of states, moved to the beams that go on")
    ap.add_argument("--mixer", choices=("s6", "gated"), default="s6")
    a = ap.parse_args()
    p = init(mixer=a.mixer)
    losses = train(p, a.steps)
    print("loss %.3f at the start, %.3f at the end of %d steps" % (losses[0], losses[-1], a.steps))
    g = torch.Generator().manual_seed(7)
    t = progressions(3, 20, g)
    lengths = torch.tensor([4, 9, 12], dtype=torch.int32, device=t.device)
    out, scores = beam_search(p, t[:, :12], lengths, a.beams, 8, move=a.move)
    for i in range(3):
        n = int(lengths[i])
        print("prompt %s" % t[i, :n].tolist())
        print("  true      %s" % t[i, n:n + 8].tolist())
        for k in range(min(2, a.beams)):
            print("  beam %d    %s   log-probability %.3f" % (k, out[i, k].tolist(), float(scores[i, k])))


if __name__ == "__main__":
    main()
