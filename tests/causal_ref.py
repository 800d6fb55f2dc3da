"""The causal mixer and beam search written out plainly in float64 torch on the
CPU, token by token, from the definitions in include/vimscan.h. Gradients come
from autograd over these steps. Test infrastructure; shares no code with the
library."""
import math

import torch

F64 = torch.float64


def f64(t):
    return None if t is None else t.detach().to("cpu", F64)


def row_lengths(lengths, batch, L):
    return [L] * batch if lengths is None else [min(max(int(v), 0), L) for v in lengths]


def conv(x, w, bias, window, lengths, silu=True):
    batch, dim, L = x.shape
    W = w.shape[1]
    if window is None:
        window = torch.zeros(batch, dim, W - 1, dtype=F64)
    ys, wins = [], []
    for b, n in enumerate(row_lengths(lengths, batch, L)):
        line = torch.cat([window[b], x[b, :, :n]], dim=1)
        pre = sum(w[:, j:j + 1] * line[:, j:j + n] for j in range(W))
        if bias is not None:
            pre = pre + bias[:, None]
        y = pre * torch.sigmoid(pre) if silu else pre
        ys.append(torch.cat([y, torch.zeros(dim, L - n, dtype=F64)], dim=1))
        wins.append(line[:, n:n + W - 1])
    return torch.stack(ys), torch.stack(wins)


def scan(u, delta, z, B, C, A, D, dt_bias, h0, lengths, softplus=True):
    batch, dim, L = u.shape
    N = A.shape[1]
    ys, hs = [], []
    for b, n in enumerate(row_lengths(lengths, batch, L)):
        h = torch.zeros(dim, N, dtype=F64) if h0 is None else h0[b]
        cols = []
        for t in range(n):
            x = delta[b, :, t] if dt_bias is None else delta[b, :, t] + dt_bias
            step = torch.logaddexp(x, torch.zeros_like(x)) if softplus else x
            h = torch.exp(step[:, None] * A) * h + (step * u[b, :, t])[:, None] * B[b, :, t][None]
            y = h @ C[b, :, t]
            if D is not None:
                y = y + D * u[b, :, t]
            if z is not None:
                y = y * z[b, :, t] * torch.sigmoid(z[b, :, t])
            cols.append(y)
        cols += [torch.zeros(dim, dtype=F64)] * (L - n)
        ys.append(torch.stack(cols, dim=1))
        hs.append(h)
    return torch.stack(ys), torch.stack(hs)


def gradients(outputs, upstream, inputs):
    """dL/d inputs for L = sum of outputs x upstream; zeros where an input does not matter."""
    loss = sum((o * g).sum() for o, g in zip(outputs, upstream) if g is not None)
    wanted = [t for t in inputs if t is not None]
    got = iter(torch.autograd.grad(loss, wanted, allow_unused=True))
    out = []
    for t in inputs:
        if t is None:
            out.append(None)
            continue
        g = next(got)
        out.append(torch.zeros_like(t) if g is None else g)
    return out


def select(logits, scores, done, eos):
    """(scores, parent, token) lists per sequence: every candidate sorted by score,
    then beam, then logit, then token."""
    batch, beams, vocab = logits.shape
    inf = math.inf
    S, P, T = [], [], []
    for b in range(batch):
        cands = []
        for k in range(beams):
            sc = float(scores[b, k])
            if done is not None and bool(done[b, k]):
                vals = [(0.0 if t == eos else -inf) for t in range(vocab)]
                logp = vals
            else:
                vals = [(-inf if math.isnan(v) else v + 0.0) for v in logits[b, k].tolist()]
                m = max(vals)
                if m == -inf:
                    logp = [-inf] * vocab
                elif m == inf:
                    n = sum(v == inf for v in vals)
                    logp = [-math.log(n) if v == inf else -inf for v in vals]
                else:
                    lse = math.log(sum(math.exp(v - m) for v in vals))
                    logp = [(v - m) - lse for v in vals]
            for t in range(vocab):
                total = sc + logp[t]
                if math.isnan(total):
                    total = -inf
                cands.append((-total, k, -vals[t], t))
        cands.sort()
        best = cands[:beams]
        S.append([-c[0] for c in best])
        P.append([b * beams + c[1] for c in best])
        T.append([c[3] for c in best])
    return torch.tensor(S, dtype=F64), torch.tensor(P, dtype=torch.int32), torch.tensor(T, dtype=torch.int32)
