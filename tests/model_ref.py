"""The gated linear recurrence, the norm and the vocabulary loss written out
plainly in float64 torch on the CPU, from the definitions in include/vimscan.h.
Gradients come from autograd over these steps. Test infrastructure; shares no
code with the library."""
import torch

from causal_ref import F64, f64, gradients, row_lengths  # noqa: F401


def gated(x, r, i, lam, z, h0, lengths, rate=8.0):
    batch, dim, L = x.shape
    k = rate * torch.logaddexp(lam, torch.zeros_like(lam))
    ys, hs = [], []
    for b, n in enumerate(row_lengths(lengths, batch, L)):
        h = torch.zeros(dim, dtype=F64) if h0 is None else h0[b]
        s = k[:, None] * torch.sigmoid(r[b, :, :n])
        a, v = torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s)) * torch.sigmoid(i[b, :, :n]) * x[b, :, :n]
        cols = []
        for t in range(n):
            h = a[:, t] * h + v[:, t]
            cols.append(h)
        y = torch.stack(cols, dim=1) if cols else torch.zeros(dim, 0, dtype=F64)
        if z is not None:
            y = y * z[b, :, :n] * torch.sigmoid(z[b, :, :n])
        ys.append(torch.cat([y, torch.zeros(dim, L - n, dtype=F64)], dim=1))
        hs.append(h)
    return torch.stack(ys), torch.stack(hs)


def norm(x, w, residual, lengths, eps, dtype):
    """(y, s) of [batch, dim, L]; s is rounded to dtype, which a gradient passes unchanged."""
    s = x if residual is None else x + residual
    s = s + (s.detach().to(dtype).to(F64) - s.detach())
    live = torch.zeros(x.shape[0], 1, x.shape[2], dtype=F64)
    for b, n in enumerate(row_lengths(lengths, x.shape[0], x.shape[2])):
        live[b, :, :n] = 1
    s = s * live
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    if w is not None:
        y = y * w[:, None]
    return y * live, s


def vocab(x, W, target):
    """(loss, lse) of [tokens, dim] activations, wherever they are; float64 in, float64 out."""
    l = x @ W.T
    top = l.max(dim=1, keepdim=True).values
    lse = (top + torch.log(torch.exp(l - top).sum(dim=1, keepdim=True)))[:, 0]
    kept = (target >= 0) & (target < W.shape[0])
    at = torch.where(kept, target, torch.zeros_like(target)).long()
    return torch.where(kept, lse - l.gather(1, at[:, None])[:, 0], torch.zeros_like(lse)), lse
