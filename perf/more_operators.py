"""Measured cases of a causal language model's other operators: the gated
linear recurrence, the root-mean-square norm with the residual's addition, and
the cross entropy over a vocabulary.

Kinds of pass, each as a program with such a model makes it:

  scan        the recurrence over a batch of prompts of different lengths, with
              the states that go in and come out
  scan_train  the same for training, then the gradients of every input
  scan_step   one new token per sequence, on a pool of states that is read at
              one slot and written at another
  norm        residual addition and norm, channel-major prompts or (seqlen 1)
              one row per token
  norm_train  the same, then the gradients of the stream and the weight
  loss        the loss of every token of a text (scoring it)
  loss_train  the same, then the gradients of the activations and the head

With `own` false, `run` computes them from elementary torch operations in 32
bits, rounded once at the end of each operator; with `own` true it calls the
package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEVICE = "cuda"
RATE = 8.0          # the recurrence's decay at a full gate is rate x softplus(lam)
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt of a small model: latency counts
        dict(name="scan-1x384x197-f32", op="scan", dtype="f32", batch=1, dim=384, seqlen=197, shortest=197, carried=False, gated=True),
        # a batch of prompts of different lengths that continue earlier text
        dict(name="scan-8x768x4097-bf16", op="scan", dtype="bf16", batch=8, dim=768, seqlen=4097, shortest=2049, carried=True,
             gated=True),
        # one long document in a wide layer, no output gate: few rows, a long axis
        dict(name="scan-1x1536x16385-bf16", op="scan", dtype="bf16", batch=1, dim=1536, seqlen=16385, shortest=16385, carried=False,
             gated=False),
        # a training step at the ordinary size
        dict(name="scan_train-8x768x4097-bf16", op="scan_train", dtype="bf16", batch=8, dim=768, seqlen=4097, shortest=4097,
             carried=False, gated=True),
        # a decode batch of a serving loop, some of its rows empty
        dict(name="scan_step-515x1536-bf16", op="scan_step", dtype="bf16", batch=515, dim=1536, padded=7, gated=True),
        # one row per decoded sequence
        dict(name="norm-64x1536-bf16", op="norm", dtype="bf16", batch=64, dim=1536, seqlen=1, shortest=1, added=True),
        # prompts of different lengths in full precision
        dict(name="norm-8x384x1025-f32", op="norm", dtype="f32", batch=8, dim=384, seqlen=1025, shortest=300, added=True),
        # a training step at the ordinary size
        dict(name="norm_train-8x768x4097-bf16", op="norm_train", dtype="bf16", batch=8, dim=768, seqlen=4097, shortest=4097, added=True),
        # token-major activations: the norm before the head, trained on rows
        dict(name="norm_train-8194x1536-bf16", op="norm_train", dtype="bf16", batch=8194, dim=1536, seqlen=1, shortest=1, added=False),
        # a short text scored against a large vocabulary
        dict(name="loss-197x768x49999-bf16", op="loss", dtype="bf16", tokens=197, dim=768, vocab=49999, ignored=0),
        # a small full-precision training step
        dict(name="loss_train-394x384x32768-f32", op="loss_train", dtype="f32", tokens=394, dim=384, vocab=32768, ignored=57),
        # two long texts in a training step with a wide head
        dict(name="loss_train-8194x1536x49999-bf16", op="loss_train", dtype="bf16", tokens=8194, dim=1536, vocab=49999, ignored=811),
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of [low, high]; odd ones are as likely as others."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


MOST_ELEMENTS = 8 * 768 * 4097          # batch x dim x seqlen of the largest listed scan or norm
MOST_PRODUCTS = 8194 * 1536 * 49999     # tokens x dim x vocab of the largest listed loss


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_step", "norm", "norm_train", "norm_train", "loss", "loss_train", "loss_train"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("loss", "loss_train"):
        # 32-bit products run at a sixteenth of the rate
        most = MOST_PRODUCTS // (16 if dtype == "f32" else 1)
        while True:
            tokens, dim, vocab = _log(rng, 1, 8194), _log(rng, 24, 1536), _log(rng, 100, 49999)
            if rng.random() < 0.6:
                dim = -(-dim // 8) * 8
            if tokens * dim * vocab <= most:
                break
        return dict(op=op, dtype=dtype, tokens=tokens, dim=dim, vocab=vocab, ignored=rng.choice([0, tokens // 10, tokens // 2]))
    if op == "scan_step":
        batch = _log(rng, 1, 515)
        return dict(op=op, dtype=dtype, batch=batch, dim=_log(rng, 24, 1536), padded=rng.randint(0, batch // 4), gated=rng.random() < 0.7)
    rows = op.startswith("norm") and rng.random() < 0.4
    while True:
        batch, dim, seqlen = _log(rng, 1, 8194 if rows else 64), _log(rng, 24, 1536), 1 if rows else _log(rng, 1, 16385)
        if batch * dim * seqlen <= MOST_ELEMENTS:
            break
    c = dict(op=op, dtype=dtype, batch=batch, dim=dim, seqlen=seqlen,
             shortest=1 if rows else rng.choice([0, min(1, seqlen), seqlen // 2, seqlen, seqlen]))
    if op.startswith("norm"):
        return dict(c, added=rng.random() < 0.7)
    return dict(c, carried=rng.random() < 0.5, gated=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _lengths(c):
    """Row lengths from `shortest` to seqlen, evenly spread (their order is drawn with the inputs)."""
    n, low, high = c["batch"], c["shortest"], c["seqlen"]
    return [high - (high - low) * i // max(1, n - 1) for i in range(n)]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1_000_003 * seed + 29)
    dt = DTYPES[case["dtype"]]
    f = torch.float32

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEVICE)

    c, s = case, dict(case=dict(case))
    if "loss" in c["op"]:
        t, d, v = c["tokens"], c["dim"], c["vocab"]
        head = torch.randn(v, d, generator=g, device=DEVICE) * (2 * d ** -0.5)
        s["target"] = torch.randint(0, v, (t,), generator=g, device=DEVICE)
        # normed activations that know something of what follows
        s["x"] = (torch.randn(t, d, generator=g, device=DEVICE) + head[s["target"]]).to(dt)
        s["W"] = head.to(dt)
        s["target"][torch.randperm(t, generator=g, device=DEVICE)[:c["ignored"]]] = -100
        if c["op"] == "loss_train":
            # the mean over what is not ignored, texts weighted
            s["dloss"] = (0.5 + uniform(t)) / max(1, t - c["ignored"])
        return s
    b, d = c["batch"], c["dim"]
    if c["op"] == "scan_step":
        # x and z are the halves of one projection's output, the gates of another's
        s["x"], s["z"] = normal(b, 2 * d).split(d, dim=1)
        s["r"], s["i"] = normal(b, 2 * d).split(d, dim=1)
        # a pool of 2 b states: this token reads the first half and writes the second
        s["h"] = normal(2 * b, d, dtype=f)
        s["slot_in"] = torch.randint(0, b, (b,), generator=g, device=DEVICE).to(torch.int32)
        s["slot_out"] = (b + torch.randperm(b, generator=g, device=DEVICE)).to(torch.int32)
        gone = torch.randperm(b, generator=g, device=DEVICE)[:c["padded"]]
        s["slot_in"][gone] = -1
        s["slot_out"][gone] = -1
    else:
        L = c["seqlen"]
        s["lengths"] = None
        if c["shortest"] < L:
            order = torch.randperm(b, generator=g, device=DEVICE)
            s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEVICE)[order]
    if c["op"].startswith("norm"):
        shape = (b, d) if L == 1 else (b, d, L)
        s["x"], s["w"] = normal(*shape), 1 + 0.1 * normal(d, dtype=f)
        # the stream has grown over the layers before
        s["residual"] = normal(*shape, scale=3.0) if c["added"] else None
        if c["op"] == "norm_train":
            s["dy"], s["dsum"] = normal(*shape), normal(*shape) if c["added"] else None
        return s
    # decays a at a full gate between 0.9 and 0.999
    top = 0.9 + 0.099 * uniform(d)
    s["lam"] = torch.log(torch.expm1(-torch.log(top) / RATE))
    if c["op"] != "scan_step":
        xz = normal(b, 2 * d, L)
        s["x"], s["z"] = xz[:, :d], xz[:, d:]
        ri = normal(b, 2 * d, L)
        s["r"], s["i"] = ri[:, :d], ri[:, d:]
        s["h0"] = normal(b, d, dtype=f) if c["carried"] else None
        if c["op"] == "scan_train":
            s["dy"] = normal(b, d, L)
            s["dh"] = normal(b, d, dtype=f) if c["carried"] else None
    if not c["gated"]:
        s["z"] = None
    return s


# ------------------------------------------------------------- plain forms
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _valid(lengths, b, L):
    if lengths is None:
        return torch.ones(b, 1, L, dtype=torch.bool, device=DEVICE)
    return (torch.arange(L, device=DEVICE) < lengths[:, None])[:, None, :]


def _recur(a, v):
    """h_t = a_t h_{t-1} + v_t over axis 2 by doubling: after the pass of stride s each entry holds its last 2 s steps."""
    s = 1
    while s < v.shape[2]:
        v = torch.cat([v[:, :, :s], v[:, :, s:] + a[:, :, s:] * v[:, :, :-s]], dim=2)
        a = torch.cat([a[:, :, :s], a[:, :, s:] * a[:, :, :-s]], dim=2)
        s *= 2
    return v


def _softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


def _gates(x, r, i, lam, ok):
    """s, a, m = sqrt(1 - a^2), sigmoid(r), sigmoid(i) and x; a step of a = 1 and m = 0 at padding."""
    sr, si = _sigmoid(torch.where(ok, r.float(), 0.0)), _sigmoid(torch.where(ok, i.float(), 0.0))
    k = RATE * _softplus(lam)
    s = torch.where(ok, k[:, None] * sr, 0.0)
    return s, torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s)), sr, si, torch.where(ok, x.float(), 0.0)


def _states(a, v, h0):
    if h0 is not None:
        v = torch.cat([(v[:, :, 0] + a[:, :, 0] * h0)[:, :, None], v[:, :, 1:]], dim=2)
    return _recur(a, v)


def plain_scan(x, r, i, lam, z, h0, lengths):
    ok = _valid(lengths, x.shape[0], x.shape[2])
    s, a, m, sr, si, xf = _gates(x, r, i, lam, ok)
    h = _states(a, m * si * xf, h0)
    y = h
    if z is not None:
        zf = torch.where(ok, z.float(), 0.0)
        y = h * (zf * _sigmoid(zf))
    return torch.where(ok, y, 0.0).to(x.dtype), h[:, :, -1].clone()


def plain_scan_grad(x, r, i, lam, z, h0, lengths, dy, dh):
    t = x.dtype
    ok = _valid(lengths, x.shape[0], x.shape[2])
    s, a, m, sr, si, xf = _gates(x, r, i, lam, ok)
    h = _states(a, m * si * xf, h0)
    gy, dz = torch.where(ok, dy.float(), 0.0), None
    if z is not None:
        zf = torch.where(ok, z.float(), 0.0)
        sz = _sigmoid(zf)
        dz = (gy * h * sz * (1 + zf * (1 - sz))).to(t)
        gy = gy * zf * sz
    # the adjoint runs back over the tokens: mu_t = gy_t + a_{t+1} mu_{t+1}
    v = gy if dh is None else torch.cat([gy[:, :, :-1], (gy[:, :, -1] + dh)[:, :, None]], dim=2)
    later = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], dim=2)
    mu = _recur(later.flip(2), v.flip(2)).flip(2)
    before = torch.cat([torch.zeros_like(h[:, :, :1]) if h0 is None else h0[:, :, None], h[:, :, :-1]], dim=2)
    # s / m goes to zero with s, 1 / m does not
    ratio = torch.where(s > 0, s / m.clamp_min(1e-30), 0.0)
    ds_s = mu * (a * a * si * xf * ratio - s * a * before)
    slope = _sigmoid(lam) / _softplus(lam)
    return dict(dx=(mu * m * si).to(t), di=(mu * m * si * xf * (1 - si)).to(t), dr=(ds_s * (1 - sr)).to(t), dz=dz,
                dlam=slope * ds_s.sum((0, 2)), dh0=None if h0 is None else a[:, :, 0] * mu[:, :, 0])


def plain_scan_step(x, r, i, lam, h, z, slot_in, slot_out):
    ok = (slot_in >= 0) & (slot_out >= 0)
    s, a, m, sr, si, xf = _gates(x[..., None], r[..., None], i[..., None], lam, torch.ones_like(ok)[:, None, None])
    new = a[..., 0] * h[slot_in.clamp_min(0).long()] + (m * si * xf)[..., 0]
    # an empty row puts slot 0 back as it is (no other row writes there)
    at = slot_out.clamp_min(0).long()
    h[at] = torch.where(ok[:, None], new, h[at])
    y = new
    if z is not None:
        y = new * (z.float() * _sigmoid(z.float()))
    return torch.where(ok[:, None], y, 0.0).to(x.dtype)


def _live(lengths, x):
    """Where a row [b, d] or prompt [b, d, L] is no padding."""
    if lengths is None:
        return torch.ones((), dtype=torch.bool, device=DEVICE)
    return _valid(lengths, x.shape[0], x.shape[2])


def plain_norm(x, w, residual, lengths):
    ok = _live(lengths, x)
    s = torch.where(ok, x if residual is None else (x.float() + residual.float()).to(x.dtype), 0.0)
    f = s.float()
    wf = w.view(-1, *([1] * (x.dim() - 2)))
    y = f / torch.sqrt(f.square().mean(1, keepdim=True) + EPS) * wf
    return torch.where(ok, y, 0.0).to(x.dtype), s


def plain_norm_grad(s, w, dy, dsum, lengths):
    ok = _live(lengths, s)
    f, g = torch.where(ok, s.float(), 0.0), torch.where(ok, dy.float(), 0.0)
    wf = w.view(-1, *([1] * (s.dim() - 2)))
    q = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
    dx = q * (wf * g) - f * q * q * q * (wf * g * f).mean(1, keepdim=True)
    if dsum is not None:
        dx = dx + dsum.float()
    dw = (g * f * q).sum([k for k in range(s.dim()) if k != 1])
    return dict(dx=torch.where(ok, dx, 0.0).to(s.dtype), dw=dw)


def _logits(x, W, target):
    """Logits in 32 bits, what is left out, and each target's column (0 where it is left out)."""
    out = (target < 0) | (target >= W.shape[0])
    return x.float() @ W.float().T, out, torch.where(out, 0, target)[:, None]


def plain_loss(x, W, target):
    l, out, at = _logits(x, W, target)
    top = l.max(dim=1, keepdim=True).values
    lse = (top + torch.log(torch.exp(l - top).sum(dim=1, keepdim=True)))[:, 0]
    return torch.where(out, 0.0, lse - l.gather(1, at)[:, 0]), lse


def plain_loss_grad(x, W, target, lse, dloss):
    l, out, at = _logits(x, W, target)
    p = torch.exp(l - lse[:, None])
    p.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    p *= torch.where(out, 0.0, dloss)[:, None]
    return dict(dx=(p @ W.float()).to(x.dtype), dW=(p.T @ x.float()).to(W.dtype))


# --------------------------------------------------------------------- run
def run(state):
    return globals()["_run_" + state["case"]["op"]](state)


def _run_scan(s):
    if own:
        import vision_mamba_selective_amd as vms
        y, h = vms.gated_scan(s["x"], s["r"], s["i"], s["lam"], z=s["z"], h0=s["h0"], lengths=s["lengths"], rate=RATE)
    else:
        y, h = plain_scan(s["x"], s["r"], s["i"], s["lam"], s["z"], s["h0"], s["lengths"])
    return dict(y=y, h=h)


def _run_scan_train(s):
    if own:
        import vision_mamba_selective_amd as vms
        rest = (s["x"], s["r"], s["i"], s["lam"])
        y, h, saved = vms.gated_scan_saved(*rest, z=s["z"], h0=s["h0"], lengths=s["lengths"], rate=RATE)
        g = vms.gated_scan_grad(*rest, saved, s["dy"], z=s["z"], dh=s["dh"], h0=s["h0"], lengths=s["lengths"], rate=RATE)
    else:
        rest = (s["x"], s["r"], s["i"], s["lam"], s["z"], s["h0"], s["lengths"])
        y, h = plain_scan(*rest)
        g = plain_scan_grad(*rest, s["dy"], s["dh"])
    return dict(y=y, h=h, **g)


def _run_scan_step(s):
    if own:
        import vision_mamba_selective_amd as vms
        y = vms.gated_scan_step(s["x"], s["r"], s["i"], s["lam"], s["h"], z=s["z"], slot_in=s["slot_in"], slot_out=s["slot_out"], rate=RATE)
    else:
        y = plain_scan_step(s["x"], s["r"], s["i"], s["lam"], s["h"], s["z"], s["slot_in"], s["slot_out"])
    return dict(y=y, h=s["h"])


def _run_norm(s):
    if own:
        import vision_mamba_selective_amd as vms
        y, stream = vms.rms_norm(s["x"], s["w"], residual=s["residual"], lengths=s["lengths"], eps=EPS)
    else:
        y, stream = plain_norm(s["x"], s["w"], s["residual"], s["lengths"])
    return dict(y=y, stream=stream) if s["case"]["added"] else dict(y=y)


def _run_norm_train(s):
    if own:
        import vision_mamba_selective_amd as vms
        y, stream = vms.rms_norm(s["x"], s["w"], residual=s["residual"], lengths=s["lengths"], eps=EPS)
        g = vms.rms_norm_grad(stream, s["w"], s["dy"], dsum=s["dsum"], lengths=s["lengths"], eps=EPS)
    else:
        y, stream = plain_norm(s["x"], s["w"], s["residual"], s["lengths"])
        g = plain_norm_grad(stream, s["w"], s["dy"], s["dsum"], s["lengths"])
    return dict(y=y, stream=stream, **g) if s["case"]["added"] else dict(y=y, **g)


def _run_loss(s):
    if own:
        import vision_mamba_selective_amd as vms
        loss, lse = vms.vocab_loss(s["x"], s["W"], s["target"])
    else:
        loss, lse = plain_loss(s["x"], s["W"], s["target"])
    return dict(loss=loss, lse=lse)


def _run_loss_train(s):
    if own:
        import vision_mamba_selective_amd as vms
        loss, lse = vms.vocab_loss(s["x"], s["W"], s["target"])
        g = vms.vocab_loss_grad(s["x"], s["W"], s["target"], lse, s["dloss"])
    else:
        loss, lse = plain_loss(s["x"], s["W"], s["target"])
        g = plain_loss_grad(s["x"], s["W"], s["target"], lse, s["dloss"])
    return dict(loss=loss, lse=lse, **g)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if "loss" in c["op"]:
        t, d, v = c["tokens"], c["dim"], c["vocab"]
        train = c["op"] == "loss_train"
        # one product gives the logits, two more the gradients
        return dict(bytes=e * d * (t + v) * (2 if train else 1) + t * (20 if train else 16), flops=(6 if train else 2) * t * d * v)
    if c["op"] == "scan_step":
        b, d = c["batch"] - c["padded"], c["dim"]
        n = 5 if c["gated"] else 4
        return dict(bytes=b * d * ((n - 1) * e + 8) + c["batch"] * d * e + 4 * d, flops=b * d * 40)
    b, d, L = c["batch"], c["dim"], c["seqlen"]
    el, out = sum(_lengths(c)) * d, b * d * L               # outputs are written whole, zeros at the padding
    if c["op"].startswith("norm"):
        r = 2 if c["added"] else 1
        nbytes, flops = e * r * (el + out) + 4 * d, 5 * el
        if c["op"] == "norm_train":                         # dy, dsum; dx, dw
            nbytes, flops = nbytes + e * (r * el + out) + 4 * d, flops + 12 * el
        return dict(bytes=nbytes, flops=flops)
    n = 4 if c["gated"] else 3
    nbytes = e * (n * el + out) + 4 * d + 4 * b * d * (2 if c["carried"] else 1)
    flops = el * 40
    if c["op"] == "scan_train":                             # dy; a gradient for each input
        nbytes += e * (el + n * out) + 4 * d + (8 * b * d if c["carried"] else 0)
        flops += el * 40
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return globals()["_exact_" + case["op"]](s)


def _walk(s):
    """The recurrence token by token: every decay, input and state, [b, d, L]."""
    b, d, L = s["x"].shape
    n = torch.full((b,), L, device=DEVICE) if s["lengths"] is None else s["lengths"].long()
    live = (torch.arange(L, device=DEVICE)[None, :] < n[:, None]).double()[:, None, :]
    k = RATE * torch.logaddexp(s["lam"], torch.zeros_like(s["lam"]))
    logs = k[:, None] * torch.special.expit(s["r"]) * live
    m = torch.sqrt(-torch.expm1(-2 * logs))
    a, v = torch.exp(-logs), m * torch.special.expit(s["i"]) * s["x"]
    h = torch.zeros(b, d, dtype=torch.float64, device=DEVICE) if s["h0"] is None else s["h0"].clone()
    first, hs = h, torch.empty(L, b, d, dtype=torch.float64, device=DEVICE)
    at, vt = a.permute(2, 0, 1).contiguous(), v.permute(2, 0, 1).contiguous()
    for j in range(L):
        h = torch.addcmul(vt[j], at[j], h, out=hs[j])
    return dict(live=live, k=k, logs=logs, m=m, a=a, at=at, h=hs.permute(1, 2, 0), first=first, last=h.clone())


def _exact_scan(s):
    f = _walk(s)
    y = f["h"] if s["z"] is None else f["h"] * s["z"] * torch.special.expit(s["z"])
    return dict(y=y * f["live"], h=f["last"])


def _exact_scan_train(s):
    f = _walk(s)
    h, z, live = f["h"], s["z"], f["live"]
    dy = s["dy"] * live
    y, gy, dz = h * live, dy, None
    if z is not None:
        p = torch.special.expit(z)
        y, gy, dz = h * z * p * live, dy * z * p, dy * h * (p + z * p * (1 - p))
    b, d, L = h.shape
    gt, carry = gy.permute(2, 0, 1).contiguous(), torch.zeros(b, d, dtype=torch.float64, device=DEVICE) if s["dh"] is None else s["dh"]
    back = torch.empty_like(gt)                              # what reaches each state
    for j in reversed(range(L)):
        torch.add(gt[j], carry, out=back[j])
        carry = back[j] * f["at"][j]
    back = back.permute(1, 2, 0)
    si, sr = torch.special.expit(s["i"]), torch.special.expit(s["r"])
    prev = torch.cat([f["first"][:, :, None], h[:, :, :-1]], dim=2)
    # d/d log a of the state: through the decay and through m
    slope = torch.where(f["m"] > 0, f["a"] ** 2 / f["m"], torch.zeros_like(f["m"]))
    dlogs = back * (slope * si * s["x"] - f["a"] * prev)
    dr = dlogs * f["k"][:, None] * sr * (1 - sr) * live
    dlam = RATE * torch.special.expit(s["lam"]) * (dlogs * sr * live).sum((0, 2))
    return dict(y=y, h=f["last"], dx=back * f["m"] * si * live, di=back * f["m"] * s["x"] * si * (1 - si) * live, dr=dr, dz=dz, dlam=dlam,
                dh0=None if s["h0"] is None else carry)


def _exact_scan_step(s):
    h = s["h"].clone()
    y = torch.zeros_like(s["x"])
    k = RATE * torch.logaddexp(s["lam"], torch.zeros_like(s["lam"]))
    for j, (read, write) in enumerate(zip(s["slot_in"].tolist(), s["slot_out"].tolist())):
        if read < 0 or write < 0:
            continue
        logs = k * torch.special.expit(s["r"][j])
        h[write] = torch.exp(-logs) * s["h"][read] + torch.sqrt(-torch.expm1(-2 * logs)) * torch.special.expit(s["i"][j]) * s["x"][j]
        y[j] = h[write] if s["z"] is None else h[write] * s["z"][j] * torch.special.expit(s["z"][j])
    return dict(y=y, h=h)


def _exact_stream(s):
    """The sum as it is kept, in the activations' type, and 1 where a token is no padding."""
    total = s["x"] if s["residual"] is None else (s["x"] + s["residual"]).to(DTYPES[s["case"]["dtype"]]).double()
    total = total if total.dim() == 3 else total[:, :, None]
    b, _, L = total.shape
    n = torch.full((b,), L, device=DEVICE) if s["lengths"] is None else s["lengths"].long()
    live = (torch.arange(L, device=DEVICE)[None, :] < n[:, None]).double()[:, None, :]
    return total * live, live


def _exact_norm(s):
    total, live = _exact_stream(s)
    power = torch.linalg.vector_norm(total, dim=1, keepdim=True) ** 2 / total.shape[1]
    y = total * torch.rsqrt(power + EPS) * s["w"][:, None]
    out = dict(y=y.view_as(s["x"]), stream=total.view_as(s["x"]))
    return out if s["case"]["added"] else dict(y=out["y"])


def _exact_norm_train(s):
    total, live = _exact_stream(s)
    dim = total.shape[1]
    dy = s["dy"].view_as(total) * live
    q = torch.rsqrt(torch.linalg.vector_norm(total, dim=1, keepdim=True) ** 2 / dim + EPS)
    unit = total * q
    inner = dy * s["w"][:, None]
    dx = (inner - unit * ((inner * unit).sum(1, keepdim=True) / dim)) * q
    if s["dsum"] is not None:
        dx = dx + s["dsum"].view_as(total) * live
    return dict(_exact_norm(s), dx=dx.view_as(s["x"]), dw=(dy * unit).sum((0, 2)))


def _exact_loss(s):
    l = s["x"] @ s["W"].T
    lse = torch.logsumexp(l, dim=1)
    loss = torch.zeros_like(lse)
    kept = ((s["target"] >= 0) & (s["target"] < s["W"].shape[0])).nonzero()[:, 0]
    loss[kept] = lse[kept] - l[kept, s["target"][kept]]
    return dict(loss=loss, lse=lse)


def _exact_loss_train(s):
    l = s["x"] @ s["W"].T
    kept = ((s["target"] >= 0) & (s["target"] < s["W"].shape[0])).nonzero()[:, 0]
    p = torch.zeros_like(l)
    p[kept] = torch.softmax(l[kept], dim=1) * s["dloss"][kept, None]
    p[kept, s["target"][kept]] -= s["dloss"][kept]
    return dict(_exact_loss(s), dx=p @ s["W"], dW=p.T @ s["x"])
