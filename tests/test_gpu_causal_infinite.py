"""Infinite inputs of the causal scan, its gradient and its single-token form,
at state sizes on both sides of a full 16, in every form of the kernels: each
output is infinite or NaN exactly where the definition makes it so, evaluated
in float64 in IEEE arithmetic, and as close as elsewhere where it is finite.

The inputs keep every exp(delta A) of a single token above 2^-40, and the
products of a whole piece far below the smallest fp32 number; B, C, D and h0
are positive, so that an infinity meets others of its own sign and most results
are infinities, not NaN. The bound on finite values is the one of
test_gpu_causal.py (400 x 2^-24 of the size, and 2^-8 for bf16)."""
import pytest
import torch

import causal_ref as ref
from gpu_util import say
from test_gpu_causal import BF16_TOL, DT, F32_TOL

pytestmark = pytest.mark.gpu
INF = float("inf")
# whole rows, rows in pieces; each narrow, then wide
SHAPES = [(2, 37, 60), (512, 100, 33), (2, 37, 301), (12, 192, 3000)]
STATES = [1, 5, 8, 12, 16]
CH = 5                       # the channel that holds the infinity, in batch row 0


def same(got, want, what):
    g = got.detach().to("cpu", torch.float64)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        bad = kind(g) != kind(want)
        if bad.any():
            i = tuple(bad.nonzero()[0].tolist())
            raise AssertionError("%s: %d of %d not alike in %s; first at %s: got %r ref %r" % (
                what, int(bad.sum()), bad.numel(), kind.__name__, i, float(g[i]), float(want[i])))
    fin = torch.isfinite(want)
    if not fin.any():
        return
    g, w = g[fin], want[fin]
    tol = F32_TOL * (float(w.square().mean().sqrt()) + w.abs())
    if got.dtype == torch.bfloat16:
        tol = tol + BF16_TOL * w.abs()
    assert ((g - w).abs() <= tol).all(), (what, float((g - w).abs().max()))


def inputs(shape, N, dtype):
    batch, dim, L = shape
    g = torch.Generator().manual_seed(L + N)
    rnd = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    dt = DT[dtype]
    t = dict(u=rnd(batch, dim, L), delta=rnd(batch, dim, L).clamp(-3, 3) * 0.5 + 1, z=rnd(batch, dim, L), dy=rnd(batch, dim, L),
             B=torch.rand(batch, N, L, generator=g) + 0.5, C=torch.rand(batch, N, L, generator=g) + 0.5)
    t = {k: v.to(dt).cuda() for k, v in t.items()}
    t["A"] = (-(torch.rand(dim, N, generator=g) * 7.5 + 0.5)).cuda()
    t["D"] = (torch.rand(dim, generator=g) + 0.5).cuda()
    t["h0"] = (torch.rand(batch, dim, N, generator=g) + 0.5).cuda()
    t["dh"] = (torch.rand(batch, dim, N, generator=g) + 0.5).cuda()
    return t


def definition(t, chans):
    """y, h, du, ddelta, dz and dh0 of batch row 0 and some channels, token by token in float64."""
    d = {k: ref.f64(v) for k, v in t.items()}
    u, delta, z, dy = (d[k][0, chans] for k in ("u", "delta", "z", "dy"))
    B, C, A, D = d["B"][0], d["C"][0], d["A"][chans], d["D"][chans]
    L = u.shape[1]
    step = torch.logaddexp(delta, torch.zeros_like(delta))
    gate = torch.sigmoid(z)
    hs, h, ys = [d["h0"][0, chans]], d["h0"][0, chans], []
    for i in range(L):
        h = torch.exp(step[:, i, None] * A) * h + (step[:, i] * u[:, i])[:, None] * B[:, i]
        hs.append(h)
        ys.append((h * C[:, i]).sum(1) + D * u[:, i])
    ungated = torch.stack(ys, 1)
    y = ungated * (z * gate)
    dz = dy * ungated * (gate * (1 + z * (1 - gate)))
    gy = dy * (z * gate)
    lam, du, dd = d["dh"][0, chans], torch.zeros_like(u), torch.zeros_like(u)
    for i in reversed(range(L)):
        lam = lam + gy[:, i, None] * C[:, i]
        through = (lam * B[:, i]).sum(1)
        back = torch.exp(step[:, i, None] * A) * lam
        du[:, i] = step[:, i] * through + gy[:, i] * D
        dd[:, i] = (u[:, i] * through + (back * hs[i] * A).sum(1)) * torch.sigmoid(delta[:, i])
        lam = back
    return dict(y=y, h=h, du=du, ddelta=dd, dz=dz, dh0=lam)


def spoil(t, name, at):
    if name in ("h0", "dh"):
        t[name][0, CH] = INF
    else:
        t[name][0, CH, at] = INF


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d-d%d-L%d" % s)
@pytest.mark.parametrize("name", ["u", "delta", "h0"])
def test_scan(name, shape, N, dtype):
    import vision_mamba_selective_amd as vms
    t = inputs(shape, N, dtype)
    spoil(t, name, shape[2] // 3)
    say("case infinite %s scan %s %d %s" % (name, shape, N, dtype))
    chans = [0, CH, shape[1] - 1]
    want = definition(t, chans)
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"])
    y, h = vms.s6_causal_scan(*args, h0=t["h0"])
    assert torch.isinf(want["y"][1]).any() and torch.isfinite(want["y"][0]).all()
    same(y[0, chans], want["y"], "y")
    same(h[0, chans], want["h"], "h")
    y2, h2, _ = vms.s6_causal_scan_saved(*args, h0=t["h0"])
    same(y2[0, chans], want["y"], "y of the saving form")
    same(h2[0, chans], want["h"], "h of the saving form")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d-d%d-L%d" % s)
@pytest.mark.parametrize("name", ["dy", "dh"])
def test_gradient(name, shape, N, dtype):
    import vision_mamba_selective_amd as vms
    t = inputs(shape, N, dtype)
    t["u"] = t["u"].abs()
    spoil(t, name, shape[2] * 2 // 3)
    say("case infinite %s gradient %s %d %s" % (name, shape, N, dtype))
    chans = [0, CH, shape[1] - 1]
    want = definition(t, chans)
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], None)
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"])
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"])
    assert torch.isinf(want["du"][1]).any() and torch.isfinite(want["du"][0]).all()
    for k in ("du", "ddelta", "dz", "dh0"):
        same(g[k][0, chans], want[k], k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("batch", [2, 3000], ids=["one row a thread", "four rows a thread"])
@pytest.mark.parametrize("name", ["u", "delta", "h0"])
def test_step(name, batch, N, dtype):
    import vision_mamba_selective_amd as vms
    t = inputs((batch, 37, 1), N, dtype)
    spoil(t, name, 0)
    say("case infinite %s step %d %d %s" % (name, batch, N, dtype))
    chans = [0, CH, 36]
    want = definition(t, chans)
    col = lambda k: t[k][:, :, 0]      # noqa: E731
    h = t["h0"].clone()
    y = vms.s6_scan_step(*(col(k).contiguous() for k in ("u", "delta", "z", "B", "C")), t["A"], t["D"], None, h)
    assert torch.isinf(want["y"][1]).all()
    same(y[0, chans], want["y"][:, 0], "y")
    same(h[0, chans], want["h"], "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [5, 16])
@pytest.mark.parametrize("dim", [37, 16], ids=["channels to spare", "whole groups"])
@pytest.mark.parametrize("lengths", [None, [50, 33]], ids=["full", "ragged"])
@pytest.mark.parametrize("name", ["u", "dy", "dh", "h0"])
def test_gradient_sums(name, lengths, dim, N, dtype):
    """dB, dC and dA with an infinity in the last channel: of its tokens' sums
    over the channels only those that hold it are infinite, and padding stays
    zero, whatever the group of 16 channels and the block of 16 tokens that
    hold the last ones are filled up with."""
    import vision_mamba_selective_amd as vms
    L, ch = 61, dim - 1
    t = inputs((2, dim, L), N, dtype)
    t["u"], t["dy"], t["z"] = t["u"].abs() + 0.1, t["dy"].abs() + 0.1, t["z"].abs() + 0.1
    if name in ("h0", "dh"):
        t[name][0, ch] = INF
    else:
        t[name][0, ch, 20] = INF
    say("case infinite sums %s %s %d %d %s" % (name, lengths, dim, N, dtype))
    len_t = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], None)
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"], lengths=len_t)
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"], lengths=len_t)
    d = {k: ref.f64(v) for k, v in t.items()}
    dB, dC, dA = torch.zeros(2, N, L, dtype=ref.F64), torch.zeros(2, N, L, dtype=ref.F64), torch.zeros(dim, N, dtype=ref.F64)
    step = torch.logaddexp(d["delta"], torch.zeros_like(d["delta"]))
    gy = d["dy"] * d["z"] * torch.sigmoid(d["z"])
    for b, n in enumerate(ref.row_lengths(lengths, 2, L)):
        hs = [d["h0"][b]]
        for i in range(n):
            hs.append(torch.exp(step[b, :, i, None] * d["A"]) * hs[-1] + (step[b, :, i] * d["u"][b, :, i])[:, None] * d["B"][b, :, i])
        lam = d["dh"][b]
        for i in reversed(range(n)):
            dC[b, :, i] = (gy[b, :, i, None] * hs[i + 1]).sum(0)
            lam = lam + gy[b, :, i, None] * d["C"][b, :, i]
            dB[b, :, i] = (lam * (step[b, :, i] * d["u"][b, :, i])[:, None]).sum(0)
            lam = torch.exp(step[b, :, i, None] * d["A"]) * lam
            dA += lam * hs[i] * step[b, :, i, None]
    assert torch.isinf(torch.cat([dB.flatten(), dC.flatten()])).any() and torch.isinf(dA[ch]).all()
    same(g["dB"], dB, "dB")
    same(g["dC"], dC, "dC")
    same(g["dA"], dA, "dA")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 37, 16])
@pytest.mark.parametrize("name", ["B", "C"])
def test_gradient_sums_of_infinite_rows(name, dim, dtype):
    """dB and dC where one entry of B or C is infinite: the lanes of a group of
    16 channels past the last one add nothing there either. All other factors
    are positive, so that the sums are infinities."""
    import vision_mamba_selective_amd as vms
    N, L, at = 7, 45, 19
    t = inputs((1, dim, L), N, dtype)
    t["u"], t["dy"] = t["u"].abs() + 0.1, t["dy"].abs() + 0.1
    t[name][0, 2, at] = INF
    say("case infinite row %s %d %s" % (name, dim, dtype))
    args = (t["u"], t["delta"], None, t["B"], t["C"], t["A"], t["D"], None)
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"])
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"])
    d = {k: ref.f64(v)[0] if v.dim() == 3 else ref.f64(v) for k, v in t.items()}
    step = torch.logaddexp(d["delta"], torch.zeros_like(d["delta"]))
    hs, dB, dC = [d["h0"]], torch.zeros(N, L, dtype=ref.F64), torch.zeros(N, L, dtype=ref.F64)
    for i in range(L):
        hs.append(torch.exp(step[:, i, None] * d["A"]) * hs[-1] + (step[:, i] * d["u"][:, i])[:, None] * d["B"][:, i])
    lam = d["dh"]
    for i in reversed(range(L)):
        dC[:, i] = (d["dy"][:, i, None] * hs[i + 1]).sum(0)
        lam = lam + d["dy"][:, i, None] * d["C"][:, i]
        dB[:, i] = (lam * (step[:, i] * d["u"][:, i])[:, None]).sum(0)
        lam = torch.exp(step[:, i, None] * d["A"]) * lam
    hit = dC if name == "B" else dB
    assert torch.isinf(hit[2]).any() and torch.isfinite(hit[:2]).all()
    same(g["dB"][0], dB, "dB")
    same(g["dC"][0], dC, "dC")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("L,lengths", [(60, None), (60, [29, 13]), (300, [299, 290]), (1100, [1100, 1001])],
                         ids=["full", "ragged", "long", "segments"])
@pytest.mark.parametrize("back", [1, 2, 9])
def test_convolution_sums(back, L, lengths, W, dtype):
    """dw of the linear convolution with an infinity `back` tokens before a
    row's end: only the taps that meet it at a token of the row are infinite."""
    import vision_mamba_selective_amd as vms
    g = torch.Generator().manual_seed(L + W)
    dim, ch = 11, 3
    x, dy = (torch.randn(2, dim, L, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    w = (torch.rand(dim, W, generator=g) + 0.5).cuda()
    n = L if lengths is None else lengths[0]
    x[0, ch, n - back] = INF
    say("case infinite convolution sums %d %s %d %s" % (back, lengths, W, dtype))
    len_t = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    got = vms.s6_causal_conv_grad(x, w, None, dy, lengths=len_t, silu=False)
    y, _ = vms.s6_causal_conv(x, w, lengths=len_t, silu=False)
    d, dyd, wd = ref.f64(x), ref.f64(dy), ref.f64(w)
    dw, dx, yd = torch.zeros(dim, W, dtype=ref.F64), torch.zeros_like(d), torch.zeros_like(d)
    for b, m in enumerate(ref.row_lengths(lengths, 2, L)):
        line = torch.cat([torch.zeros(dim, W - 1, dtype=ref.F64), d[b, :, :m]], dim=1)
        for j in range(W):
            dw[:, j] += (dyd[b, :, :m] * line[:, j:j + m]).sum(1)
            yd[b, :, :m] += wd[:, j, None] * line[:, j:j + m]
            k = W - 1 - j
            dx[b, :, :m - k] += wd[:, j, None] * dyd[b, :, k:m]
    assert int(torch.isinf(dw).sum()) == min(back, W)
    same(got["dw"], dw, "dw")
    same(got["dx"], dx, "dx")
    same(y, yd, "y")
