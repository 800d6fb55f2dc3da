"""GPU parity of the causal mixer (s6_causal_conv, s6_causal_scan, their
single-token forms and their gradients) with float64 references.

Bounds, set from the arithmetic: a state is a sum of terms that each passed
through at most a few hundred fp32 roundings (2^-24 relative each, the
hardware exp2's argument and result among them) before they decayed, so an
fp32 result stays within a few hundred times 2^-24 of its typical size: |got -
ref| <= F32_TOL (rms + |ref|), F32_TOL = 400 x 2^-24. Sums over tokens, rows or
channels of such values obey the same bound. A bf16 result adds the round to
8 significant bits: 2^-8 |ref|."""
import pytest
import torch

import causal_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

F32_TOL = 400 * 2.0 ** -24
BF16_TOL = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(got, want, what):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g = got.detach().to("cpu", torch.float64)
    assert torch.isfinite(want).all(), what
    assert torch.isfinite(g).all(), "%s: non-finite values" % what
    rms = float(want.square().mean().sqrt()) if want.numel() else 0.0
    tol = F32_TOL * (rms + want.abs())
    if got.dtype == torch.bfloat16:
        tol = tol + BF16_TOL * want.abs()
    bad = (g - want).abs() > tol
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d beyond the bound; first at %s: got %r ref %r" % (
            what, int(bad.sum()), bad.numel(), i, float(g[i]), float(want[i])))


def make(seed, dtype, batch, dim, L, N, W, lengths, carried, strided, gate=True, params=True):
    """Inputs on the GPU; padding of ragged rows holds NaN."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def rnd(*s, scale=1.0, d=torch.float32):
        return (torch.randn(*s, generator=g) * scale).to(d)

    def act(rows, scale=1.0):
        if strided:                    # rows of a wider tensor, a span of longer rows
            big = rnd(batch, rows + 3, L + 5, scale=scale, d=dt).cuda()
            return big[:, 2:2 + rows, 3:3 + L]
        return rnd(batch, rows, L, scale=scale, d=dt).cuda()

    t = dict(x=act(dim), u=act(dim), delta=act(dim, 0.5), z=act(dim) if gate else None, B=act(N), C=act(N), dy=act(dim))
    t["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    if lengths is not None:
        for name in ("x", "u", "delta", "z", "B", "C", "dy"):
            if t[name] is not None:
                for b, n in enumerate(ref.row_lengths(lengths, batch, L)):
                    t[name][b, :, n:] = float("nan")
    t["A"] = (-(torch.arange(N) + 1.0) * (0.5 + torch.rand(dim, N, generator=g))).cuda()
    t["D"] = rnd(dim).cuda() if params else None
    t["dt_bias"] = (rnd(dim) * 0.5 - 2).cuda() if params else None
    t["w"] = (rnd(dim, W) / W ** 0.5).cuda()
    t["bias"] = rnd(dim).cuda() if params else None
    t["window"] = rnd(batch, dim, W - 1, d=dt).cuda() if carried else None
    t["h0"] = rnd(batch, dim, N, scale=0.5).cuda() if carried else None
    t["dh"] = rnd(batch, dim, N).cuda() if carried else None
    t["dwindow"] = rnd(batch, dim, W - 1, d=dt).cuda() if carried else None
    return t


def doubles(t):
    """The same values in float64 on the CPU, padding as zero, leaves for autograd."""
    out = {}
    for k, v in t.items():
        if v is None or not v.is_floating_point():
            out[k] = v
            continue
        out[k] = ref.f64(v).nan_to_num(nan=0.0).requires_grad_()
    return out


# batch, dim, L, dstate, width, lengths, carried, strided
CASES = [
    (1, 1, 1, 1, 2, None, False, False),
    (2, 17, 37, 16, 4, None, True, False),
    (3, 16, 32, 16, 4, [32, 0, 1], True, False),
    (2, 5, 16, 5, 3, [3, 16], False, True),
    (4, 33, 65, 16, 4, [65, 64, 33, 2], True, True),
    (1, 40, 300, 8, 8, None, False, True),
    (2, 18, 129, 16, 2, [0, 0], True, False),
    (2, 19, 111, 12, 5, [-4, 999], True, False),
    (1, 3, 1030, 16, 6, [1029], False, False),
    (2, 20, 2100, 3, 7, [2100, 1100], True, False),
]
IDS = ["b%d-d%d-L%d-N%d-w%d-%s" % (c[0], c[1], c[2], c[3], c[4], "ragged" if c[5] else "full") for c in CASES]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("silu", [True, False], ids=["silu", "linear"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_conv(case, silu, dtype):
    import vision_mamba_selective_amd as vms
    batch, dim, L, N, W, lengths, carried, strided = case
    t = make(11 + L, dtype, *case, params=silu)
    say("case conv %s silu=%s %s" % (case, silu, dtype))
    y, wo = vms.s6_causal_conv(t["x"], t["w"], t["bias"], window=t["window"], lengths=t["lengths"], silu=silu)
    g = vms.s6_causal_conv_grad(t["x"], t["w"], t["bias"], t["dy"], window=t["window"], dwindow=t["dwindow"],
                                lengths=t["lengths"], silu=silu)
    d = doubles(t)
    ry, rw = ref.conv(d["x"], d["w"], d["bias"], d["window"], lengths, silu)
    close(y, ry.detach(), "y")
    assert torch.equal(ref.f64(wo), rw.detach())
    want = ref.gradients([ry, rw], [d["dy"].detach(), None if d["dwindow"] is None else d["dwindow"].detach()],
                         [d["x"], d["w"], d["bias"], d["window"]])
    for name, r in zip(("dx", "dw", "dbias", "dwindow"), want):
        if r is not None:
            close(g[name], r, name)
    if not carried:
        assert g["dwindow"] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False], ids=["gate", "nogate"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_scan(case, gate, dtype):
    import vision_mamba_selective_amd as vms
    batch, dim, L, N, W, lengths, carried, strided = case
    t = make(23 + L, dtype, *case, gate=gate, params=gate)
    say("case scan %s gate=%s %s" % (case, gate, dtype))
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    kw = dict(h0=t["h0"], lengths=t["lengths"])
    y, h = vms.s6_causal_scan(*args, **kw)
    y2, h2, saved = vms.s6_causal_scan_saved(*args, **kw)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    d = doubles(t)
    leaves = [d[k] for k in ("u", "delta", "z", "B", "C", "A", "D", "dt_bias", "h0")]
    ry, rh = ref.scan(*leaves, lengths)
    close(y, ry.detach(), "y")
    close(h, rh.detach(), "h")
    want = ref.gradients([ry, rh], [d["dy"].detach(), None if d["dh"] is None else d["dh"].detach()], leaves)
    for name, r in zip(("du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0"), want):
        if r is not None:
            close(g[name], r, name)
    again = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    for k in g:
        assert (g[k] is None and again[k] is None) or torch.equal(g[k], again[k]), k


def test_scan_without_softplus():
    import vision_mamba_selective_amd as vms
    case = CASES[4]
    t = make(5, "f32", *case, params=False)
    t["delta"] = t["delta"].abs() * 0.2
    say("case scan without softplus")
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], None, None)
    y, h, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"], lengths=t["lengths"], delta_softplus=False)
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"], lengths=t["lengths"], delta_softplus=False)
    d = doubles(t)
    leaves = [d[k] for k in ("u", "delta", "z", "B", "C", "A", "h0")]
    ry, rh = ref.scan(*leaves[:6], None, None, leaves[6], case[5], softplus=False)
    close(y, ry.detach(), "y")
    want = ref.gradients([ry, rh], [d["dy"].detach(), d["dh"].detach()], leaves)
    for name, r in zip(("du", "ddelta", "dz", "dB", "dC", "dA", "dh0"), want):
        close(g[name], r, name)


def test_prompt_in_two_halves_is_the_prompt():
    """The states carried from one call to the next stand for the earlier text."""
    import vision_mamba_selective_amd as vms
    batch, dim, L, N, W = 2, 20, 203, 16, 4
    t = make(31, "f32", batch, dim, L, N, W, None, True, False)
    say("case prompt in two halves")
    rest = (t["A"], t["D"], t["dt_bias"])
    u, win = vms.s6_causal_conv(t["x"], t["w"], t["bias"], window=t["window"])
    y, h = vms.s6_causal_scan(t["u"], t["delta"], t["z"], t["B"], t["C"], *rest, h0=t["h0"])
    w1, h1, us, ys = t["window"], t["h0"], [], []
    for a, b in ((0, 90), (90, 92), (92, L)):
        part = lambda k: t[k][:, :, a:b]     # noqa: E731  (spans: strided inputs)
        p, w1 = vms.s6_causal_conv(part("x"), t["w"], t["bias"], window=w1)
        us.append(p)
        q, h1 = vms.s6_causal_scan(part("u"), part("delta"), part("z"), part("B"), part("C"), *rest, h0=h1)
        ys.append(q)
    assert torch.equal(torch.cat(us, 2), u) and torch.equal(w1, win)
    close(torch.cat(ys, 2), ref.f64(y), "y")
    close(h1, ref.f64(h), "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 2), (3, 40, 16, 4), (5, 130, 5, 3), (2, 300, 16, 8), (7, 65, 10, 4)],
                         ids=lambda s: "b%d-d%d-N%d-w%d" % s)
def test_steps(shape, dtype):
    """Single tokens on pools: forks (two rows read one slot), rows without a
    slot, slots outside the pool, strided inputs."""
    import vision_mamba_selective_amd as vms
    batch, dim, N, W = shape
    g = torch.Generator().manual_seed(7 + dim)
    dt = DT[dtype]
    say("case steps %s %s" % (shape, dtype))
    slots = 2 * batch + 1
    rnd = lambda *s, d=dt: torch.randn(*s, generator=g).to(d).cuda()   # noqa: E731
    xz, bc = rnd(batch, 3 * dim + 1), rnd(batch, 2 * N + 3)
    x, u, z = xz[:, :dim], xz[:, dim:2 * dim], xz[:, 2 * dim:3 * dim]
    B, C = bc[:, 1:1 + N], bc[:, 2 + N:2 + 2 * N]
    delta = rnd(batch, dim)
    A = -(torch.rand(dim, N, generator=g) + 0.5).cuda() * 3
    D, dtb, bias = rnd(dim, d=torch.float32), rnd(dim, d=torch.float32), rnd(dim, d=torch.float32)
    w = rnd(dim, W, d=torch.float32)
    window, h = rnd(slots, dim, W - 1), rnd(slots, dim, N, d=torch.float32)
    w0, h0 = window.clone(), h.clone()
    si = [0] * batch                                  # every row forks slot 0
    so = [batch + i for i in range(batch)]
    if batch > 2:
        si[1], so[1] = -1, batch + 1
    if batch > 4:
        si[3], so[4] = slots, slots + 5
    ti, to = torch.tensor(si, dtype=torch.int32).cuda(), torch.tensor(so, dtype=torch.int32).cuda()
    yc = vms.s6_conv_step(x, w, bias, window, slot_in=ti, slot_out=to)
    ys = vms.s6_scan_step(u, delta, z, B, C, A, D, dtb, h, slot_in=ti, slot_out=to)
    want_w, want_h = ref.f64(w0), ref.f64(h0)
    for i in range(batch):
        if not (0 <= si[i] < slots and 0 <= so[i] < slots):
            assert not yc[i].any() and not ys[i].any()
            continue
        col = lambda v: ref.f64(v)[i:i + 1, :, None]   # noqa: E731
        ry, rw = ref.conv(col(x), ref.f64(w), ref.f64(bias), ref.f64(w0)[si[i]][None], None)
        close(yc[i], ry[0, :, 0], "conv y %d" % i)
        want_w[so[i]] = rw[0]
        ry, rh = ref.scan(col(u), col(delta), col(z), col(B), col(C), ref.f64(A), ref.f64(D), ref.f64(dtb), ref.f64(h0)[si[i]][None], None)
        close(ys[i], ry[0, :, 0], "scan y %d" % i)
        want_h[so[i]] = rh[0]
    assert torch.equal(ref.f64(window), want_w)
    close(h, want_h, "h")
    untouched = [s for s in range(slots) if s not in so]
    assert torch.equal(h[untouched], h0[untouched])


def test_steps_in_place_follow_the_prompt():
    """Without slots a row's state is slot b, in place: token after token gives the prompt's outputs."""
    import vision_mamba_selective_amd as vms
    batch, dim, L, N, W = 2, 37, 21, 16, 4
    t = make(41, "f32", batch, dim, L, N, W, None, True, False)
    say("case steps follow the prompt")
    u, win = vms.s6_causal_conv(t["x"], t["w"], t["bias"], window=t["window"])
    y, h = vms.s6_causal_scan(t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"], h0=t["h0"])
    pw, ph = t["window"].clone(), t["h0"].clone()
    at = lambda k, i: t[k][:, :, i].contiguous()   # noqa: E731
    for i in range(L):
        close(vms.s6_conv_step(at("x", i), t["w"], t["bias"], pw), ref.f64(u[:, :, i]), "u %d" % i)
        ys = vms.s6_scan_step(at("u", i), at("delta", i), at("z", i), at("B", i), at("C", i), t["A"], t["D"], t["dt_bias"], ph)
        close(ys, ref.f64(y[:, :, i]), "y %d" % i)
    assert torch.equal(pw, win)
    close(ph, ref.f64(h), "h")


def test_gradient_against_differences():
    """Directional derivatives: differences of the float64 forward along random
    directions equal the library's gradient times the direction. The central
    difference's own error is step^2 |f'''|, 1e-8 here; the fp32 gradient's is
    F32_TOL times the norm of gradient and direction."""
    import vision_mamba_selective_amd as vms
    case = (2, 9, 40, 16, 4, [40, 23], True, False)
    t = make(51, "f32", *case)
    say("case gradient against differences")
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"], lengths=t["lengths"])
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"], lengths=t["lengths"])
    d = {k: (v.detach() if isinstance(v, torch.Tensor) else v) for k, v in doubles(t).items()}
    names = ("u", "delta", "z", "B", "C", "A", "D", "dt_bias", "h0")
    keys = ("du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0")

    def loss(v):
        y, h = ref.scan(*[v[k] for k in names], case[5])
        return float((y * d["dy"]).sum() + (h * d["dh"]).sum())

    gen = torch.Generator().manual_seed(3)
    for name, key in zip(names, keys):
        e = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        step = 1e-4
        num = (loss({**d, name: d[name] + step * e}) - loss({**d, name: d[name] - step * e})) / (2 * step)
        grad = ref.f64(g[key])
        got = float((grad * e).sum())
        tol = F32_TOL * float(grad.norm() * e.norm()) + 1e-5 * max(1.0, abs(num))
        assert abs(got - num) <= tol, (key, got, num)


def test_autograd():
    """The differentiable ops give the library's gradients, and only where asked."""
    import vision_mamba_selective_amd as vms
    case = (2, 20, 50, 16, 4, [50, 31], True, True)
    t = make(61, "bf16", *case)
    say("case autograd")
    leaf = {k: (v.detach().clone().requires_grad_() if v is not None and v.is_floating_point() else v) for k, v in t.items()}
    u, win = vms.s6_causal_conv_autograd(leaf["x"], leaf["w"], leaf["bias"], leaf["window"], leaf["lengths"])
    y, h = vms.s6_causal_scan_autograd(u, leaf["delta"], leaf["z"], leaf["B"], leaf["C"], leaf["A"], leaf["D"], leaf["dt_bias"],
                                       leaf["h0"], leaf["lengths"])
    dy = t["dy"].nan_to_num(nan=0.0)
    torch.autograd.backward([y, h], [dy, t["dh"]])
    args = (u.detach(), t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"], lengths=t["lengths"])
    g = vms.s6_causal_scan_grad(*args, saved, dy, dh=t["dh"], h0=t["h0"], lengths=t["lengths"])
    gc = vms.s6_causal_conv_grad(t["x"], t["w"], t["bias"], g["du"], window=t["window"], lengths=t["lengths"])
    for name, want in (("delta", g["ddelta"]), ("z", g["dz"]), ("B", g["dB"].bfloat16()), ("C", g["dC"].bfloat16()),
                       ("A", g["dA"]), ("D", g["dD"]), ("dt_bias", g["ddt_bias"]), ("h0", g["dh0"]), ("x", gc["dx"]),
                       ("w", gc["dw"]), ("bias", gc["dbias"]), ("window", gc["dwindow"])):
        assert torch.equal(leaf[name].grad, want), name
    assert leaf["u"].grad is None


def test_values_that_overflow_elsewhere():
    """An infinite value at a row's token stays in its own channel's row and
    after its own token; z far below zero closes the gate to exactly zero."""
    import vision_mamba_selective_amd as vms
    t = make(71, "f32", 2, 18, 60, 16, 4, None, False, False)
    say("case infinities")
    t["u"][0, 5, 40] = float("inf")
    t["z"][1] = -1e30
    y, h = vms.s6_causal_scan(t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    fin = torch.isfinite(y[0])
    assert fin[:5].all() and fin[6:].all() and fin[5, :40].all() and not fin[5, 40]
    assert not y[1].any()
    assert torch.isfinite(h[1]).all() and not torch.isfinite(h[0, 5]).all()
