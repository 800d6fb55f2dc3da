"""GPU parity of the gated linear recurrence (gated_scan, its gradient and its
single-token form) with float64 references. Bounds as in test_gpu_causal.py: a
state is a sum of terms that passed through at most a few hundred fp32
roundings before they decayed, a bf16 result adds its rounding."""
import math

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import DT, close

pytestmark = pytest.mark.gpu


def make(seed, dtype, batch, dim, L, lengths, carried, strided, gate=True):
    """Inputs on the GPU; padding of ragged rows holds NaN."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def rnd(*s, d=torch.float32):
        return torch.randn(*s, generator=g).to(d).cuda()

    def act():
        if strided:                    # rows of a wider tensor, a span of longer rows
            return rnd(batch, dim + 3, L + 5, d=dt)[:, 2:2 + dim, 3:3 + L]
        return rnd(batch, dim, L, d=dt)

    t = dict(x=act(), r=act(), i=act(), z=act() if gate else None, dy=act())
    t["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    if lengths is not None:
        for name in ("x", "r", "i", "z", "dy"):
            if t[name] is not None:
                for b, n in enumerate(ref.row_lengths(lengths, batch, L)):
                    t[name][b, :, n:] = float("nan")
    top = 0.9 + 0.099 * torch.rand(dim, generator=g)             # decays at a full gate
    t["lam"] = torch.log(torch.expm1(-torch.log(top) / 8)).cuda()
    t["h0"] = rnd(batch, dim) if carried else None
    t["dh"] = rnd(batch, dim) if carried else None
    return t


def doubles(t):
    out = {}
    for k, v in t.items():
        out[k] = v if v is None or not v.is_floating_point() else ref.f64(v).nan_to_num(nan=0.0).requires_grad_()
    return out


# batch, dim, L, lengths, carried, strided: every form (16 lanes, 64, four waves, eight) and its edges
CASES = [
    (1, 1, 1, None, False, False),
    (2, 17, 37, None, True, False),
    (3, 16, 128, [128, 0, 1], True, False),
    (2, 5, 129, [3, 129], False, True),
    (4, 33, 256, [256, 255, 129, 2], True, True),
    (1, 40, 257, None, False, True),
    (2, 19, 511, [-4, 999], True, False),
    (2, 18, 512, [0, 0], True, False),
    (3, 7, 1024, [513, 1024, 512], True, False),
    (1, 3, 1025, [1024], False, False),
    (2, 20, 2100, [2100, 1100], True, True),
    (2, 300, 2049, [2049, 1], True, False),
    (3, 700, 300, [300, 129, 0], True, True),
    (2, 1024, 384, None, True, False),
    (2, 1030, 1025, [1025, 513], True, False),
    (1, 3, 4097, None, True, False),
    (1, 2, 9000, [8193], True, True),
]
IDS = ["b%d-d%d-L%d-%s" % (c[0], c[1], c[2], "ragged" if c[3] else "full") for c in CASES]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False], ids=["gate", "nogate"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_scan_and_gradient(case, gate, dtype):
    import vision_mamba_selective_amd as vms
    t = make(7 + case[2], dtype, *case, gate=gate)
    say("case gated %s gate=%s %s" % (case, gate, dtype))
    args, kw = (t["x"], t["r"], t["i"], t["lam"]), dict(z=t["z"], h0=t["h0"], lengths=t["lengths"])
    y, h = vms.gated_scan(*args, **kw)
    y2, h2, saved = vms.gated_scan_saved(*args, **kw)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    g = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    again = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    d = doubles(t)
    leaves = [d[k] for k in ("x", "r", "i", "lam", "z", "h0")]
    ry, rh = ref.gated(*leaves, case[3])
    close(y, ry.detach(), "y")
    close(h, rh.detach(), "h")
    want = ref.gradients([ry, rh], [d["dy"].detach(), None if d["dh"] is None else d["dh"].detach()], leaves)
    for name, w in zip(("dx", "dr", "di", "dlam", "dz", "dh0"), want):
        if w is None:
            assert g[name] is None
            continue
        close(g[name], w, name)
        assert torch.equal(g[name], again[name]), name


@pytest.mark.parametrize("lam", [-120.0, -60.0, -15.0, 0.0, 5.0, 40.0])
def test_decays_from_none_to_full(lam):
    """From decays that fp32 cannot tell from 1 to ones that leave nothing, in
    the recurrence and its gradient. With lam = -120 no state changes. Decays
    are held at 2^-126 or more, so what true decays take below that times a
    state of at most 2^6 stays somewhere below 2^-120."""
    import vision_mamba_selective_amd as vms
    say("case gated lam=%g" % lam)
    t = make(3, "f32", 2, 5, 300, None, True, False)
    t["lam"] = torch.full((5,), lam).cuda()
    args, kw = (t["x"], t["r"], t["i"], t["lam"]), dict(z=t["z"], h0=t["h0"])
    y, h, saved = vms.gated_scan_saved(*args, **kw)
    g = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    d = doubles(t)
    leaves = [d[k] for k in ("x", "r", "i", "lam", "z", "h0")]
    ry, rh = ref.gated(*leaves, None)
    close(y, ry.detach(), "y")
    close(h, rh.detach(), "h")
    want = ref.gradients([ry, rh], [d["dy"].detach(), d["dh"].detach()], leaves)
    for name, w in zip(("dx", "dr", "di", "dlam", "dz", "dh0"), want):
        if lam < -87 and name in ("dx", "di", "dr", "dlam"):
            # s below 2^-126 counts as zero: the results are below the root of that
            assert float(g[name].abs().max()) < 1e-17 and float(w.abs().max()) < 1e-17, name
        elif name == "dh0":
            gone = w.abs() < 2.0 ** -120
            assert float(g[name].cpu()[gone].abs().sum()) <= 10 * 2.0 ** -120
            close(g[name].cpu().masked_fill(gone, 0.0), w.masked_fill(gone, 0.0), name)
        else:
            close(g[name], w, name)


def test_gradient_against_differences():
    """Central differences of the fp32 forward pass along one direction for all
    inputs together, step 2^-6. The loss is a sum of 2 x 4 x 140 products of
    magnitude about 1, each off by at most 16 x 2^-24 of its size: 2e-6 x 33
    (their root sum of squares), over 2 steps of 2^-6 that is 2e-3; the third
    derivative adds 2^-12 / 6 times a few tens: 4e-3."""
    import vision_mamba_selective_amd as vms
    say("case gated differences")
    t = make(5, "f32", 2, 4, 140, None, True, False)
    keys = ("x", "r", "i", "lam", "z", "h0")
    g = torch.Generator().manual_seed(9)
    way = {k: torch.randn(t[k].shape, generator=g).cuda() / 30 for k in keys}

    def loss(e):
        v = {k: t[k] + e * way[k] for k in keys}
        y, h = vms.gated_scan(v["x"], v["r"], v["i"], v["lam"], z=v["z"], h0=v["h0"])
        return float((y.double() * t["dy"].double()).sum() + (h.double() * t["dh"].double()).sum())
    _, _, saved = vms.gated_scan_saved(t["x"], t["r"], t["i"], t["lam"], z=t["z"], h0=t["h0"])
    got = vms.gated_scan_grad(t["x"], t["r"], t["i"], t["lam"], saved, t["dy"], z=t["z"], dh=t["dh"], h0=t["h0"])
    along = sum(float((got["d" + k].double() * way[k].double()).sum()) for k in keys)
    e = 2.0 ** -6
    assert abs((loss(e) - loss(-e)) / (2 * e) - along) < 6e-3, (along, (loss(e) - loss(-e)) / (2 * e))


@pytest.mark.parametrize("L", [5, 140, 600, 1500, 5000])
def test_non_finite_inputs_reach_only_what_they_are_part_of(L):
    """An infinite state stays infinite under any decay, also where the decays'
    product underflows; NaN at a token reaches that channel's later tokens and,
    in the gradient, what depends on it; other channels and rows keep their bits."""
    import vision_mamba_selective_amd as vms
    say("case gated non-finite %d" % L)
    t = make(21, "f32", 2, 3, L, None, True, False)
    t["lam"] = torch.tensor([0.0, 3.0, 20.0]).cuda()
    args = lambda: (t["x"], t["r"], t["i"], t["lam"])           # noqa: E731
    clean_y, clean_h, clean_saved = vms.gated_scan_saved(*args(), h0=t["h0"])
    clean = vms.gated_scan_grad(*args(), clean_saved, t["dy"], h0=t["h0"], dh=t["dh"])
    h0 = t["h0"].clone()
    h0[0, 2] = math.inf
    y, h = vms.gated_scan(*args(), h0=h0)
    assert bool((y[0, 2] == math.inf).all()) and float(h[0, 2]) == math.inf
    assert torch.equal(y[1], clean_y[1]) and torch.equal(y[0, :2], clean_y[0, :2]) and torch.equal(h[1], clean_h[1])
    dh = t["dh"].clone()
    dh[1, 2] = -math.inf
    g = vms.gated_scan_grad(*args(), clean_saved, t["dy"], h0=t["h0"], dh=dh)
    assert float(g["dh0"][1, 2]) == -math.inf
    assert torch.equal(g["dx"][0], clean["dx"][0]) and torch.equal(g["dx"][1, :2], clean["dx"][1, :2])
    at = L // 2
    for name in ("x", "r", "i"):
        old = t[name]
        t[name] = old.clone()
        t[name][1, 1, at] = math.nan
        y, h, saved = vms.gated_scan_saved(*args(), h0=t["h0"])
        assert bool(y[1, 1, at:].isnan().all()) and bool(h[1, 1].isnan())
        assert torch.equal(y[1, 1, :at], clean_y[1, 1, :at])
        assert torch.equal(y[0], clean_y[0]) and torch.equal(y[1, ::2], clean_y[1, ::2])
        g = vms.gated_scan_grad(*args(), saved, t["dy"], h0=t["h0"], dh=t["dh"])
        assert bool(g["dlam"][1].isnan()) and not bool(g["dlam"][::2].isnan().any())
        assert torch.equal(g["dx"][0], clean["dx"][0]) and torch.equal(g["dx"][1, ::2], clean["dx"][1, ::2])
        if name == "r":
            assert bool(g["dx"][1, 1, :at].isnan().all())       # its decay is NaN
        else:
            assert torch.equal(g["dh0"], clean["dh0"])          # the adjoint does not read x or i
        t[name] = old


# batch, dim, slots, gate
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,gate", [(1, 1, True), (3, 7, False), (5, 64, True), (2, 1537, True), (70, 33, False)])
def test_step(batch, dim, gate, dtype):
    """Slots that are read together, written elsewhere, kept and left out; rows of a wider tensor."""
    import vision_mamba_selective_amd as vms
    say("case gated step %s" % ((batch, dim, gate, dtype),))
    t = make(batch + dim, dtype, 1, dim, 1, None, False, False)
    g = torch.Generator().manual_seed(dim)
    wide = torch.randn(batch, 4 * dim + 3, generator=g).to(DT[dtype]).cuda()
    x, r, i, z = (wide[:, 1 + k * dim:1 + (k + 1) * dim] for k in range(4))
    pool = torch.randn(3 * batch, dim, generator=g).cuda()
    si = torch.randint(0, batch, (batch,), generator=g).to(torch.int32)
    so = (batch + torch.randperm(2 * batch, generator=g)[:batch]).to(torch.int32)
    if batch > 2:
        si[0], so[1], so[2] = -1, 3 * batch, -7
    h = pool.clone()
    y = vms.gated_scan_step(x, r, i, t["lam"], h, z=z if gate else None, slot_in=si.cuda(), slot_out=so.cuda())
    want_h, want_y = ref.f64(pool), torch.zeros(batch, dim, dtype=torch.float64)
    written = torch.zeros(3 * batch, dtype=torch.bool)
    for b in range(batch):
        a, o = int(si[b]), int(so[b])
        if not (0 <= a < 3 * batch and 0 <= o < 3 * batch):
            continue
        one = [ref.f64(v[b])[None, :, None] for v in (x, r, i)]
        ry, rh = ref.gated(*one, ref.f64(t["lam"]), ref.f64(z[b])[None, :, None] if gate else None, ref.f64(pool[a])[None], None)
        want_h[o], want_y[b] = rh[0], ry[0, :, 0]
        written[o] = True
    close(h, want_h, "h")
    close(y, want_y, "y")
    assert torch.equal(h.cpu()[~written], pool.cpu()[~written])
    # without slots row b keeps to slot b, in place
    h = pool.clone()
    y = vms.gated_scan_step(x, r, i, t["lam"], h, z=z if gate else None)
    ry, rh = ref.gated(*(ref.f64(v)[:, :, None] for v in (x, r, i)), ref.f64(t["lam"]), ref.f64(z)[:, :, None] if gate else None,
                       ref.f64(pool[:batch]), None)
    close(h[:batch], rh, "h in place")
    close(y, ry[:, :, 0], "y in place")
    assert torch.equal(h[batch:], pool[batch:])


def test_steps_continue_a_prompt():
    """A prompt's last tokens one at a time, from the state of what is before them."""
    import vision_mamba_selective_amd as vms
    say("case gated continue")
    t = make(8, "f32", 3, 21, 300, None, True, False)
    cut = lambda v, a, b: v[:, :, a:b]                            # noqa: E731
    acts = [t[k] for k in ("x", "r", "i", "z")]
    y, h = vms.gated_scan(*acts[:3], t["lam"], z=acts[3], h0=t["h0"])
    _, state = vms.gated_scan(*(cut(v, 0, 290) for v in acts[:3]), t["lam"], z=cut(acts[3], 0, 290), h0=t["h0"])
    for k in range(290, 300):
        one = vms.gated_scan_step(*(v[:, :, k].contiguous() for v in acts[:3]), t["lam"], state, z=acts[3][:, :, k].contiguous())
        close(one, ref.f64(y[:, :, k]), "y %d" % k)
    close(state, ref.f64(h), "h")


def test_autograd_matches_the_calls():
    import vision_mamba_selective_amd as vms
    say("case gated autograd")
    t = make(13, "bf16", 2, 9, 700, [700, 31], True, True)
    leaf = {k: t[k].detach().clone().requires_grad_() for k in ("x", "r", "i", "lam", "z", "h0")}
    y, h = vms.gated_scan_autograd(leaf["x"], leaf["r"], leaf["i"], leaf["lam"], z=leaf["z"], h0=leaf["h0"], lengths=t["lengths"])
    torch.autograd.backward([y, h], [t["dy"], t["dh"]])
    args, kw = (t["x"], t["r"], t["i"], t["lam"]), dict(z=t["z"], h0=t["h0"], lengths=t["lengths"])
    _, _, saved = vms.gated_scan_saved(*args, **kw)
    g = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    for k in leaf:
        assert torch.equal(leaf[k].grad, g["d" + k]), k
    y, h = vms.gated_scan_autograd(leaf["x"], leaf["r"], leaf["i"], leaf["lam"])
    assert torch.autograd.grad(h.sum(), leaf["lam"])[0].shape == (9,)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(y.float().sum(), leaf["lam"], create_graph=True)[0].sum(), leaf["x"])
