"""The causal mixer and beam search as a program uses them: the example model,
HIP graphs, streams, workloads at full size, offsets past 32 bits, and what the
Python layer refuses."""
import importlib.util
import os

import pytest
import torch

import causal_ref as ref
from gpu_util import say
from test_gpu_causal import close, make

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("causal_lm", os.path.join(ROOT, "examples", "causal_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_learns(lm):
    say("case example training")
    losses = lm.train(lm.init(), 60)
    assert losses[-1] < 0.6 * losses[0], (losses[0], losses[-1])


def test_beam_search_scores_are_the_sequences_log_probabilities(lm):
    """Decoding with states from a ragged prompt batch, beams forking as they
    go: each beam's score equals the log-probability of its tokens computed by
    the whole-sequence forward pass, and beam 0 of one beam is the greedy path.
    Both sides are fp32 sums of 7 log-probabilities of magnitude up to 10
    through a few hundred roundings: 2e-4."""
    p = lm.init(seed=3)
    lm.train(p, 20)
    g = torch.Generator().manual_seed(5)
    t = lm.progressions(5, 16, g)
    lengths = torch.tensor([3, 16, 1, 7, 12], dtype=torch.int32).cuda()
    say("case example beam search")
    out, scores = lm.beam_search(p, t, lengths, 4, 7)
    one, _ = lm.beam_search(p, t, lengths, 1, 7)
    for i in range(5):
        n = int(lengths[i])
        for k in range(4):
            seq = torch.cat([t[i, :n], out[i, k].long()])[None]
            with torch.no_grad():
                logp = torch.log_softmax(lm.forward(p, seq)[0].double(), dim=1)
            want = sum(float(logp[n - 1 + j, seq[0, n + j]]) for j in range(7))
            assert abs(float(scores[i, k]) - want) < 2e-4, (i, k, float(scores[i, k]), want)
        assert (scores[i].diff() <= 0).all()
        seq = t[i, :n]
        for j in range(7):
            with torch.no_grad():
                nxt = lm.forward(p, seq[None])[0, -1].argmax()
            assert int(nxt) == int(one[i, 0, j])
            seq = torch.cat([seq, nxt[None]])


def test_graph_replays():
    """A captured decode step, selection and reorder, replayed with eager work
    and synchronizations between: every replay equals the eager result."""
    import vision_mamba_selective_amd as vms
    say("case graph")
    batch, beams, dim, N, W, V = 3, 4, 40, 16, 4, 9000
    n = batch * beams
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s, d=torch.float32: torch.randn(*s, generator=g).to(d).cuda()   # noqa: E731
    x, u, delta, z, B, C = rnd(n, dim), rnd(n, dim), rnd(n, dim), rnd(n, dim), rnd(n, N), rnd(n, N)
    w, bias, A, D, dtb = rnd(dim, W), rnd(dim), -rnd(dim, N).abs(), rnd(dim), rnd(dim)
    window, h = rnd(2 * n, dim, W - 1), rnd(2 * n, dim, N)
    so = torch.arange(n, 2 * n, dtype=torch.int32).cuda()
    logits, scores = rnd(batch, beams, V), rnd(batch, beams)
    state = rnd(2, n, 300)
    lx = rnd(2, dim, 700)
    lB, lC = rnd(2, N, 700), rnd(2, N, 700)

    def all_of_it():
        s, p, t = vms.beam_select(logits, scores)
        si = p.flatten()
        yc = vms.s6_conv_step(x, w, bias, window, slot_in=si, slot_out=so)
        ys = vms.s6_scan_step(u, delta, z, B, C, A, D, dtb, h, slot_in=si, slot_out=so)
        out = vms.beam_reorder(state, p, out=torch.empty_like(state))
        c, _ = vms.s6_causal_conv(lx, w, bias)
        y, hl, saved = vms.s6_causal_scan_saved(c, lx, lx, lB, lC, A, D, dtb)
        gr = vms.s6_causal_scan_grad(c, lx, lx, lB, lC, A, D, dtb, saved, lx)
        gc = vms.s6_causal_conv_grad(lx, w, bias, gr["du"])
        return [s, p, t, yc, ys, window.clone(), h.clone(), out, c, y, hl] + [v for v in list(gr.values()) + list(gc.values()) if v is not None]

    eager = [v.clone() for v in all_of_it()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of_it()
    for r in range(5):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, eager)):
            assert torch.equal(a, b), (r, i)
        again = all_of_it()
        assert all(torch.equal(a, b) for a, b in zip(again, eager)), r


def test_side_stream():
    """Calls follow the current stream: work queued before them on a side stream is seen, the default stream's is not waited for."""
    import vision_mamba_selective_amd as vms
    say("case side stream")
    t = make(81, "f32", 2, 40, 500, 16, 4, None, True, False)
    args = (t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    want = vms.s6_causal_scan(t["u"], *args, h0=t["h0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        u = torch.full_like(t["u"], float("nan"))
        for _ in range(20):
            u.copy_(t["u"])
        got = vms.s6_causal_scan(u, *args, h0=t["h0"])
        v = [a.clone() for a in got]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(v, want))


# batch, dim, L, shortest: the repository's workloads and shapes that take each form of the scan
FULL = [(8, 768, 4097, 2049), (1, 1536, 16385, 16385), (64, 768, 197, 1), (1, 384, 197, 197), (2, 96, 3000, 0), (512, 100, 33, 33)]


@pytest.mark.parametrize("shape", FULL, ids=lambda s: "b%d-d%d-L%d" % s[:3])
def test_full_size(shape):
    """Every form at its own size; the float64 reference recomputes sampled
    rows and channels from copies of exactly those."""
    import vision_mamba_selective_amd as vms
    batch, dim, L, short = shape
    lengths = None if short == L else [L - (L - short) * i // max(1, batch - 1) for i in range(batch)]
    t = make(91, "bf16", batch, dim, L, 16, 4, lengths, True, False)
    say("case full size %s" % (shape,))
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    kw = dict(h0=t["h0"], lengths=t["lengths"])
    y, h, saved = vms.s6_causal_scan_saved(*args, **kw)
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    y2, h2 = vms.s6_causal_scan(*args, **kw)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    b = batch // 2
    chans = sorted({0, dim // 2 + 1, dim - 1})
    n = L if lengths is None else max(0, min(L, lengths[b]))
    cut = lambda v: ref.f64(v[b:b + 1][:, chans]).nan_to_num(nan=0.0).requires_grad_()   # noqa: E731
    leaves = [cut(t["u"]), cut(t["delta"]), cut(t["z"]), ref.f64(t["B"][b:b + 1]).nan_to_num(nan=0.0),
              ref.f64(t["C"][b:b + 1]).nan_to_num(nan=0.0)] + \
             [ref.f64(t[k][chans]).requires_grad_() for k in ("A", "D", "dt_bias")] + [cut(t["h0"])]
    ry, rh = ref.scan(*leaves, [n])
    close(y[b:b + 1][:, chans], ry.detach(), "y")
    close(h[b:b + 1][:, chans], rh.detach(), "h")
    wrt = [leaves[i] for i in (0, 1, 2, 8)]
    want = ref.gradients([ry, rh], [cut(t["dy"]).detach(), cut(t["dh"]).detach()], wrt)
    for k, r in zip(("du", "ddelta", "dz", "dh0"), want):
        close(g[k][b:b + 1][:, chans], r, k)


@pytest.mark.parametrize("shape", [(3, 130, 700), (1, 200, 1500), (40, 48, 65)], ids=lambda s: "b%d-d%d-L%d" % s)
def test_sums_over_channels_and_rows(shape):
    """dB, dC (over many channels), dA, dD, ddt_bias, dw, dbias (over many rows
    and tokens) against torch's own float64 sums of the per-channel terms: the
    reference runs the recurrence for all channels at once."""
    import vision_mamba_selective_amd as vms
    batch, dim, L = shape
    t = make(101, "f32", batch, dim, L, 16, 4, None, True, False)
    say("case sums %s" % (shape,))
    args = (t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"])
    _, _, saved = vms.s6_causal_scan_saved(*args, h0=t["h0"])
    g = vms.s6_causal_scan_grad(*args, saved, t["dy"], dh=t["dh"], h0=t["h0"])
    gc = vms.s6_causal_conv_grad(t["x"], t["w"], t["bias"], t["dy"], window=t["window"], dwindow=t["dwindow"])
    d = {k: (None if v is None else ref.f64(v)) for k, v in t.items()}
    x = d["delta"] + d["dt_bias"][:, None]
    step = torch.logaddexp(x, torch.zeros_like(x))
    h, hs = d["h0"], []
    for i in range(L):
        h = torch.exp(step[:, :, i, None] * d["A"]) * h + (step * d["u"])[:, :, i, None] * d["B"][:, None, :, i]
        hs.append(h)
    gy = d["dy"] * d["z"] * torch.sigmoid(d["z"])
    lam = d["dh"]
    dB, dC, dA = torch.zeros_like(d["B"]), torch.zeros_like(d["C"]), torch.zeros_like(d["A"])
    dx = torch.zeros_like(x)
    for i in reversed(range(L)):
        dC[:, :, i] = (gy[:, :, i, None] * hs[i]).sum(1)
        lam = lam + gy[:, :, i, None] * d["C"][:, None, :, i]
        dB[:, :, i] = (lam * (step * d["u"])[:, :, i, None]).sum(1)
        back = lam * torch.exp(step[:, :, i, None] * d["A"])
        q = back * (hs[i - 1] if i else d["h0"])
        dA += (q * step[:, :, i, None]).sum(0)
        dx[:, :, i] = ((q * d["A"]).sum(-1) + d["u"][:, :, i] * (lam * d["B"][:, None, :, i]).sum(-1)) * torch.sigmoid(x[:, :, i])
        lam = back
    for k, r in (("dB", dB), ("dC", dC), ("dA", dA), ("dD", (gy * d["u"]).sum((0, 2))), ("ddt_bias", dx.sum((0, 2))), ("dh0", lam)):
        close(g[k], r, k)
    leaves = [d[k].requires_grad_() for k in ("x", "w", "bias", "window")]
    ry, rw = ref.conv(leaves[0], leaves[1], leaves[2], leaves[3], None)
    want = ref.gradients([ry, rw], [d["dy"], d["dwindow"]], leaves)
    for k, r in zip(("dx", "dw", "dbias", "dwindow"), want):
        close(gc[k], r, k)


def test_offsets_past_32_bits():
    """Inputs whose batch stride and pools whose slots lie past 2^32 bytes and
    2^31 elements give what compact copies give."""
    import vision_mamba_selective_amd as vms
    say("case long offsets")
    t = make(111, "bf16", 2, 20, 70, 16, 4, [70, 33], False, False)
    far = (1 << 31) + 64
    big = torch.empty(far + 64 * 70, dtype=torch.bfloat16, device="cuda")

    def away(v, k):
        w = big[k:].as_strided(v.shape, (far, 70, 1))
        w.copy_(v)
        return w
    rest = (t["A"], t["D"], t["dt_bias"])
    u = away(t["u"], 0)
    a = vms.s6_causal_scan(u, t["delta"], t["z"], t["B"], t["C"], *rest, lengths=t["lengths"])
    b = vms.s6_causal_scan(t["u"], t["delta"], t["z"], t["B"], t["C"], *rest, lengths=t["lengths"])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(vms.s6_causal_conv(u, t["w"], t["bias"], lengths=t["lengths"])[0],
                       vms.s6_causal_conv(t["u"], t["w"], t["bias"], lengths=t["lengths"])[0])
    del big, u
    # 9,000 slots of 16,384 channels: 2.4e9 values of h
    dim, slots = 16384, 9000
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    h = torch.empty(slots, dim, 16, device="cuda")
    window = torch.empty(slots, dim, 3, device="cuda")
    used = [8990, 8991, 0]
    for s in used:
        h[s], window[s] = rnd(dim, 16), rnd(dim, 3)
    sh, sw = h[used].clone(), window[used].clone()
    x, B, C, A, w = rnd(2, dim), rnd(2, 16), rnd(2, 16), -rnd(dim, 16).abs(), rnd(dim, 4)
    ids = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()   # noqa: E731
    p = (vms.s6_scan_step(x, x, x, B, C, A, None, None, h, slot_in=ids(8990, 0), slot_out=ids(8995, 8996)),
         vms.s6_conv_step(x, w, None, window, slot_in=ids(8990, 0), slot_out=ids(8995, 8996)), h[8995:8997], window[8995:8997])
    ch, cw = torch.zeros(5, dim, 16, device="cuda"), torch.zeros(5, dim, 3, device="cuda")
    ch[:3], cw[:3] = sh, sw
    q = (vms.s6_scan_step(x, x, x, B, C, A, None, None, ch, slot_in=ids(0, 2), slot_out=ids(3, 4)),
         vms.s6_conv_step(x, w, None, cw, slot_in=ids(0, 2), slot_out=ids(3, 4)), ch[3:], cw[3:])
    assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_python_refusals():
    import vision_mamba_selective_amd as vms
    say("case refusals")
    t = make(121, "f32", 2, 8, 20, 16, 4, None, True, False)
    good = dict(u=t["u"], delta=t["delta"], z=t["z"], B=t["B"], C=t["C"], A=t["A"], Dskip=t["D"], dt_bias=t["dt_bias"])

    def scan(**kw):
        a = dict(good)
        extra = {k: kw.pop(k) for k in list(kw) if k not in a}
        a.update(kw)
        return vms.s6_causal_scan(**a, **extra)
    scan()
    bad = [dict(u=t["u"].half()), dict(delta=t["delta"].bfloat16()), dict(B=t["B"][:, :8]), dict(A=t["A"].double()), dict(A=t["A"].t()),
           dict(z=t["z"][:, :, :19]), dict(u=t["u"].transpose(1, 2).contiguous().transpose(1, 2)), dict(dt_bias=t["dt_bias"].cpu()),
           dict(h0=t["h0"].bfloat16()), dict(lengths=torch.tensor([1, 2]).cuda()), dict(lengths=torch.tensor([1], dtype=torch.int32).cuda()),
           dict(out=torch.empty(2, 8, 20, device="cuda").bfloat16()), dict(h_out=t["h0"][:1]), dict(Dskip=t["D"][:4]), dict(A=None)]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            scan(**kw)
    from vision_mamba_selective_amd._native import ScanError
    with pytest.raises(ScanError):
        scan(out=t["u"])                                             # the output may not be an input
    with pytest.raises(ScanError):
        scan(h0=t["h0"], h_out=t["h0"])
    y, h, saved = vms.s6_causal_scan_saved(**good)
    with pytest.raises(ValueError):
        vms.s6_causal_scan_grad(t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"], saved[:64], t["dy"])
    with pytest.raises(ValueError):
        vms.s6_causal_scan_grad(t["u"], t["delta"], t["z"], t["B"], t["C"], t["A"], t["D"], t["dt_bias"], None, t["dy"])
    with pytest.raises(ValueError):
        vms.s6_causal_conv(t["x"], t["w"], window=t["window"][:, :, :2].contiguous())
    pool = torch.zeros(2, 8, 16, device="cuda")
    two = lambda v: v[:, :, 0]     # noqa: E731
    with pytest.raises((ValueError, ScanError)):
        vms.s6_scan_step(two(t["u"]), two(t["delta"]), None, two(t["B"]), two(t["C"]), t["A"], None, None, pool)
    c = lambda v: v[:, :, 0].contiguous()     # noqa: E731
    with pytest.raises(TypeError):
        vms.s6_scan_step(c(t["u"]), c(t["delta"]), None, c(t["B"]), c(t["C"]), t["A"], None, None, pool,
                         slot_in=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ScanError):
        vms.s6_scan_step(c(t["u"]), c(t["delta"]), None, c(t["B"]), c(t["C"]), t["A"], None, None, pool[:1])
    logits, scores = torch.zeros(2, 3, 9, device="cuda"), torch.zeros(2, 3, device="cuda")
    for kw in (dict(scores=scores[:, :2]), dict(scores=scores.double()), dict(logits=logits.half()), dict(logits=logits.transpose(1, 2)),
               dict(done=scores), dict(done=scores.bool()), dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            vms.beam_select(**{**dict(logits=logits, scores=scores), **kw})
    with pytest.raises(ScanError):
        vms.beam_select(logits, scores, done=scores.bool(), eos=9)
    state, parent = torch.zeros(2, 6, 4, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for args in ((state, parent.long()), (state, parent[:1]), (state.transpose(1, 2), parent), (state[:, :, :2], parent)):
        with pytest.raises((TypeError, ValueError)):
            vms.beam_reorder(*args)
    with pytest.raises(ValueError):
        vms.beam_reorder(state, parent, out=state.bfloat16())
