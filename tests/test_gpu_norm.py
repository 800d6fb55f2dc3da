"""GPU parity of the norm with the residual's addition and of its gradient with
float64 references.

Bounds: a result is a product of four factors, one of them from a sum of up to
8,192 squares taken over at most 64 partial sums in turn: fewer than 100
roundings of 2^-24 relative each, within F32_TOL (rms + |ref|) of
test_gpu_causal.py (400 x 2^-24). ds is the difference of q w dy and s q^3 mean(w
dy s), which cancel (all of it where dim = 1), so its bound goes by the first of
them: by Cauchy and Schwarz the second's rms over a token is at most as large:
100 x 2^-24 times that rms and its own more. dw adds up to
70,000 terms in at most 600 steps, of errors like a random walk's. A bf16
result adds its rounding. s is rounded once: equal to the reference's bits."""
import math

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import BF16_TOL, DT, F32_TOL, close

pytestmark = pytest.mark.gpu
EPS = 1e-5


def make(seed, dtype, batch, dim, L, lengths, strided):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def rnd(*s, d=torch.float32):
        return torch.randn(*s, generator=g).to(d).cuda()

    def act():
        if strided:
            return rnd(batch, dim + 3, L + 5, d=dt)[:, 2:2 + dim, 3:3 + L]
        return rnd(batch, dim, L, d=dt)
    t = dict(x=act(), residual=act(), dy=act(), dsum=act(), w=1 + 0.3 * rnd(dim))
    t["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    if lengths is not None:
        for name in ("x", "residual", "dy", "dsum"):
            for b, n in enumerate(ref.row_lengths(lengths, batch, L)):
                t[name][b, :, n:] = float("nan")
    return t


def close_difference(got, want, part):
    """close() with the error that the parts of a difference may have added."""
    got, bf16 = got.cpu().double(), got.dtype == torch.bfloat16
    tol = F32_TOL * (want.square().mean().sqrt() + want.abs()) + part + (BF16_TOL * (want.abs() + part) if bf16 else 0.0)
    assert torch.isfinite(got).all() and bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


def check(t, lengths, added, weighted, rows, dtype):
    """rows: the tensors go in as [rows, dim]."""
    import vision_mamba_selective_amd as vms
    flat = (lambda v: v[:, :, 0]) if rows else (lambda v: v)
    w = t["w"] if weighted else None
    kw = dict(eps=EPS, lengths=t["lengths"])
    y, s = vms.rms_norm(flat(t["x"]), w, residual=flat(t["residual"]) if added else None, **kw)
    g = vms.rms_norm_grad(s, w, flat(t["dy"]), dsum=flat(t["dsum"]) if added else None, **kw)
    again = vms.rms_norm_grad(s, w, flat(t["dy"]), dsum=flat(t["dsum"]) if added else None, **kw)
    clean = {k: ref.f64(t[k]).nan_to_num(nan=0.0) for k in ("x", "residual", "dy", "dsum", "w")}
    leaf = clean["x"].requires_grad_()
    lw = clean["w"].requires_grad_() if weighted else None
    ry, rs = ref.norm(leaf, lw, clean["residual"] if added else None, lengths, EPS, DT[dtype])
    full = (lambda v: v[:, :, None]) if rows else (lambda v: v)
    close(full(y), ry.detach(), "y")
    if added:
        assert torch.equal(ref.f64(full(s)), rs.detach()), "s"
    want = ref.gradients([ry, rs] if added else [ry], [clean["dy"], clean["dsum"]], [leaf, lw])
    q = 1 / torch.sqrt(rs.detach().square().mean(1, keepdim=True) + EPS)
    part = q * clean["dy"] * (clean["w"].detach()[:, None] if weighted else 1.0)
    part = 100 * 2.0 ** -24 * (part.abs() + part.square().mean(1, keepdim=True).sqrt() * (1 + (rs.detach() * q).abs()))
    close_difference(full(g["dx"]), want[0], part)
    if weighted:
        close(g["dw"], want[1], "dw")
        assert torch.equal(g["dw"], again["dw"])
    else:
        assert g["dw"] is None
    assert torch.equal(g["dx"], again["dx"])


# batch, dim, L, lengths, strided
CASES = [
    (1, 1, 2, None, False),
    (2, 3, 33, None, True),
    (3, 24, 31, [31, 0, 1], False),
    (2, 129, 64, [63, 33], True),
    (1, 768, 197, None, False),
    (2, 769, 65, [65, 32], True),
    (1, 1537, 40, None, False),
    (2, 1700, 37, [5, 37], False),
    (5, 7, 500, [500, 499, 40, -3, 999], False),
    (1, 3500, 33, None, False),
    (3, 400, 129, [129, 64, 128], True),
    (2, 24, 72, [72, 65], False),
    (2, 500, 73, None, True),
    (3, 900, 68, [66, 68, 1], False),
    (40, 100, 1001, None, False),
    (36, 200, 961, [961 - 30 * k for k in range(36)], True),
]
IDS = ["b%d-d%d-L%d-%s" % (c[0], c[1], c[2], "ragged" if c[3] else "full") for c in CASES]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("added,weighted", [(True, True), (False, True), (True, False)], ids=["add", "plain", "noweight"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_prompts(case, added, weighted, dtype):
    say("case norm %s %s %s %s" % (case, added, weighted, dtype))
    check(make(case[1], dtype, *case), case[3], added, weighted, False, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("added,weighted", [(True, True), (False, True), (True, False)], ids=["add", "plain", "noweight"])
@pytest.mark.parametrize("rows,dim,lengths", [
    (1, 1, None), (1, 384, None), (3, 255, [1, 0, 7]), (5, 512, None), (7, 257, None), (66, 1536, None), (2, 2049, [0, 1]), (3, 4096, None),
    (2, 4097, None), (3, 8192, None), (2, 8191, None), (2051, 24, None), (2600, 30, None), (520, 1030, None)], ids=str)
def test_rows(rows, dim, lengths, added, weighted, dtype):
    say("case norm rows %d %d %s %s %s" % (rows, dim, added, weighted, dtype))
    check(make(dim, dtype, rows, dim, 1, lengths, False), lengths, added, weighted, True, dtype)


def test_layouts_of_one_token():
    """[rows, dim], [rows, dim, 1] and the last token of prompts (channel
    stride above 1) agree within their bound; row strides are free."""
    import vision_mamba_selective_amd as vms
    say("case norm layouts")
    g = torch.Generator().manual_seed(2)
    long = torch.randn(6, 40, 9, generator=g).cuda()
    w = torch.rand(40, generator=g).cuda()
    last = long[:, :, -1:]
    dense = last.contiguous()
    want, _ = ref.norm(ref.f64(dense), ref.f64(w), None, None, EPS, torch.float32)
    wide = torch.zeros(6, 50).cuda()
    wide[:, 5:45] = dense[:, :, 0]
    for x in (last, dense, dense[:, :, 0], wide[:, 5:45], dense[:1].expand(6, 40, 1)[:1]):
        y, s = vms.rms_norm(x, w, eps=EPS)
        assert s is x and y.shape == x.shape
        close(y.reshape(-1, 40), want[:y.shape[0], :, 0], "y")


def test_stream_in_place():
    """sum_out may be the residual: the same bits as into a new tensor."""
    import vision_mamba_selective_amd as vms
    for shape in ((4, 900, 70), (5, 700), (2, 3300, 33)):
        say("case norm in place %s" % (shape,))
        g = torch.Generator().manual_seed(1)
        x, res, w = (torch.randn(*v, generator=g).cuda() for v in (shape, shape, shape[1:2]))
        y, s = vms.rms_norm(x, w, residual=res)
        stream = res.clone()
        y2, s2 = vms.rms_norm(x, w, residual=stream, sum_out=stream)
        assert s2 is stream or s2.data_ptr() == stream.data_ptr()
        assert torch.equal(y, y2) and torch.equal(s, stream)
        with pytest.raises(Exception, match="overlap"):
            vms.rms_norm(x, w, residual=res, sum_out=x)
        with pytest.raises(Exception, match="overlap"):
            vms.rms_norm(x, w, residual=res, out=res)


@pytest.mark.parametrize("shape", [(2, 50, 40), (3, 50)], ids=["prompts", "rows"])
def test_non_finite_and_extreme_tokens_stay_alone(shape):
    """A token with a NaN or an infinity does not change the others; a token of
    zeros gives zeros (eps > 0), and large and small values keep their norm."""
    import vision_mamba_selective_amd as vms
    say("case norm non-finite %s" % (shape,))
    g = torch.Generator().manual_seed(4)
    x, dy, w = (torch.randn(*v, generator=g).cuda() for v in (shape, shape, shape[1:2]))
    y0, _ = vms.rms_norm(x, w)
    g0 = vms.rms_norm_grad(x, w, dy)
    at = (1, slice(None), 33) if len(shape) == 3 else (1, slice(None))
    others = torch.ones(shape, dtype=torch.bool).cuda()
    others[at] = False
    for v in (math.nan, math.inf, -math.inf):
        bad = x.clone()
        bad[at][7] = v
        y, _ = vms.rms_norm(bad, w)
        d = vms.rms_norm_grad(bad, w, dy)
        assert torch.equal(y[others], y0[others]) and torch.equal(d["dx"][others], g0["dx"][others])
        assert bool(y[at].isnan().any())
    scaled = x.clone()
    scaled[at] = 0
    assert float(vms.rms_norm(scaled, w)[0][at].abs().max()) == 0
    assert bool(torch.isfinite(vms.rms_norm_grad(scaled, w, dy)["dx"]).all())
    for v in (2.0 ** 40, 2.0 ** -40):
        scaled = x.clone()
        scaled[at] = x[at] * v
        y, _ = vms.rms_norm(scaled, w, eps=0.0)
        want, _ = ref.norm(ref.f64(scaled.view(shape[0], shape[1], -1)), ref.f64(w), None, None, 0.0, torch.float32)
        close(y.view(shape[0], shape[1], -1), want, "scaled")


def test_gradient_against_differences():
    """Central differences along one direction, step 2^-6: 2 x 30 x 40 products
    of magnitude 1 with errors of a few 2^-24 (root sum of squares 49 x 4 x
    2^-24 = 1.2e-5), over 2^-5: 4e-4; the third derivative adds 2^-12 / 6 times a
    few units."""
    import vision_mamba_selective_amd as vms
    say("case norm differences")
    g = torch.Generator().manual_seed(6)
    x, res, dy, dsum = (torch.randn(2, 30, 40, generator=g).cuda() for _ in range(4))
    w = torch.rand(30, generator=g).cuda() + 0.5
    way = torch.randn(2, 30, 40, generator=g).cuda() / 30
    ww = torch.randn(30, generator=g).cuda() / 30

    def loss(e):
        y, s = vms.rms_norm(x + e * way, w + e * ww, residual=res)
        return float((y.double() * dy.double()).sum() + (s.double() * dsum.double()).sum())
    _, s = vms.rms_norm(x, w, residual=res)
    d = vms.rms_norm_grad(s, w, dy, dsum=dsum)
    along = float((d["dx"].double() * way.double()).sum() + (d["dw"].double() * ww.double()).sum())
    e = 2.0 ** -6
    assert abs((loss(e) - loss(-e)) / (2 * e) - along) < 2e-3


def test_autograd_matches_the_calls():
    import vision_mamba_selective_amd as vms
    say("case norm autograd")
    for shape, lengths in (((2, 70, 45), [45, 9]), ((9, 70), None)):
        g = torch.Generator().manual_seed(3)
        x, res, dy, ds = (torch.randn(*shape, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
        w = torch.rand(70, generator=g).cuda()
        lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
        lx, lr, lw = (v.clone().requires_grad_() for v in (x, res, w))
        y, s = vms.rms_norm_autograd(lx, lw, residual=lr, lengths=lens)
        torch.autograd.backward([y, s], [dy, ds])
        y0, s0 = vms.rms_norm(x, w, residual=res, lengths=lens)
        d = vms.rms_norm_grad(s0, w, dy, dsum=ds, lengths=lens)
        assert torch.equal(y, y0) and torch.equal(s, s0)
        assert torch.equal(lx.grad, d["dx"]) and torch.equal(lr.grad, d["dx"]) and torch.equal(lw.grad, d["dw"])
        lx.grad = None
        y, s = vms.rms_norm_autograd(lx, None, lengths=lens)
        assert s is lx
        (y * dy).sum().backward()
        assert torch.equal(lx.grad, vms.rms_norm_grad(x, None, dy, lengths=lens)["dx"])
        with pytest.raises(RuntimeError):
            y, _ = vms.rms_norm_autograd(lx, lw)
            torch.autograd.grad(torch.autograd.grad(y.float().sum(), lx, create_graph=True)[0].float().sum(), lw)
