"""The gated recurrence, the norm and the vocabulary loss as a program uses them:
together, in HIP graphs, on side streams and threads, with workspaces of exactly
the stated size, on tensors that are written in place, at full size, with
offsets past 32 bits; and what the Python layer refuses."""
import gc
import threading

import pytest
import torch

import model_ref as ref
from gpu_util import say
from test_gpu_causal import DT, close
from test_gpu_gated import doubles, make

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


def i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Layers:
    """Two layers of norm, recurrence and projection, a norm and a loss: everything of a training step but the autograd graph."""

    def __init__(self, seed, dtype=torch.float32, batch=3, dim=40, L=150, vocab=700):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, d=dtype: torch.randn(*s, generator=g).to(d).cuda()         # noqa: E731
        self.x, self.lens = rnd(batch, dim, L), i32(*[max(1, L - 37 * k) for k in range(batch)])
        self.w = [1 + 0.1 * rnd(dim, d=torch.float32) for _ in range(3)]
        self.gates = [(rnd(batch, dim, L), rnd(batch, dim, L), rnd(dim, d=torch.float32) - 4) for _ in range(2)]
        self.dy = rnd(batch, dim, L)
        self.head = rnd(vocab, dim) * 0.2
        self.target = torch.randint(-20, vocab, (batch * L,), generator=g).cuda()
        self.pool, self.si, self.so = rnd(2 * batch, dim, d=torch.float32), i32(*range(batch)), i32(*range(batch, 2 * batch))

    def step(self):
        import vision_mamba_selective_amd as vms
        out, stream, kept = [], self.x, []
        y, _ = vms.rms_norm(stream, self.w[0], lengths=self.lens)
        for k, (r, i, lam) in enumerate(self.gates):
            y, h, saved = vms.gated_scan_saved(y, r, i, lam, z=r, lengths=self.lens)
            y, stream = vms.rms_norm(y, self.w[k + 1], residual=stream, lengths=self.lens)
            out += [y, h, stream]
            kept.append((stream, saved))
        rows = y.transpose(1, 2).reshape(-1, y.shape[1])
        loss, lse = vms.vocab_loss(rows, self.head, self.target)
        g = vms.vocab_loss_grad(rows, self.head, self.target, lse, torch.ones_like(loss))
        dy = g["dx"].view(y.shape[0], -1, y.shape[1]).transpose(1, 2).contiguous()
        n = vms.rms_norm_grad(stream, self.w[2], dy, dsum=self.dy, lengths=self.lens)
        r, i, lam = self.gates[1]
        s = vms.gated_scan_grad(self.x, r, i, lam, kept[1][1], n["dx"], z=r, lengths=self.lens)
        one = vms.gated_scan_step(self.x[:, :, 0].contiguous(), r[:, :, 0].contiguous(), i[:, :, 0].contiguous(), lam, self.pool,
                                  slot_in=self.si, slot_out=self.so)
        token, _ = vms.rms_norm(one, self.w[0])
        return out + [loss, lse, g["dx"], g["dW"], n["dx"], n["dw"], one, token, self.pool.clone()] + [v for v in s.values() if v is not None]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_replays(dtype):
    """A captured run of them together, replayed with eager work and synchronizations between: every replay equals the eager result."""
    say("case model graph %s" % dtype)
    m = Layers(1, DT[dtype])
    eager = [v.clone() for v in m.step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.step()
    for r in range(5):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), r
        assert all(torch.equal(a, b) for a, b in zip(m.step(), eager)), r


def test_captured_backward_pass():
    """A training step through the autograd forms, captured as torch asks: after
    a run on a side stream, with no eager graph of the same leaves alive."""
    import vision_mamba_selective_amd as vms
    say("case model captured backward")
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()            # noqa: E731
    x, w, r, i, lam, W = rnd(2, 48, 130), rnd(48), rnd(2, 48, 130), rnd(2, 48, 130), rnd(48), rnd(300, 48)
    leaves = [x, w, r, i, lam, W]
    target = torch.randint(-20, 300, (260,), generator=g).cuda()
    dloss = torch.ones(260).cuda()

    def step():
        y, _ = vms.rms_norm_autograd(x, w)
        y, _ = vms.gated_scan_autograd(y, r, i, lam, z=r)
        y, _ = vms.rms_norm_autograd(y, None, residual=x)
        loss = vms.vocab_loss_autograd(y.transpose(1, 2).reshape(260, 48), W, target)
        return [loss.detach()] + list(torch.autograd.grad(loss, leaves, grad_outputs=dloss))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [v.clone() for v in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    # an eager graph of the same leaves: refused before anything is captured
    for call in (lambda: vms.rms_norm_autograd(x, w)[0], lambda: vms.rms_norm_autograd(x.detach(), None, residual=x)[0],
                 lambda: vms.gated_scan_autograd(x.detach(), r.detach(), i.detach(), lam)[0],
                 lambda: vms.vocab_loss_autograd(x.detach()[0].t().contiguous(), W, target[:130])):
        alive = call()
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="eager graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
        del alive
    gc.collect()                     # the exceptions' frames hold the refused calls' graphs
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), k
        assert all(torch.equal(a, b) for a, b in zip(step(), eager)), k


def test_two_graphs_share_a_workspace():
    """Both graphs' calls use one workspace; replayed in turn on one stream each gives its own result."""
    import vision_mamba_selective_amd as vms
    say("case model shared workspace")
    cases, size = [], 0
    for seed, tokens in ((1, 300), (2, 130)):
        g = torch.Generator().manual_seed(seed)
        x, W = torch.randn(tokens, 33, generator=g).bfloat16().cuda(), torch.randn(500, 33, generator=g).bfloat16().cuda()
        cases.append((x, W, torch.randint(0, 500, (tokens,), generator=g).cuda(), torch.ones(tokens).cuda()))
        size = max(size, vms.vocab_workspace_bytes(1, tokens, 33, 500, torch.bfloat16), vms.vocab_workspace_bytes(0, tokens, 33, 500, torch.bfloat16))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def both(x, W, t, d):
        loss, lse = vms.vocab_loss(x, W, t, workspace=ws)
        g = vms.vocab_loss_grad(x, W, t, lse, d, workspace=ws)
        return loss, g["dx"], g["dW"]
    want = [[v.clone() for v in both(*c)] for c in cases]
    graphs, got = [], []
    for c in cases:
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(both(*c))
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        ws.fill_(0xA5)
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in set(order):
            assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), order


def test_two_threads_two_streams():
    say("case model threads")
    ms = [Layers(5), Layers(6, torch.bfloat16, batch=2, dim=65, L=300)]
    alone = [[v.clone() for v in m.step()] for m in ms]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[k] = ms[k].step()
            s.synchronize()
        except Exception as e:
            errors.append(e)
    th = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in th:
        t.start()
    for t in th:
        t.join()
    assert not errors, errors
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[k], alone[k])), k


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_calls_run_on_the_tensors_device():
    import vision_mamba_selective_amd as vms
    say("case model other device")
    g = torch.Generator().manual_seed(3)
    x, w, W = torch.randn(9, 40, generator=g), torch.rand(40, generator=g), torch.randn(70, 40, generator=g)

    def all_of(d):
        y, _ = vms.rms_norm(x.to(d), w.to(d))
        loss, lse = vms.vocab_loss(y, W.to(d), torch.arange(9, device=d))
        s, h = vms.gated_scan(*(x[:, :, None].expand(9, 40, 5).contiguous().to(d) for _ in range(3)), w.to(d))
        return [v.cpu() for v in (y, loss, lse, s, h)]
    with torch.cuda.device(0):
        assert all(torch.equal(a, b) for a, b in zip(all_of("cuda:1"), all_of("cuda:0")))


def guarded(n):
    whole = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole[:n], whole[n:]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_workspaces_of_the_stated_size(dtype):
    """What stands behind a workspace keeps its bytes."""
    import vision_mamba_selective_amd as vms
    from vision_mamba_selective_amd import _native as nat
    rnd = lambda *s: torch.randn(*s, device="cuda").to(dtype)                      # noqa: E731
    for batch, dim, L in ((1, 1, 1), (3, 17, 128), (2, 40, 129), (1, 3, 513), (2, 5, 4097), (700, 3, 300)):
        say("case gated workspace %s" % ((batch, dim, L),))
        x, lam = rnd(batch, dim, L), torch.zeros(dim, device="cuda")
        saved, gs = guarded(vms.gated_workspace_bytes(nat.VS_GATED_SAVED, batch, dim, L))
        ws, gw = guarded(vms.gated_workspace_bytes(nat.VS_GATED_GRAD, batch, dim, L))
        vms.gated_scan_saved(x, x, x, lam, saved=saved)
        vms.gated_scan_grad(x, x, x, lam, saved, x, workspace=ws)
        assert bool((gs == 0xA5).all()) and bool((gw == 0xA5).all())
    for shape in ((1, 1), (3, 70), (2051, 24), (513, 520), (600, 2100), (2, 30, 33), (3, 900, 65)):
        say("case norm workspace %s" % (shape,))
        x = rnd(*shape)
        ws, guard = guarded(vms.norm_workspace_bytes(shape[0], shape[1], shape[2] if len(shape) == 3 else 1))
        vms.rms_norm_grad(x, torch.ones(shape[1], device="cuda"), x, workspace=ws)
        assert bool((guard == 0xA5).all())
    for tokens, dim, vocab in ((1, 1, 1), (5, 7, 33), (130, 30, 257), (1000, 130, 40), (40, 300, 3001), (2100, 33, 700), (1030, 40, 12500)):
        say("case vocab workspace %s" % ((tokens, dim, vocab),))
        x, W, t = rnd(tokens, dim), rnd(vocab, dim), torch.randint(0, vocab, (tokens,), device="cuda")
        ws, guard = guarded(vms.vocab_workspace_bytes(nat.VS_VOCAB_LOSS, tokens, dim, vocab, dtype))
        _, lse = vms.vocab_loss(x, W, t, workspace=ws)
        wg, gg = guarded(vms.vocab_workspace_bytes(nat.VS_VOCAB_GRAD, tokens, dim, vocab, dtype))
        vms.vocab_loss_grad(x, W, t, lse, torch.ones(tokens, device="cuda"), workspace=wg)
        assert bool((guard == 0xA5).all()) and bool((gg == 0xA5).all())


def writers():
    """Every call that writes a caller's tensor: its name, the call, and the tensors that it writes."""
    import vision_mamba_selective_amd as vms
    rnd = lambda *s: torch.randn(*s, device="cuda")                                # noqa: E731
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")                # noqa: E731
    x, lam, row = rnd(2, 8, 40), rnd(8), rnd(2, 8)
    y, h, s, yr, pool = rnd(2, 8, 40), rnd(2, 8), u8(vms.gated_workspace_bytes(0, 2, 8, 40)), rnd(2, 8), rnd(2, 8)
    wg, wn = u8(vms.gated_workspace_bytes(1, 2, 8, 40)), u8(vms.norm_workspace_bytes(2, 8, 40))
    W, t = rnd(9, 8), torch.arange(2).cuda()
    wl, wv = (u8(vms.vocab_workspace_bytes(k, 2, 8, 9, torch.float32)) for k in range(2))
    total = rnd(2, 8, 40)
    yield "scan", lambda: vms.gated_scan(x, x, x, lam, out=y, h_out=h), [y, h]
    yield "saved", lambda: vms.gated_scan_saved(x, x, x, lam, out=y, h_out=h, saved=s), [y, h, s]
    yield "grad", lambda: vms.gated_scan_grad(x, x, x, lam, s, x, workspace=wg), [wg]
    yield "step", lambda: vms.gated_scan_step(row, row, row, lam, pool, out=yr), [pool, yr]
    yield "norm", lambda: vms.rms_norm(x, lam, residual=y, out=total, sum_out=y), [total, y]
    yield "norm grad", lambda: vms.rms_norm_grad(x, lam, x, workspace=wn), [wn]
    yield "loss", lambda: vms.vocab_loss(row, W, t, workspace=wl), [wl]
    yield "loss grad", lambda: vms.vocab_loss_grad(row, W, t, h[:, 0].contiguous(), h[:, 1].contiguous(), workspace=wv), [wv]


def test_written_tensors_get_a_new_version_and_no_gradient():
    for name, call, written in writers():
        say("case written %s" % name)
        before = [v._version for v in written]
        call()
        assert all(v._version > b for v, b in zip(written, before)), name
        for v in written:
            if v.is_floating_point():
                v.requires_grad_()
                with pytest.raises(ValueError, match="requires a gradient"):
                    call()
                with torch.no_grad():
                    call()
                v.requires_grad_(False)


# batch, dim, L, shortest: sizes that take each form of the recurrence
FULL = [(8, 768, 4097, 2049), (1, 1536, 16385, 16385), (64, 768, 197, 1), (1, 384, 197, 197), (2, 96, 3000, 0), (512, 100, 33, 33), (1, 24, 16385, 1)]


@pytest.mark.parametrize("shape", FULL, ids=lambda s: "b%d-d%d-L%d" % s[:3])
def test_gated_full_size(shape):
    """The float64 reference recomputes sampled rows and channels; dlam is the sum of what batches of one row give."""
    import vision_mamba_selective_amd as vms
    batch, dim, L, short = shape
    lengths = None if short == L else [L - (L - short) * i // max(1, batch - 1) for i in range(batch)]
    t = make(91, "bf16", batch, dim, L, lengths, True, False)
    say("case gated full size %s" % (shape,))
    args, kw = (t["x"], t["r"], t["i"], t["lam"]), dict(z=t["z"], h0=t["h0"], lengths=t["lengths"])
    y, h, saved = vms.gated_scan_saved(*args, **kw)
    g = vms.gated_scan_grad(*args, saved, t["dy"], dh=t["dh"], **kw)
    b, chans = batch // 2, sorted({0, dim // 2 + 1, dim - 1})
    n = L if lengths is None else max(0, min(L, lengths[b]))
    d = doubles({k: t[k][b:b + 1][:, chans] for k in ("x", "r", "i", "z", "h0", "dy", "dh")} | {"lam": t["lam"][chans]})
    leaves = [d[k] for k in ("x", "r", "i", "lam", "z", "h0")]
    ry, rh = ref.gated(*leaves, [n])
    close(y[b:b + 1][:, chans], ry.detach(), "y")
    close(h[b:b + 1][:, chans], rh.detach(), "h")
    wrt = [leaves[k] for k in (0, 1, 2, 4, 5)]
    want = ref.gradients([ry, rh], [d["dy"].detach(), d["dh"].detach()], wrt)
    for k, r in zip(("dx", "dr", "di", "dz", "dh0"), want):
        close(g[k][b:b + 1][:, chans], r, k)
    if 1 < batch <= 8:
        total = 0
        for k in range(batch):
            part = [v[k:k + 1] for v in args[:3]]
            one = dict(z=t["z"][k:k + 1], h0=t["h0"][k:k + 1], lengths=None if lengths is None else t["lengths"][k:k + 1])
            _, _, s = vms.gated_scan_saved(*part, t["lam"], **one)
            total = total + vms.gated_scan_grad(*part, t["lam"], s, t["dy"][k:k + 1], dh=t["dh"][k:k + 1], **one)["dlam"].double()
        close(g["dlam"], total.cpu(), "dlam")


def test_offsets_past_32_bits():
    """Tensors whose batch strides, slots and rows lie past 2^32 bytes and 2^31 elements give what compact copies give."""
    import vision_mamba_selective_amd as vms
    say("case model long offsets")
    t = make(3, "bf16", 2, 20, 70, [70, 33], False, False)
    far = (1 << 31) + 64
    big = torch.zeros(far + 64 * 70, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 20, 70), (far, 70, 1))
    x.copy_(t["x"])
    for a, b in ((vms.gated_scan(v, t["r"], t["i"], t["lam"], lengths=t["lengths"]) for v in (x, t["x"])),
                 (vms.rms_norm(v, None, residual=t["r"], lengths=t["lengths"]) for v in (x, t["x"]))):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    rows = x[:, :, 0]
    W, target = torch.randn(50, 20).bfloat16().cuda(), torch.tensor([3, 7]).cuda()
    rows = big.as_strided((2, 20), (far, 1))
    # an x_stride of 2^28 or more is refused, not truncated
    from vision_mamba_selective_amd._native import ScanError
    with pytest.raises(ScanError):
        vms.vocab_loss(rows, W, target)
    near = big.as_strided((2, 20), ((1 << 28) - 8, 1))
    near.copy_(t["x"][:, :, 0])
    assert all(torch.equal(p, q) for p, q in zip(vms.vocab_loss(near, W, target), vms.vocab_loss(near.contiguous(), W, target)))
    del big, x, rows, near
    dim, slots = 1 << 17, 17000                                    # 2.2e9 states
    h = torch.empty(slots, dim, device="cuda")
    h[[16990, 0]] = torch.randn(2, dim, device="cuda")
    small = torch.cat([h[[16990, 0]], torch.zeros(2, dim, device="cuda")])
    r, lam = torch.randn(2, dim, device="cuda"), torch.randn(dim, device="cuda")
    a = vms.gated_scan_step(r, r, r, lam, h, slot_in=i32(16990, 0), slot_out=i32(16995, 16996))
    b = vms.gated_scan_step(r, r, r, lam, small, slot_in=i32(0, 1), slot_out=i32(2, 3))
    assert torch.equal(a, b) and torch.equal(h[16995:16997], small[2:])


def test_python_refusals():
    import vision_mamba_selective_amd as vms
    from vision_mamba_selective_amd._native import ScanError
    say("case model refusals")
    t = make(2, "f32", 2, 8, 20, None, True, False)
    good = dict(x=t["x"], r=t["r"], i=t["i"], lam=t["lam"], z=t["z"], h0=t["h0"])
    refused = (TypeError, ValueError, ScanError)
    for kw in (dict(x=t["x"].half()), dict(r=t["r"].bfloat16()), dict(i=t["i"][:, :, :19]), dict(lam=t["lam"].double()), dict(lam=t["lam"][:4]),
               dict(z=t["z"].cpu()), dict(h0=t["h0"].bfloat16()), dict(x=t["x"].transpose(1, 2).contiguous().transpose(1, 2)), dict(rate="8"),
               dict(rate=-1.0), dict(rate=None), dict(lengths=torch.tensor([1, 2]).cuda()), dict(out=t["x"]), dict(h0=t["h0"], h_out=t["h0"]),
               dict(lam=None), dict(x=t["x"][:0], r=t["r"][:0], i=t["i"][:0], z=None, h0=None)):
        with pytest.raises(refused):
            vms.gated_scan(**{**good, **kw})
    vms.gated_scan(**good, rate=0)
    row = t["x"][:, :, 0].contiguous()
    for kw in (dict(h=torch.zeros(1, 8).cuda()), dict(h=torch.zeros(2, 9).cuda()), dict(slot_in=torch.zeros(2).long().cuda()), dict(x=t["x"][:, :, 0])):
        with pytest.raises(refused):
            vms.gated_scan_step(**{**dict(x=row, r=row, i=row, lam=t["lam"], h=torch.zeros(2, 8).cuda()), **kw})
    w = torch.ones(8).cuda()
    for kw in (dict(x=t["x"].double()), dict(x=t["x"][0, 0]), dict(w=w.bfloat16()), dict(w=w[:4]), dict(residual=t["r"].bfloat16()),
               dict(residual=t["r"][:, :, :5]), dict(eps=-1.0), dict(eps="x"), dict(lengths=torch.tensor([1.0, 2.0]).cuda()), dict(out=t["x"]),
               dict(sum_out=t["r"]), dict(x=t["x"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(refused):
            vms.rms_norm(**{**dict(x=t["x"], w=w), **kw})
    x, W, target = torch.zeros(5, 8).cuda(), torch.zeros(30, 8).cuda(), torch.zeros(5).long().cuda()
    for kw in (dict(x=x.half()), dict(x=x[None]), dict(W=W[:, :7]), dict(W=W.bfloat16()), dict(W=W.t().contiguous().t()), dict(target=target.float()),
               dict(target=target[:4]), dict(target=target.cpu()), dict(x=x[:0], target=target[:0]), dict(W=W[:0]), dict(x=x.t().contiguous().t()),
               dict(workspace=torch.zeros(8, dtype=torch.uint8).cuda())):
        with pytest.raises(refused):
            vms.vocab_loss(**{**dict(x=x, W=W, target=target), **kw})
    loss, lse = vms.vocab_loss(x, W, target)
    for kw in (dict(lse=lse[:4]), dict(dloss=lse.double()), dict(lse=None), dict(dloss=lse[:, None])):
        with pytest.raises(refused):
            vms.vocab_loss_grad(**{**dict(x=x, W=W, target=target, lse=lse, dloss=lse), **kw})
