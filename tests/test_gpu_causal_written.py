"""Tensors that the causal mixer's and beam search's calls write in place, seen
from autograd: a written tensor gets a new version, so that a backward pass
that saved its former values is refused, as after torch's own in-place
operations."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
B, DIM, L, N, W, K, V = 2, 12, 40, 8, 4, 3, 50


def rnd(*s):
    return torch.randn(*s, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    """Every call that writes a caller's tensor: its name, the call, and the tensors that it writes."""
    import vision_mamba_selective_amd as vms
    from vision_mamba_selective_amd import _native as nat
    x, w, row = rnd(B, DIM, L), rnd(DIM, W), rnd(B, DIM)
    Bm, Cm, A = rnd(B, N, L), rnd(B, N, L), -rnd(DIM, N).abs()
    u8 = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device="cuda")      # noqa: E731
    ws = lambda op, inner=N: u8(vms.s6_workspace_bytes(op, B, DIM, inner, L))    # noqa: E731
    y, win, h, yr = rnd(B, DIM, L), rnd(B, DIM, W - 1), rnd(B, DIM, N), rnd(B, DIM)
    yield "conv", lambda: vms.s6_causal_conv(x, w, out=y, window_out=win), [y, win]
    wc = ws(nat.VS_S6_CONV_GRAD, W)
    yield "conv grad", lambda: vms.s6_causal_conv_grad(x, w, None, x, workspace=wc), [wc]
    pool = rnd(B, DIM, W - 1)
    yield "conv step", lambda: vms.s6_conv_step(row, w, None, pool, out=yr), [pool, yr]
    wf = ws(nat.VS_S6_SCAN)
    yield "scan", lambda: vms.s6_causal_scan(x, x, None, Bm, Cm, A, out=y, h_out=h, workspace=wf), [y, h, wf]
    sv = ws(nat.VS_S6_SAVED)
    yield "saving scan", lambda: vms.s6_causal_scan_saved(x, x, None, Bm, Cm, A, out=y, h_out=h, saved=sv, workspace=wf), [y, h, sv, wf]
    wg = ws(nat.VS_S6_GRAD)
    yield "scan grad", lambda: vms.s6_causal_scan_grad(x, x, None, Bm, Cm, A, None, None, sv, x, workspace=wg), [wg]
    hp = rnd(B, DIM, N)
    bt, ct = rnd(B, N), rnd(B, N)
    yield "scan step", lambda: vms.s6_scan_step(row, row, None, bt, ct, A, None, None, hp, out=yr), [hp, yr]
    logits, scores = rnd(B, K, V), rnd(B, K)
    out = (rnd(B, K), i32([[0] * K] * B), i32([[0] * K] * B))
    wb = u8(vms.beam_workspace_bytes(B, K, V))
    yield "select", lambda: vms.beam_select(logits, scores, out=out, workspace=wb), list(out) + [wb]
    state, parent, other = rnd(2, B * K, 5), i32([[0, 0, 1], [3, 5, 5]]), rnd(2, B * K, 5)
    yield "reorder", lambda: vms.beam_reorder(state, parent), [state]
    yield "reorder to another", lambda: vms.beam_reorder(state, parent, out=other), [other]


NAMES = ["conv", "conv grad", "conv step", "scan", "saving scan", "scan grad", "scan step", "select", "reorder", "reorder to another"]


@pytest.mark.parametrize("name", NAMES)
def test_versions(name):
    say("case versions %s" % name)
    call, written = next((c, t) for n, c, t in calls() if n == name)
    before = [t._version for t in written]
    call()
    after = [t._version for t in written]
    assert all(a > b for a, b in zip(after, before)), (before, after)


def test_all_calls_are_named():
    assert [n for n, _, _ in calls()] == NAMES


@pytest.mark.parametrize("how", ["step", "reorder", "window_out", "copy_"])
def test_an_overwritten_window_is_refused(how):
    """The convolution's backward reads the window again: what stands there now is not what the forward pass read."""
    import vision_mamba_selective_amd as vms
    say("case overwritten window %s" % how)
    x, w, window = rnd(B, DIM, L).requires_grad_(), rnd(DIM, W).requires_grad_(), rnd(B, DIM, W - 1)
    y, _ = vms.s6_causal_conv_autograd(x, w, None, window)
    y.sum().backward()                                        # untouched: accepted
    y, _ = vms.s6_causal_conv_autograd(x, w, None, window)
    with torch.no_grad():
        if how == "step":
            vms.s6_conv_step(rnd(B, DIM), w, None, window)
        elif how == "reorder":
            vms.beam_reorder(window[None], i32([[1, 0]]))      # a view has its base's version
        elif how == "window_out":
            vms.s6_causal_conv(x, w, window_out=window)
        else:
            window.copy_(rnd(B, DIM, W - 1))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_overwritten_states_are_refused():
    import vision_mamba_selective_amd as vms
    say("case overwritten states")
    u, d, Bm, Cm = rnd(B, DIM, L).requires_grad_(), rnd(B, DIM, L), rnd(B, N, L), rnd(B, N, L)
    A, h = -rnd(DIM, N).abs(), rnd(B, DIM, N)
    y, _ = vms.s6_causal_scan_autograd(u, d, None, Bm, Cm, A, h0=h)
    vms.s6_scan_step(rnd(B, DIM), rnd(B, DIM), None, rnd(B, N), rnd(B, N), A, None, None, h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_inference_tensors_are_written():
    """They have no version and no backward pass can save them: a prompt's states from inference mode are decoded on outside it."""
    import vision_mamba_selective_amd as vms
    say("case inference tensors")
    w, row, A = rnd(DIM, W), rnd(B, DIM), -rnd(DIM, N).abs()
    plain = rnd(B, DIM, W - 1)
    with torch.inference_mode():
        pool, h = plain.clone(), rnd(B, DIM, N)
        vms.s6_conv_step(row, w, None, pool)
        vms.s6_conv_step(row, w, None, plain)                  # an ordinary tensor inside inference mode
    vms.s6_conv_step(row, w, None, pool)
    vms.s6_conv_step(row, w, None, plain)
    vms.s6_scan_step(row, row, None, rnd(B, N), rnd(B, N), A, None, None, h)
    assert torch.equal(pool, plain) and plain._version >= 2


@pytest.mark.parametrize("name", ["window", "h", "state", "out"])
def test_written_tensors_that_require_a_gradient_are_refused(name):
    """The write is not part of the graph: a gradient through it would be wrong. Without gradients it goes through."""
    import vision_mamba_selective_amd as vms
    say("case written tensors with gradients %s" % name)
    w, row, A = rnd(DIM, W), rnd(B, DIM), -rnd(DIM, N).abs()
    t = {"window": rnd(B, DIM, W - 1), "h": rnd(B, DIM, N), "state": rnd(2, B * K, 5), "out": rnd(B, DIM, L)}[name].requires_grad_()
    parent, x = i32([[0, 0, 1], [3, 5, 5]]), rnd(B, DIM, L)
    bt, ct = rnd(B, N), rnd(B, N)
    call = {"window": lambda v: vms.s6_conv_step(row, w, None, v),
            "h": lambda v: vms.s6_scan_step(row, row, None, bt, ct, A, None, None, v),
            "state": lambda v: vms.beam_reorder(v, parent),
            "out": lambda v: vms.s6_causal_conv(x, w, out=v)}[name]
    for v in (t, t * 1):                                       # a leaf, and a tensor of the graph
        was = v.detach().clone()
        with pytest.raises(ValueError, match="%s .*requires a gradient" % name):
            call(v)
        assert torch.equal(v, was)
        with torch.no_grad():
            call(v)
        call(v.detach())
