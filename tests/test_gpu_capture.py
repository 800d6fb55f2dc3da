"""Which differentiable calls may be captured in a HIP graph: those that a
captured backward pass could not be made of are refused before anything is
captured, the others are not."""
import gc

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture
def leaves():
    """Leaves of both mixers, the norm and the loss, and a training step of them all."""
    import vision_mamba_selective_amd as vms
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()            # noqa: E731
    p = dict(x=rnd(2, 48, 130), w=rnd(48), r=rnd(2, 48, 130), i=rnd(2, 48, 130), lam=rnd(48), W=rnd(300, 48), taps=rnd(48, 4), bias=rnd(48),
             B=rnd(2, 16, 130), C=rnd(2, 16, 130), A=(-torch.rand(48, 16, generator=g) - 0.1).cuda().requires_grad_(), D=rnd(48), dt=rnd(48))
    target = torch.randint(-20, 300, (260,), generator=g).cuda()

    def step():
        y, _ = vms.rms_norm_autograd(p["x"], p["w"])
        u, _ = vms.s6_causal_conv_autograd(y, p["taps"], p["bias"])
        y, _ = vms.gated_scan_autograd(u, p["r"], p["i"], p["lam"], z=p["r"])
        y, _ = vms.s6_causal_scan_autograd(y, p["r"], p["i"], p["B"], p["C"], p["A"], p["D"], p["dt"])
        y, _ = vms.rms_norm_autograd(y, None, residual=p["x"])
        return vms.vocab_loss_autograd(y.transpose(1, 2).reshape(260, 48), p["W"], target)
    return p, step, target


def settle():
    gc.collect()                     # an exception's frames hold the refused call's graph
    torch.cuda.synchronize()


def replays(graph, got, eager):
    for k in range(3):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), k


def test_without_gradients_a_living_eager_graph_does_not_matter(leaves):
    """Captured under no_grad the calls record no graph: nothing is refused."""
    import vision_mamba_selective_amd as vms
    say("case capture no_grad")
    p, step, target = leaves
    alive = step()
    torch.cuda.synchronize()

    def calls():
        y, _ = vms.rms_norm_autograd(p["x"], p["w"])
        z, h = vms.gated_scan_autograd(y, p["r"], p["i"], p["lam"])
        return y, z, h, vms.vocab_loss_autograd(z.transpose(1, 2).reshape(260, 48), p["W"], target)
    with torch.no_grad():
        eager = [v.clone() for v in calls()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls()
    replays(graph, got, eager)
    assert alive.requires_grad


def test_streams_that_are_captured_together(leaves):
    """A leaf whose gradient node was made on another stream of the same capture is no eager graph's."""
    import vision_mamba_selective_amd as vms
    say("case capture two streams")
    p, _, _ = leaves
    side = torch.cuda.Stream()

    def calls():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a, _ = vms.rms_norm_autograd(p["x"], p["w"])
        main.wait_stream(side)
        b, _ = vms.rms_norm_autograd(p["r"], p["w"])
        return a, b
    eager = [v.detach().clone() for v in calls()]
    settle()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    with torch.no_grad():
        replays(graph, got, eager)


def refused(call):
    """The call is refused while capturing, before it launches anything, for an eager graph that is alive."""
    with pytest.raises(RuntimeError, match="eager graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            call()
    settle()


def test_leaves_behind_other_operations_are_seen(leaves):
    """Leaves that enter through torch's operations, the causal mixer's, or both, of a
    living eager graph; an eager graph that leads to an input itself; and the causal
    mixer's own calls. Freed, the eager graph is in no one's way."""
    import vision_mamba_selective_amd as vms
    say("case capture leaves behind operations")
    p, _, target = leaves
    x, w, r, i, lam, taps, bias, W = (p[k] for k in ("x", "w", "r", "i", "lam", "taps", "bias", "W"))
    plain = {k: v.detach() for k, v in p.items()}
    fixed = plain["x"]

    def conv():
        return vms.s6_causal_conv_autograd(fixed, taps, bias)[0]

    def scan():
        return vms.s6_causal_scan_autograd(fixed, plain["r"], plain["i"], plain["B"], plain["C"], p["A"], plain["D"], plain["dt"])[0]
    calls = {
        "torch operation, norm": lambda: vms.rms_norm_autograd(x * 2, plain["w"])[0],
        "torch operation, weight": lambda: vms.rms_norm_autograd(fixed, w.exp())[0],
        "torch operation, residual": lambda: vms.rms_norm_autograd(fixed, None, residual=x + 1)[0],
        "torch operations, recurrence": lambda: vms.gated_scan_autograd(fixed, (r * 2).tanh(), plain["i"], plain["lam"])[0],
        "torch operation, loss": lambda: vms.vocab_loss_autograd(fixed[0].t().contiguous(), W * 2, target[:130]),
        "convolution": conv,
        "scan": scan,
        "convolution, recurrence": lambda: vms.gated_scan_autograd(conv(), plain["r"], plain["i"], plain["lam"])[0],
    }
    for name, call in calls.items():
        say("case capture %s" % name)
        alive = call()
        torch.cuda.synchronize()
        refused(call)
        del alive
        settle()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        eager = call().detach().clone()
        with torch.no_grad():
            replays(graph, [got], [eager])
        del got, graph
        settle()
    made = x * 2                                               # an eager graph of its own
    torch.cuda.synchronize()
    refused(lambda: vms.rms_norm_autograd(made, plain["w"])[0])
    del made
    settle()


def test_captured_step_of_both_mixers(leaves):
    """A whole training step, both mixers' forward and backward passes among it,
    captured as torch asks: every replay equals the eager result."""
    say("case capture whole step")
    p, step, _ = leaves
    names = [k for k in p]
    dloss = torch.ones(260).cuda()

    def whole():
        loss = step()
        return [loss.detach()] + list(torch.autograd.grad(loss, [p[k] for k in names], grad_outputs=dloss))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [v.clone() for v in whole()]
    torch.cuda.current_stream().wait_stream(side)
    settle()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = whole()
    replays(graph, got, eager)
