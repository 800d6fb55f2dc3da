"""What the entry points of the gated recurrence, the norm and the vocabulary
loss refuse, on the CPU: every call below fails its validation before any HIP
call. Addresses are made up and far apart."""
import pytest
import torch

from test_causal_abi_cpu import ALIAS, ALIGN, DTYPE, NULL, SHAPE, UNSUP, WS, arr, at, call, lib
from vision_mamba_selective_amd import _calls
from vision_mamba_selective_amd import _native as nat

INF, NAN = float("inf"), float("nan")
COMMON = [(dict(dtype=7), DTYPE), (dict(batch=0), SHAPE), (dict(dim=-1), SHAPE), (dict(L=0), SHAPE), (dict(L=1 << 27), UNSUP)]

GATED = dict(batch=2, dim=8, L=33, dtype=nat.VS_BF16, x=at(0), r=at(1), i=at(2), z=at(3), strides=None, lam=at(4), rate=8.0, h0=at(5),
             lengths=at(6), y=at(7), h_out=at(8), saved=at(9), saved_bytes=1 << 30, stream=None)
GATED_BAD = COMMON + [
    (dict(batch=65536), SHAPE), (dict(dim=1 << 20), UNSUP), (dict(batch=1 << 10, dim=1 << 14, L=4), UNSUP), (dict(rate=-1.0), UNSUP),
    (dict(rate=INF), UNSUP), (dict(rate=NAN), UNSUP), (dict(x=None), NULL), (dict(r=None), NULL), (dict(i=None), NULL), (dict(lam=None), NULL),
    (dict(r=at(1) + 1), ALIGN), (dict(dtype=nat.VS_F32, z=at(3) + 2), ALIGN), (dict(lam=at(4) + 2), ALIGN), (dict(lengths=at(6) + 1), ALIGN),
    (dict(strides=arr(-1, 33, 264, 33, 264, 33, 264, 33, 264, 33)), SHAPE),
    (dict(strides=arr(264, 33, 264, 1 << 27, 264, 33, 264, 33, 264, 33)), UNSUP),
    (dict(strides=arr(264, 33, 264, 33, 1 << 44, 33, 264, 33, 264, 33)), UNSUP)]
FORWARD = [(dict(y=None), NULL), (dict(y=at(0) + 64), ALIAS), (dict(y=at(4)), ALIAS), (dict(h_out=at(5)), ALIAS), (dict(h_out=at(7) + 4), ALIAS),
           (dict(y=at(7) + 1), ALIGN), (dict(h0=at(5) + 2), ALIGN), (dict(h_out=at(8) + 2), ALIGN),
           (dict(strides=arr(1 << 20, 33, 264, 33, 264, 33, 264, 33), y=at(0) + (1 << 20)), ALIAS)]


@pytest.mark.parametrize("kw,code", GATED_BAD + FORWARD)
def test_gated_scan_refuses(kw, code):
    assert call("gated_scan", GATED, [k for k in GATED if not k.startswith("saved")], **kw) == code
    assert lib.vs_last_error() != b""


@pytest.mark.parametrize("kw,code", GATED_BAD + FORWARD + [
    (dict(saved=None), WS), (dict(saved_bytes=60), WS), (dict(saved=at(9) + 2), ALIGN), (dict(saved=at(7)), ALIAS), (dict(saved=at(2)), ALIAS)])
def test_saving_gated_scan_refuses(kw, code):
    assert call("gated_scan_saved", GATED, list(GATED), **kw) == code


GGRAD = dict(batch=2, dim=8, L=33, dtype=nat.VS_BF16, x=at(0), r=at(1), i=at(2), z=at(3), dy=at(4), strides=None, lam=at(5), rate=8.0,
             lengths=at(6), saved=at(7), saved_bytes=1 << 30, dh=at(8), dx=at(9), dr=at(10), di=at(11), dz=at(12), dlam=at(13), dh0=at(14),
             ws=at(15), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [c for c in GATED_BAD if "lam" not in c[0]] + [
    (dict(lam=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dr=None), NULL), (dict(di=None), NULL), (dict(dz=None), NULL),
    (dict(dlam=None), NULL), (dict(saved=None), WS), (dict(saved_bytes=60), WS), (dict(ws=None), WS), (dict(ws_bytes=60), WS),
    (dict(dx=at(4)), ALIAS), (dict(dr=at(9)), ALIAS), (dict(dlam=at(5)), ALIAS), (dict(dh0=at(8)), ALIAS), (dict(ws=at(7)), ALIAS),
    (dict(di=at(11) + 1), ALIGN), (dict(dh0=at(14) + 1), ALIGN), (dict(strides=arr(264, 33, 264, 33, 264, 33, 264, 33, -1, 33)), SHAPE)])
def test_gated_gradient_refuses(kw, code):
    assert call("gated_scan_grad", GGRAD, list(GGRAD), **kw) == code


GSTEP = dict(batch=2, dim=8, dtype=nat.VS_F32, x=at(0), r=at(1), i=at(2), z=at(3), strides=None, lam=at(4), rate=8.0, h=at(5), slots=4,
             si=at(6), so=at(7), y=at(8), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(dim=0), SHAPE), (dict(dim=1 << 20), UNSUP),
    (dict(batch=65535, dim=(1 << 20) - 1), UNSUP), (dict(rate=-0.5), UNSUP), (dict(slots=0), SHAPE), (dict(slots=1 << 31), UNSUP),
    (dict(si=None, slots=1), SHAPE), (dict(so=None, slots=1), SHAPE), (dict(x=None), NULL), (dict(h=None), NULL), (dict(y=None), NULL),
    (dict(strides=arr(8, -1, 8, 8)), SHAPE), (dict(strides=arr(8, 8, 1 << 28, 8)), UNSUP), (dict(si=at(6) + 2), ALIGN), (dict(h=at(5) + 2), ALIGN),
    (dict(x=at(0) + 2), ALIGN), (dict(y=at(0)), ALIAS), (dict(y=at(5) + 4), ALIAS), (dict(h=at(2)), ALIAS)])
def test_gated_step_refuses(kw, code):
    assert call("gated_scan_step", GSTEP, list(GSTEP), **kw) == code


NORM = dict(batch=2, dim=8, L=33, dtype=nat.VS_BF16, x=at(0), res=at(1), strides=None, w=at(2), eps=1e-6, lengths=at(3), y=at(4), sum=at(5),
            stream=None)
NORM_BAD = COMMON + [
    (dict(dim=8193), UNSUP), (dict(batch=1 << 31, L=1), UNSUP), (dict(batch=1 << 26, L=1), UNSUP), (dict(batch=1 << 20, L=1024), UNSUP),
    # launches of 2^32 threads: a row form of four waves, of sixteen, rows that lie apart, tiles
    (dict(batch=1 << 24, dim=2048, L=1), UNSUP), (dict(batch=1 << 22, dim=2056, L=1), UNSUP),
    (dict(batch=1 << 22, L=1, strides=arr(16, 2, 16, 2, 16, 2)), UNSUP), (dict(batch=1 << 21, L=32), UNSUP),
    (dict(eps=-1.0), UNSUP), (dict(eps=NAN), UNSUP), (dict(eps=INF), UNSUP), (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=at(0) + 1), ALIGN),
    (dict(w=at(2) + 2), ALIGN), (dict(lengths=at(3) + 2), ALIGN), (dict(y=at(4) + 1), ALIGN), (dict(y=at(0)), ALIAS), (dict(y=at(2)), ALIAS),
    (dict(strides=arr(-1, 33, 264, 33, 264, 33)), SHAPE), (dict(strides=arr(264, 1 << 27, 264, 33, 264, 33)), UNSUP)]


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(res=None), NULL), (dict(sum=None), NULL), (dict(res=at(1) + 1), ALIGN), (dict(sum=at(5) + 1), ALIGN), (dict(y=at(1)), ALIAS),
    (dict(sum=at(4)), ALIAS), (dict(sum=at(0)), ALIAS), (dict(sum=at(1) + 64), ALIAS), (dict(sum=at(2)), ALIAS),
    (dict(sum=at(1), y=at(1) + 64), ALIAS), (dict(sum=at(1), y=at(0)), ALIAS), (dict(sum=at(1), w=at(1)), ALIAS), (dict(sum=at(1), x=at(1) + 2), ALIAS),
    # the residual's rows lie apart: the sum, which is dense, is not the same tensor
    (dict(sum=at(1), strides=arr(264, 33, 300, 33)), ALIAS), (dict(sum=at(1), strides=arr(264, 33, 264, 40)), ALIAS)])
def test_norm_refuses(kw, code):
    assert call("rms_norm", NORM, list(NORM), **kw) == code


NGRAD = dict(batch=2, dim=8, L=33, dtype=nat.VS_BF16, x=at(0), dy=at(1), dsum=at(2), strides=None, w=at(3), eps=1e-6, lengths=at(4), y=at(5),
             dw=at(6), ws=at(7), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [c for c in NORM_BAD if not {"w", "lengths", "y"} & set(c[0])] + [
    (dict(dy=None), NULL), (dict(y=None), NULL), (dict(ws=None), WS), (dict(ws_bytes=60), WS), (dict(dy=at(1) + 1), ALIGN), (dict(dw=at(6) + 2), ALIGN),
    (dict(ws=at(7) + 2), ALIGN), (dict(y=at(0)), ALIAS), (dict(y=at(2)), ALIAS), (dict(dw=at(3)), ALIAS), (dict(ws=at(5)), ALIAS)])
def test_norm_gradient_refuses(kw, code):
    assert call("rms_norm_grad", NGRAD, list(NGRAD), **kw) == code


VOCAB = dict(tokens=5, dim=24, vocab=100, dtype=nat.VS_BF16, x=at(0), ldx=0, W=at(1), target=at(2), bits=64, loss=at(3), lse=at(4), ws=at(5),
             ws_bytes=1 << 40, stream=None)
VOCAB_BAD = [
    (dict(dtype=4), DTYPE), (dict(tokens=0), SHAPE), (dict(dim=0), SHAPE), (dict(vocab=-4), SHAPE), (dict(dim=65537), UNSUP),
    (dict(tokens=1 << 24), UNSUP), (dict(vocab=1 << 24), UNSUP), (dict(tokens=1 << 20, vocab=1 << 20), UNSUP), (dict(bits=16), UNSUP),
    (dict(tokens=1 << 18, dim=1 << 16), UNSUP), (dict(vocab=1 << 18, dim=1 << 16), UNSUP),
    (dict(ldx=23), SHAPE), (dict(ldx=-1), SHAPE), (dict(ldx=1 << 28), UNSUP), (dict(x=None), NULL), (dict(W=None), NULL), (dict(target=None), NULL),
    (dict(x=at(0) + 1), ALIGN), (dict(W=at(1) + 2), ALIGN), (dict(target=at(2) + 4), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=64), WS),
    (dict(ws=at(5) + 8), ALIGN), (dict(ws=at(1)), ALIAS)]


@pytest.mark.parametrize("kw,code", VOCAB_BAD + [
    (dict(loss=None), NULL), (dict(lse=None), NULL), (dict(lse=at(4) + 2), ALIGN), (dict(loss=at(4)), ALIAS), (dict(loss=at(0)), ALIAS),
    (dict(lse=at(2)), ALIAS)])
def test_vocab_loss_refuses(kw, code):
    assert call("vocab_loss", VOCAB, list(VOCAB), **kw) == code


VGRAD = dict(tokens=5, dim=24, vocab=100, dtype=nat.VS_BF16, x=at(0), ldx=0, W=at(1), target=at(2), bits=32, lse=at(3), dloss=at(4), dx=at(6),
             dW=at(7), ws=at(5), ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,code", [c for c in VOCAB_BAD if "target" not in c[0]] + [
    (dict(lse=None), NULL), (dict(dloss=None), NULL), (dict(dx=None), NULL), (dict(dW=None), NULL), (dict(target=at(2) + 2), ALIGN),
    (dict(dloss=at(4) + 2), ALIGN), (dict(dx=at(6) + 1), ALIGN), (dict(dx=at(0)), ALIAS), (dict(dW=at(1)), ALIAS), (dict(dW=at(6)), ALIAS)])
def test_vocab_gradient_refuses(kw, code):
    assert call("vocab_loss_grad", VGRAD, list(VGRAD), **kw) == code


def test_workspaces():
    f = lib.gated_workspace_bytes
    for op in (nat.VS_GATED_SAVED, nat.VS_GATED_GRAD):
        for bad in ((0, 8, 33), (2, 0, 33), (2, 8, 0), (2, 8, 1 << 27), (1 << 16, 8, 33), (1 << 12, 1 << 12, 33)):
            assert f(op, *bad) == 0, (op, bad)
    assert f(5, 2, 8, 33) == 0 and f(nat.VS_GATED_GRAD, 2, 8, 33) == 2 * 8 * 4
    # a state of 4 bytes for 128 tokens of short rows, for 512 of long ones
    assert f(nat.VS_GATED_SAVED, 2, 8, 129) == 2 * 8 * 2 * 4 and f(nat.VS_GATED_SAVED, 2, 8, 4097) == 2 * 8 * 9 * 4
    assert lib.norm_workspace_bytes(2, 8, 33) == 2 * 2 * 8 * 4 and lib.norm_workspace_bytes(3, 8, 1) >= 4 * 8 * 4
    for bad in ((0, 8, 33), (2, 8193, 33), (2, 8, 0)):
        assert lib.norm_workspace_bytes(*bad) == 0
    g = lib.vocab_workspace_bytes
    for bad in ((0, 24, 100), (5, 0, 100), (5, 24, 0), (5, 65537, 100), (1 << 24, 24, 100)):
        for op in (nat.VS_VOCAB_LOSS, nat.VS_VOCAB_GRAD):
            assert g(op, *bad, nat.VS_BF16) == 0
    assert g(2, 5, 24, 100, nat.VS_BF16) == 0 and g(0, 5, 24, 100, 9) == 0
    # the loss keeps 8 bytes for a token and a tile of the vocabulary, not its logits
    assert g(nat.VS_VOCAB_LOSS, 8194, 1536, 49999, nat.VS_BF16) < 8194 * 49999 * 2 // 10
    # the gradient a piece of them: 512 MB, and sums of dx
    assert g(nat.VS_VOCAB_GRAD, 8194, 1536, 200000, nat.VS_BF16) < (600 << 20) + 8194 * 1536 * 12


ENTRIES = [("gated_scan", 10), ("gated_scan_saved", 11), ("gated_scan_grad", 12), ("gated_scan_step", 10), ("rms_norm", 7), ("rms_norm_grad", 7),
           ("vocab_loss", 4), ("vocab_loss_grad", 6)]


@pytest.mark.parametrize("name,n", ENTRIES, ids=[e[0] for e in ENTRIES])
def test_binding_arguments(name, n):
    f = getattr(_calls, name)
    for count in (0, n - 1, n + 1):
        with pytest.raises(TypeError, match="expected %d arguments" % n):
            f(*[None] * count)
    with pytest.raises(ValueError, match="is required"):
        f(*[None] * n)
    with pytest.raises(TypeError, match="must be a tensor"):
        f(*[3] * n)
    for dt in (torch.float32, torch.float64):
        with pytest.raises((TypeError, ValueError)):
            f(*[torch.zeros(2, 3, 4, dtype=dt)] * n)          # not on the GPU, or not one of the types
