"""What the causal mixer's and beam search's entry points refuse, on the CPU:
every call below fails its validation before any HIP call. Addresses are made
up and far apart."""
import ctypes

import pytest

from vision_mamba_selective_amd import _native as nat

NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUP, WS = -1, -2, -3, -4, -5, -6, -8
lib = nat.lib


def at(i):
    return (1 << 44) + (i << 38)


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def call(name, defaults, order, **kw):
    a = dict(defaults)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(lib, name)(*[a[k] for k in order])


SCAN = dict(batch=2, dim=8, dstate=16, L=33, dtype=nat.VS_BF16, flags=1, u=at(0), delta=at(1), z=at(2), B=at(3), C=at(4),
            strides=None, A=at(5), D=at(6), bias=at(7), h0=at(8), lengths=at(9), y=at(10), h_out=at(11), saved=at(12),
            saved_bytes=1 << 30, ws=at(13), ws_bytes=1 << 30, stream=None)
SCAN_ORDER = [k for k in SCAN if k not in ("saved", "saved_bytes")]
COMMON = [
    (dict(dtype=7), DTYPE), (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(dim=-1), SHAPE), (dict(L=0), SHAPE),
    (dict(dim=1 << 20), UNSUP), (dict(L=1 << 27), UNSUP),
]
SCAN_BAD = COMMON + [
    (dict(dstate=0), SHAPE), (dict(dstate=17), UNSUP), (dict(flags=2), UNSUP), (dict(flags=4), UNSUP),
    (dict(u=None), NULL), (dict(delta=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(A=None), NULL),
    (dict(u=at(0) + 1), ALIGN), (dict(dtype=nat.VS_F32, z=at(2) + 2), ALIGN), (dict(A=at(5) + 2), ALIGN),
    (dict(h0=at(8) + 2), ALIGN), (dict(lengths=at(9) + 1), ALIGN),
    (dict(strides=arr(-1, 33, 264, 33, 264, 33, 528, 33, 528, 33)), SHAPE),
    (dict(strides=arr(264, 1 << 27, 264, 33, 264, 33, 528, 33, 528, 33)), UNSUP),
    (dict(strides=arr(1 << 44, 33, 264, 33, 264, 33, 528, 33, 528, 33)), UNSUP),
]


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(y=None), NULL), (dict(y=at(0) + 64), ALIAS), (dict(y=at(3) + 2), ALIAS), (dict(h_out=at(8)), ALIAS),
    (dict(h_out=at(10)), ALIAS), (dict(y=at(10) + 1), ALIGN), (dict(y=at(9)), ALIAS),
    (dict(L=20000, ws=None), WS), (dict(L=20000, ws_bytes=100), WS), (dict(L=20000, ws=at(1)), ALIAS),
    # y lies in the gap of a strided u's rows: the span counts
    (dict(strides=arr(1 << 20, 33, 264, 33, 264, 33, 528, 33, 528, 33), y=at(0) + (1 << 20)), ALIAS),
])
def test_scan_refuses(kw, code):
    assert call("s6_causal_scan", SCAN, SCAN_ORDER, **kw) == code
    assert lib.vs_last_error() != b""


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(y=None), NULL), (dict(saved=None), WS), (dict(saved_bytes=64), WS), (dict(saved=at(10)), ALIAS), (dict(saved=at(2)), ALIAS)])
def test_saving_scan_refuses(kw, code):
    assert call("s6_causal_scan_saved", SCAN, list(SCAN), **kw) == code


GRAD = dict(batch=2, dim=8, dstate=16, L=33, dtype=nat.VS_BF16, flags=1, u=at(0), delta=at(1), z=at(2), B=at(3), C=at(4),
            dy=at(5), strides=None, A=at(6), D=at(7), bias=at(8), lengths=at(9), saved=at(10), saved_bytes=1 << 30, dh=at(11),
            du=at(12), dd=at(13), dz=at(14), dB=at(15), dC=at(16), dA=at(17), dD=at(18), dbias=at(19), dh0=at(20), ws=at(21),
            ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [c for c in SCAN_BAD if "h0" not in c[0] and "strides" not in c[0]] + [
    (dict(dy=None), NULL), (dict(saved=None), NULL), (dict(saved_bytes=64), WS), (dict(du=None), NULL), (dict(dz=None), NULL),
    (dict(dA=None), NULL), (dict(dB=at(15) + 2), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=64), WS), (dict(du=at(5)), ALIAS),
    (dict(dB=at(16)), ALIAS), (dict(dh0=at(11)), ALIAS), (dict(dh0=at(21) + 64), ALIAS), (dict(ws=at(10)), ALIAS),
    (dict(strides=arr(264, 33, 264, 33, 264, 33, 528, 33, 528, 33, -1, 33)), SHAPE)])
def test_gradient_refuses(kw, code):
    assert call("s6_causal_scan_grad", GRAD, list(GRAD), **kw) == code


CONV = dict(batch=2, dim=8, width=4, L=33, dtype=nat.VS_F32, flags=1, x=at(0), strides=None, w=at(1), bias=at(2), window=at(3),
            lengths=at(4), y=at(5), window_out=at(6), stream=None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(width=1), SHAPE), (dict(width=9), UNSUP), (dict(flags=2), UNSUP), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(y=None), NULL), (dict(x=at(0) + 2), ALIGN), (dict(window=at(3) + 1), ALIGN), (dict(bias=at(2) + 1), ALIGN),
    (dict(y=at(0)), ALIAS), (dict(window_out=at(3)), ALIAS), (dict(window_out=at(5) + 4), ALIAS),
    (dict(strides=arr(264, -33)), SHAPE)])
def test_conv_refuses(kw, code):
    assert call("s6_causal_conv", CONV, list(CONV), **kw) == code


CONVG = dict(batch=2, dim=8, width=4, L=33, dtype=nat.VS_F32, flags=1, x=at(0), dy=at(1), strides=None, w=at(2), bias=at(3),
             window=at(4), lengths=at(5), dwo=at(6), dx=at(7), dw=at(8), db=at(9), dwin=at(10), ws=at(11), ws_bytes=1 << 30,
             stream=None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(width=1), SHAPE), (dict(width=9), UNSUP), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(db=None), NULL),
    (dict(ws=None), WS), (dict(ws_bytes=16), WS), (dict(dx=at(1)), ALIAS), (dict(dwin=at(6)), ALIAS), (dict(dw=at(11)), ALIAS)])
def test_conv_gradient_refuses(kw, code):
    assert call("s6_causal_conv_grad", CONVG, list(CONVG), **kw) == code


CSTEP = dict(batch=2, dim=8, width=4, dtype=nat.VS_F32, flags=1, x=at(0), sx=0, w=at(1), bias=at(2), window=at(3), slots=4,
             si=at(4), so=at(5), y=at(6), stream=None)
STEP_BAD = [(dict(dtype=3), DTYPE), (dict(batch=0), SHAPE), (dict(dim=0), SHAPE), (dict(slots=0), SHAPE), (dict(slots=1 << 31), UNSUP),
            (dict(si=None, slots=1), SHAPE), (dict(so=None, slots=1), SHAPE), (dict(y=None), NULL), (dict(si=at(4) + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", STEP_BAD + [
    (dict(width=1), SHAPE), (dict(width=9), UNSUP), (dict(flags=8), UNSUP), (dict(x=None), NULL), (dict(window=None), NULL),
    (dict(sx=-8), SHAPE), (dict(sx=1 << 28), UNSUP), (dict(y=at(0)), ALIAS), (dict(y=at(3)), ALIAS), (dict(window=at(0)), ALIAS)])
def test_conv_step_refuses(kw, code):
    assert call("s6_conv_step", CSTEP, list(CSTEP), **kw) == code


SSTEP = dict(batch=2, dim=8, dstate=16, dtype=nat.VS_F32, flags=1, u=at(0), delta=at(1), z=at(2), B=at(3), C=at(4), strides=None,
             A=at(5), D=at(6), bias=at(7), h=at(8), slots=4, si=at(9), so=at(10), y=at(11), stream=None)


@pytest.mark.parametrize("kw,code", STEP_BAD[:-1] + [
    (dict(si=at(9) + 2), ALIGN), (dict(dstate=0), SHAPE), (dict(dstate=17), UNSUP), (dict(flags=2), UNSUP), (dict(u=None), NULL), (dict(h=None), NULL), (dict(B=None), NULL),
    (dict(strides=arr(8, 8, 8, -1, 16)), SHAPE), (dict(h=at(8) + 2), ALIGN), (dict(y=at(8) + 4), ALIAS), (dict(h=at(3)), ALIAS)])
def test_scan_step_refuses(kw, code):
    assert call("s6_scan_step", SSTEP, list(SSTEP), **kw) == code


SELECT = dict(batch=2, beams=4, vocab=100, dtype=nat.VS_F32, logits=at(0), strides=None, scores=at(1), done=at(2), eos=3,
              os=at(3), op=at(4), ot=at(5), ws=at(6), ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(batch=0), SHAPE), (dict(batch=1 << 16), UNSUP), (dict(beams=0), SHAPE), (dict(beams=33), UNSUP),
    (dict(vocab=0), SHAPE), (dict(vocab=1 << 30), UNSUP), (dict(logits=None), NULL), (dict(scores=None), NULL), (dict(ot=None), NULL),
    (dict(eos=100), SHAPE), (dict(eos=-1), SHAPE), (dict(strides=arr(-1, 100)), SHAPE), (dict(strides=arr(1 << 40, 100)), UNSUP),
    (dict(ws=None), WS), (dict(ws_bytes=8), WS), (dict(ws=at(6) + 4), ALIGN), (dict(logits=at(0) + 1), ALIGN), (dict(op=at(4) + 2), ALIGN),
    (dict(os=at(1)), ALIAS), (dict(ot=at(4)), ALIAS), (dict(ws=at(0)), ALIAS)])
def test_select_refuses(kw, code):
    assert call("beam_select", SELECT, list(SELECT), **kw) == code


REORDER = dict(layers=2, batch=2, beams=4, row=64, layer=0, state=at(0), parent=at(1), out=at(2), stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), SHAPE), (dict(batch=0), SHAPE), (dict(beams=0), SHAPE), (dict(beams=33), UNSUP), (dict(row=0), SHAPE),
    (dict(row=1 << 36), UNSUP), (dict(layer=500), SHAPE), (dict(layer=-1), SHAPE), (dict(layer=1 << 58), UNSUP), (dict(state=None), NULL),
    (dict(parent=None), NULL), (dict(out=None), NULL), (dict(parent=at(1) + 2), ALIGN), (dict(out=at(0) + 64), ALIAS), (dict(out=at(1)), ALIAS),
    (dict(layers=65536), UNSUP)])
def test_reorder_refuses(kw, code):
    assert call("beam_reorder", REORDER, list(REORDER), **kw) == code


def test_workspaces():
    f = lib.s6_workspace_bytes
    for op in range(4):
        for bad in ((0, 8, 16, 33), (2, 0, 16, 33), (2, 8, 0, 33), (2, 8, 17, 33), (2, 8, 16, 0), (2, 8, 16, 1 << 27), (1 << 16, 8, 16, 33)):
            assert f(op, *bad) == 0, (op, bad)
    assert f(9, 2, 8, 16, 33) == 0
    assert f(nat.VS_S6_SCAN, 64, 1536, 16, 197) == 0               # rows enough to fill the chip: not cut
    assert f(nat.VS_S6_SCAN, 1, 768, 16, 4097) > 0
    # saved: a state for each 16 tokens and an ungated output for each token, in 256-byte regions
    assert f(nat.VS_S6_SAVED, 2, 8, 16, 33) == 2 * 8 * 3 * 16 * 4 + ((2 * 8 * 33 * 4 + 255) // 256) * 256
    assert f(nat.VS_S6_CONV_GRAD, 2, 8, 4, 33) == 2 * 8 * 5 * 4
    assert lib.beam_workspace_bytes(2, 4, 100) == 2 * 4 * 5 * 8
    for bad in ((0, 4, 100), (2, 33, 100), (2, 4, 0), (2, 4, 1 << 30), (1 << 16, 4, 100)):
        assert lib.beam_workspace_bytes(*bad) == 0


def test_python_refuses_host_tensors():
    import torch

    import vision_mamba_selective_amd as vms
    x = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError):
        vms.s6_causal_conv(x, torch.zeros(2, 4))
    with pytest.raises(TypeError):
        vms.s6_causal_conv(x.half(), torch.zeros(2, 4))
    with pytest.raises(ValueError):
        vms.s6_scan_step(x, x, x, x, x, torch.zeros(2, 4), None, None, torch.zeros(1, 2, 4))
    with pytest.raises(ValueError):
        vms.beam_select(x, torch.zeros(1, 2))
    with pytest.raises(ValueError):
        vms.beam_reorder(x, torch.zeros(1, 2, dtype=torch.int32))
