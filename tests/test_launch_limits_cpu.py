"""Sizes that pass every check of a tensor, but need 2^32 threads or more along
an axis of a launch (2^24 workgroups of 256): they are refused, not launched.
Addresses are made up and far apart."""
import ctypes

import pytest

from vision_mamba_selective_amd import _native as nat

UNSUP = -6
lib = nat.lib


def at(i):
    return (1 << 45) + (i << 41)


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def refused(code):
    assert code == UNSUP, (code, lib.vs_last_error())
    assert b"launch" in lib.vs_last_error()


def test_conv():
    refused(lib.s6_causal_conv(1, 1 << 10, 4, 1 << 26, nat.VS_BF16, 0, at(0), None, at(1), None, None, None, at(2), None, None))


@pytest.mark.parametrize("dim,L", [(1 << 13, (1 << 26) - 1), ((1 << 20) - 1, 1 << 19)])
def test_conv_gradient(dim, L):
    refused(lib.s6_causal_conv_grad(1, dim, 4, L, nat.VS_BF16, 0, at(0), at(1), None, at(2), None, None, None, None, at(3), at(4), at(5), None,
                                    at(6), 1 << 60, None))


def test_select():
    refused(lib.beam_select(65535, 32, 1 << 17, nat.VS_BF16, at(0), None, at(1), None, 0, at(2), at(3), at(4), at(5), 1 << 60, None))


@pytest.mark.parametrize("row", [(1 << 36) - 16, (1 << 32) + 3], ids=["16 bytes a thread", "1 byte a thread"])
def test_reorder(row):
    refused(lib.beam_reorder(1, 1, 2, row, 0, at(0), at(1), at(2), None))
