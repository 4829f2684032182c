"""Outputs that overlap one another or an input in a way that the kernels cannot serve are refused, on
the host before anything reaches a GPU (fake device addresses, never dereferenced)."""
import ctypes

import pytest

from trellis_decode_gemv_gb300 import binding as B

X, R, W, Y, H = (i << 24 for i in range(1, 6))
SHAPE = 2


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


@pytest.mark.parametrize("kw", [
    dict(y=H), dict(y=X, h=X), dict(y=R, h=R), dict(y=H + 512), dict(y=H + 2 * 256 * 3 - 16), dict(h=Y + 16),     # one another
    dict(y=X, xs=512), dict(h=X, xs=512), dict(y=R, rs=264), dict(h=R, rs=264),                                   # an input of another stride
    dict(y=X + 16), dict(y=X - 16), dict(h=R + 512), dict(y=X + 2 * 1024, xs=1024), dict(h=R + 2 * 2048 + 496, rs=2048),
    dict(y=X + 528, xs=1024), dict(y=W), dict(h=W - 2 * 256 * 3 + 16)])
def test_norm(lib, kw):
    a = dict(x=X, xs=256, r=R, rs=256, w=W, eps=1e-5, rows=3, n=256, y=Y, h=H) | kw
    assert lib.exl3_rms_norm(*a.values(), None) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(h=X, xs=512), dict(h=R, rs=512), dict(h=X + 16), dict(h=W), dict(q=X), dict(q=R), dict(q=W), dict(q=H), dict(q=H + 2 * 256 * 3 - 16),
    dict(qs=X), dict(qs=R + 512 * 3 - 16), dict(qs=W + 16), dict(qs=H), dict(q=Y, qs=Y), dict(qs=Y + 2 * 256 * 3 - 4),
    dict(q=X + 512, xs=512)])
def test_norm_i8(lib, kw):
    a = dict(x=X, xs=256, r=R, rs=256, w=W, eps=1e-5, rows=3, n=256, s=(ctypes.c_void_p * 2)(None, None), outs=2, q=Y, qs=6 << 24, h=H) | kw
    assert lib.exl3_rms_norm_i8(*a.values(), None) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(qo=Y, ko=Y), dict(ko=Y + 2 * 512 * 3 - 16), dict(qo=X, qos=1024), dict(ko=R, kos=512),      # one another; an input of another stride
    dict(qo=X + 16), dict(qo=R), dict(ko=X), dict(ko=R - 16),
    dict(q=X, qs=768, k=X + 1024, ks=768, qo=X + 16, qos=768, ko=Y), dict(q=X, qs=768, k=X + 1024, ks=768, qo=X, qos=768, ko=X + 1008, kos=768),
    dict(q=X, qs=768, k=X + 1024, ks=768, qo=X + 1024, qos=768, ko=X, kos=768)])
def test_rotary(lib, kw):
    a = dict(q=X, qs=512, qo=Y, qos=512, qh=4, k=R, ks=256, ko=H, kos=256, kh=2, dim=128, part=64, inter=0, pos=W, f=W, factor=1.0, tokens=3) | kw
    assert lib.exl3_rotary(*a.values(), None) == SHAPE


FORK = dict(parent=1, ctx=2, ring=3, state=4, state_out=5, table=6, ctx_out=7, table_out=8, src=9, dst=10, n=11, ws=12)
WRITTEN = ("ring", "state_out", "ctx_out", "table_out", "src", "dst", "n", "ws")


@pytest.mark.parametrize("one,other", [(a, b) for a in WRITTEN for b in FORK if a != b])
def test_fork(lib, one, other):
    at = {name: i << 24 for name, i in FORK.items()} | {one: FORK[other] << 24}
    a = dict(parent=0, rows=3, ctx=0, requests=2, size=16, pages=8, ring=0, cap=8, state=0, state_out=0, table=0, stride=4, ctx_out=0,
             table_out=0, src=0, dst=0, n=0, ws=0, wsb=64) | at
    assert lib.exl3_kv_fork(*a.values(), None) == SHAPE


@pytest.mark.parametrize("kw", [dict(table_out=(6 << 24) + 4 * 4 * 2 - 4), dict(src=(9 << 24) - 8, n=(9 << 24) - 12), dict(ring=(12 << 24) + 32),
                                dict(state_out=(4 << 24) + 4)])
def test_fork_that_overlaps_in_part(lib, kw):
    at = {name: i << 24 for name, i in FORK.items()} | kw
    a = dict(parent=0, rows=3, ctx=0, requests=2, size=16, pages=8, ring=0, cap=8, state=0, state_out=0, table=0, stride=4, ctx_out=0,
             table_out=0, src=0, dst=0, n=0, ws=0, wsb=64) | at
    assert lib.exl3_kv_fork(*a.values(), None) == SHAPE


@pytest.mark.parametrize("by", [4, 8])
def test_nothing_overlaps_an_empty_ring(lib, by):
    """A ring of no places may lie anywhere (the call is refused for what overlaps besides)."""
    at = {name: i << 24 for name, i in FORK.items()} | dict(ring=(5 << 24) + by, dst=9 << 24)
    a = dict(parent=0, rows=3, ctx=0, requests=2, size=16, pages=8, ring=0, cap=0, state=0, state_out=0, table=0, stride=4, ctx_out=0,
             table_out=0, src=0, dst=0, n=0, ws=0, wsb=64) | at
    assert lib.exl3_kv_fork(*a.values(), None) == SHAPE


def test_the_stride_of_one_row_says_nothing(lib):
    """(Refused for two outputs in one place, not for an arithmetic of strides.)"""
    a = dict(x=X, xs=(1 << 63) - 8, r=R, rs=1 << 62, w=W, eps=1e-5, rows=1, n=256, y=Y, h=Y)
    assert lib.exl3_rms_norm(*a.values(), None) == SHAPE
