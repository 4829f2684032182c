"""Refusals of the norm, rotary and fork entry points, on the host before anything
reaches a GPU (fake device addresses, never dereferenced), and the rotary
frequencies, which are computed on the host."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from trellis_decode_gemv_gb300 import binding as B

A = 0x10000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def _norm(lib, **kw):
    a = dict(x=A, xs=256, r=A, rs=256, w=A, eps=1e-5, rows=3, n=256, y=A, h=A) | kw
    return lib.exl3_rms_norm(*a.values(), None)


def _norm_i8(lib, **kw):
    signs = kw.pop("signs", (A, None))
    a = dict(x=A, xs=256, r=A, rs=256, w=A, eps=1e-5, rows=3, n=256, s=(ctypes.c_void_p * 5)(*signs), outs=len(signs), q=A,
             qs=A, h=A) | kw
    return lib.exl3_rms_norm_i8(*a.values(), None)


NORM_ERRORS = [(dict(rows=-1), 5), (dict(n=0), 2), (dict(n=B.MAX_NORM + 128, xs=1 << 20, rs=1 << 20), 2), (dict(n=252), 2),
               (dict(xs=248), 2), (dict(xs=260), 2), (dict(rs=128), 2), (dict(eps=-1.0), 2), (dict(eps=NAN), 2), (dict(eps=INF), 2),
               (dict(x=None), 1), (dict(w=None), 1), (dict(x=A + 8), 6), (dict(r=A + 2), 6), (dict(w=A + 4), 6), (dict(h=A + 8), 6),
               (dict(rows=0), 0)]


@pytest.mark.parametrize("kw,status", NORM_ERRORS + [(dict(y=None), 1), (dict(y=A + 8), 6)])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", NORM_ERRORS + [
    (dict(q=None), 1), (dict(qs=None), 1), (dict(s=None), 1), (dict(q=A + 8), 6), (dict(qs=A + 2), 6), (dict(outs=0), 5),
    (dict(outs=5), 5), (dict(signs=(A, A + 8)), 6), (dict(n=136, xs=136, rs=136), 2)])
def test_norm_i8_refusals(lib, kw, status):
    assert _norm_i8(lib, **kw) == status


def _rotary(lib, **kw):
    a = dict(q=A, qs=512, qo=A, qos=512, qh=4, k=A, ks=256, ko=A, kos=256, kh=2, dim=128, part=64, inter=0, pos=A, f=A, factor=1.0,
             tokens=3) | kw
    return lib.exl3_rotary(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 5), (dict(dim=120), 2), (dict(dim=528, qs=1 << 14, qos=1 << 14, ks=1 << 14, kos=1 << 14), 2), (dict(part=8), 2),
    (dict(part=0), 2), (dict(part=144), 2), (dict(part=72), 2), (dict(qh=0), 2), (dict(kh=-1), 2), (dict(qs=504), 2), (dict(qs=516), 2),
    (dict(qos=256), 2), (dict(ks=128), 2), (dict(kos=260), 2), (dict(factor=NAN), 2), (dict(factor=INF), 2), (dict(q=None), 1),
    (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(f=None), 1), (dict(q=A + 8), 6),
    (dict(qo=A + 2), 6), (dict(k=A + 4), 6), (dict(ko=A + 8), 6), (dict(pos=A + 2), 6), (dict(f=A + 4), 6), (dict(tokens=0), 0)])
def test_rotary_refusals(lib, kw, status):
    assert _rotary(lib, **kw) == status


def _fork(lib, **kw):
    a = dict(parent=A, rows=3, ctx=A, requests=2, size=16, pages=8, ring=A, cap=8, state=A, state_out=A, table=A, stride=4, ctx_out=A,
             table_out=A, src=A, dst=A, n=A, ws=A, wsb=64) | kw
    return lib.exl3_kv_fork(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 5), (dict(rows=B.MAX_REQUESTS + 1), 5), (dict(requests=-1), 5), (dict(requests=B.MAX_REQUESTS + 1), 5),
    (dict(size=8), 2), (dict(pages=0), 2), (dict(stride=0), 2), (dict(cap=-1), 2), (dict(parent=None), 1), (dict(ctx=None), 1),
    (dict(ring=None), 1), (dict(state=None), 1), (dict(state_out=None), 1), (dict(table=None), 1), (dict(ctx_out=None), 1),
    (dict(table_out=None), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(n=None), 1), (dict(ws=None), 7), (dict(wsb=31), 7),
    (dict(ws=A + 8), 6), (dict(parent=A + 2), 6), (dict(table_out=A + 1), 6), (dict(n=A + 2), 6)])
def test_fork_refusals(lib, kw, status):
    assert _fork(lib, **kw) == status


def test_fork_workspace_bytes(lib):
    size = lib.exl3_kv_fork_workspace_bytes
    assert size(0) == 0 and size(-4) == 0 and size(1) >= 2 and size(1 << 20) >= 2 << 20


def _struct(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, pages=4, kv_heads=2, page_size=16, head_dim=64) | kw
    return B.Exl3KvCacheStruct(*(a[n] for n, _ in B.Exl3KvCacheStruct._fields_))


def _copy(lib, second=None, **kw):
    caches = (B.Exl3KvCacheStruct * 2)(_struct(), _struct(**(second or {})))
    a = dict(caches=caches, layers=2, src=A, dst=A, n=A, pairs=3) | kw
    return lib.exl3_kv_copy(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=-1), 5), (dict(layers=B.MAX_LAYERS + 1), 5), (dict(pairs=-1), 5), (dict(caches=None), 1), (dict(src=None), 1),
    (dict(dst=None), 1), (dict(n=None), 1), (dict(src=A + 2), 6), (dict(dst=A + 1), 6), (dict(n=A + 2), 6), (dict(second=dict(pages=5)), 2),
    (dict(second=dict(kv_heads=1)), 2), (dict(second=dict(page_size=32)), 2), (dict(second=dict(head_dim=128)), 2),
    (dict(second=dict(k=None)), 1), (dict(second=dict(v=A + 8)), 6), (dict(second=dict(page_size=9)), 2), (dict(layers=0), 0),
    (dict(pairs=0), 0)])
def test_copy_refusals(lib, kw, status):
    assert _copy(lib, **kw) == status


def _shared(lib, **kw):
    a = dict(cache=ctypes.byref(_struct()), q=A, qs=256, heads=4, start=A, seq=A, requests=2, tokens=3, max_new=2, table=A, stride=4, gs=A,
             pl=A, groups=1, max_group=2, scale=0.125, out=A, os=256, lse=A, ws=A, wsb=1 << 30) | kw
    return lib.exl3_attention_shared(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), 1), (dict(heads=3), 2), (dict(stride=0), 2), (dict(qs=248), 2), (dict(os=260), 2), (dict(requests=-1), 5),
    (dict(requests=B.MAX_REQUESTS), 5), (dict(groups=-1), 5), (dict(groups=B.MAX_REQUESTS), 5), (dict(tokens=-1), 5), (dict(max_new=0), 5),
    (dict(max_group=0), 5), (dict(q=None), 1), (dict(start=None), 1), (dict(gs=None), 1), (dict(pl=None), 1), (dict(out=None), 1),
    (dict(q=A + 2), 6), (dict(gs=A + 2), 6), (dict(pl=A + 1), 6), (dict(lse=A + 2), 6), (dict(ws=A + 4), 6), (dict(ws=None), 7),
    (dict(wsb=64), 7), (dict(requests=0), 0), (dict(tokens=0), 0)])
def test_attention_shared_refusals(lib, kw, status):
    assert _shared(lib, **kw) == status


def test_attention_shared_workspace_bytes(lib):
    size = lib.exl3_attention_shared_workspace_bytes
    few, more, many = size(32, 8, 128, 1, 8, 8), size(32, 8, 128, 1, 8, 9), size(32, 8, 128, 1, 64, 64)
    assert lib.exl3_attention_workspace_bytes(32, 8, 128, 1) < few < more < many
    rows = 32 * (2 * (128 + 2) * 4 + 2 * 4)            # a token's: two parts, and where they lie
    assert rows <= more - few <= rows + 4 * 256
    for bad in ((0, 8, 128, 1, 1, 1), (33, 8, 128, 1, 1, 1), (32, 8, 96, 1, 1, 1), (32, 8, 128, 0, 1, 1), (32, 8, 128, 1, 0, 1),
                (32, 8, 128, 1, 1, 0)):
        assert size(*bad) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    x, w = torch.zeros((2, 256), dtype=torch.float16), torch.ones(256, dtype=torch.float16)
    pos, f = torch.zeros(2, dtype=torch.int32), B.exl3_rotary_freqs(64, device="cpu")
    for call in (lambda: B.exl3_rms_norm(x, w, 1e-5), lambda: B.exl3_rms_norm_i8(x, w, 1e-5, [None]),
                 lambda: B.exl3_rotary(x.view(2, 4, 64), None, pos, f), lambda: B.exl3_rotary(x, None, pos, f),
                 lambda: B.exl3_kv_fork(pos, pos, 16, 8, pos, pos, torch.zeros((1, 4), dtype=torch.int32)),
                 lambda: B.exl3_rotary_freqs(63), lambda: B.exl3_rotary_freqs(64, scaling="other"),
                 lambda: B.exl3_rotary_freqs(64, scaling="llama3", low=4.0, high=4.0), lambda: B.Exl3KvCacheGroup([])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dim", [16, 64, 96, 128])
@pytest.mark.parametrize("scaling,scale", [("none", 1.0), ("linear", 3.5), ("ntk", 8.0), ("llama3", 8.0), ("yarn", 32.0)])
def test_rotary_frequencies(dim, scaling, scale):
    """The 64-bit fractions of a turn: off by at most half of 2^-64 of a turn, 2 pi 2^-65 < 2^-62 radians, from the formula's
    radians, of which either side's powers and logarithms take 2^-48 at most (a few 2^-52)."""
    f = B.exl3_rotary_freqs(dim, base=500000.0, scaling=scaling, scale=scale, original=4096, device="cpu")
    ref, factor = BO.frequencies(dim, 500000.0, scaling, scale, 4096)
    got = np.array([int(t) % 2 ** 64 for t in f.freqs.tolist()], np.float64) * 2.0 ** -64 * 2 * math.pi
    assert f.rotary_dim == dim and math.isclose(f.factor, factor, rel_tol=1e-15)
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -48 + 2.0 ** -62).all()


def test_rotary_frequencies_of_their_own():
    f = B.Exl3RotaryFreqs([0.0, -1.0, 7.0], factor=2.0, device="cpu")
    turns = [t / 2 ** 64 for t in f.freqs.tolist()]
    assert turns[0] == 0 and math.isclose(turns[1], -1 / (2 * math.pi)) and math.isclose(turns[2], 7 / (2 * math.pi) - 1, rel_tol=1e-9)
    assert f.factor == 2.0 and f.rotary_dim == 6


# ---- the oracle of the forks, pinned by hand -------------------------------------------

def test_oracle_fork_by_hand():
    table = [[3, 4, 9], [5, 6, 9]]                     # 20 and 32 tokens, pages of 16; the ring holds 7, 8, then nothing
    ring, state = np.array([0, 7, 8, 0, 0, 0]), [1, 2]
    got = BO.fork([0, 0, -1, 0, 0], [20, 32], 16, 10, ring, state, np.array(table))
    assert got["block_table"].tolist() == [[3, 4, -1], [3, 7, -1], [-1] * 3, [3, 8, -1], [-1] * 3]
    assert got["copy_from"].tolist() == [-1, 4, -1, 4, -1] and got["copy_to"].tolist() == [-1, 7, -1, 8, -1]
    assert got["copy_tokens"].tolist() == [0, 4, 0, 4, 0] and got["ctx_len"].tolist() == [20, 20, 0, 20, 0]
    assert got["free_state"].tolist() == [3, 2, 1] and got["free_pages"].tolist() == [0, 7, 8, 5, 6, 0]
