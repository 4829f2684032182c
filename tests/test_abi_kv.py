"""Refusals of the cache and attention entry points, on the host before anything
reaches a GPU (fake device addresses, never dereferenced)."""
import ctypes

import pytest

from trellis_decode_gemv_gb300 import binding as B

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def _cache(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, pages=4, kv_heads=2, page_size=16, head_dim=64) | kw
    return ctypes.byref(B.Exl3KvCacheStruct(*(a[n] for n, _ in B.Exl3KvCacheStruct._fields_)))


CACHE_ERRORS = [(dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(head_dim=96), 2),
                (dict(head_dim=256), 2), (dict(kv_heads=0), 2), (dict(pages=0), 2),
                (dict(pages=1 << 30, kv_heads=2), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
                (dict(v_scale=None), 1), (dict(k=A + 8), 6), (dict(v=A + 1), 6), (dict(k_scale=A + 2), 6)]


def _plan(lib, **kw):
    a = dict(ctx=A, new=A, requests=2, tokens=4, page=16, ring=A, cap=8, state=A, out=A, table=A, stride=4, seq=A,
             start=A, slot=A, pos=A) | kw
    return lib.exl3_kv_plan(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(requests=-1), 5), (dict(requests=B.MAX_REQUESTS + 1), 5), (dict(tokens=-1), 5), (dict(page=17), 2),
    (dict(stride=0), 2), (dict(cap=-1), 2), (dict(ctx=None), 1), (dict(new=None), 1), (dict(ring=None), 1),
    (dict(state=None), 1), (dict(out=None), 1), (dict(table=None), 1), (dict(seq=None), 1), (dict(start=None), 1),
    (dict(slot=None), 1), (dict(pos=None), 1), (dict(ctx=A + 2), 6), (dict(slot=A + 4), 6), (dict(table=A + 1), 6),
])
def test_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status


def _append(lib, cache=None, k=A, ks=128, v=A, vs=128, slot=A, tokens=3):
    return lib.exl3_kv_append(cache if cache is not None else _cache(), k, ks, v, vs, slot, tokens, None)


@pytest.mark.parametrize("kw,status", CACHE_ERRORS)
def test_append_and_attention_check_the_cache(lib, kw, status):
    assert _append(lib, cache=_cache(**kw)) == status
    assert _attend(lib, cache=_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 5), (dict(ks=64), 2), (dict(vs=132), 2), (dict(k=None), 1), (dict(v=None), 1),
    (dict(slot=None), 1), (dict(k=A + 8), 6), (dict(v=A + 2), 6), (dict(slot=A + 4), 6), (dict(tokens=0), 0),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def _attend(lib, **kw):
    a = dict(cache=_cache(), q=A, qs=256, heads=4, start=A, seq=A, requests=2, tokens=3, max_new=2, table=A, stride=4,
             scale=0.125, out=A, os=256, lse=A, ws=A, wsb=1 << 30) | kw
    return lib.exl3_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), 2), (dict(heads=3), 2), (dict(stride=0), 2), (dict(qs=248), 2), (dict(qs=260), 2),
    (dict(os=128), 2), (dict(requests=-1), 5), (dict(requests=B.MAX_REQUESTS + 1), 5), (dict(tokens=-1), 5),
    (dict(max_new=0), 5), (dict(q=None), 1), (dict(start=None), 1), (dict(seq=None), 1), (dict(table=None), 1),
    (dict(out=None), 1), (dict(q=A + 2), 6), (dict(out=A + 8), 6), (dict(lse=A + 2), 6), (dict(table=A + 2), 6),
    (dict(ws=None), 7), (dict(wsb=64), 7), (dict(ws=A + 4), 6), (dict(requests=0), 0), (dict(tokens=0), 0),
])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


def test_no_cache_at_all(lib):
    assert lib.exl3_kv_append(None, A, 128, A, 128, A, 1, None) == 1
    assert lib.exl3_attention(None, A, 256, 4, A, A, 1, 1, 1, A, 1, 1.0, A, 256, None, A, 1 << 30, None) == 1


def test_attention_workspace_bytes(lib):
    size = lib.exl3_attention_workspace_bytes
    assert size(32, 8, 128, 1) >= 256 and size(32, 8, 128, 4096) >= size(32, 8, 128, 1)
    for bad in ((0, 8, 128, 1), (32, 0, 128, 1), (33, 8, 128, 1), (32, 8, 96, 1), (32, 8, 128, 0)):
        assert size(*bad) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    import torch
    k = torch.zeros((2, 1, 16, 64), dtype=torch.int8)
    s = torch.zeros((2, 1))
    with pytest.raises(ValueError):
        B.Exl3KvCache.from_tensors(k, k, s, s)             # not on a GPU
    with pytest.raises(ValueError):
        B.Exl3KvCache.from_tensors(k, k[:1], s, s)
    with pytest.raises(ValueError):
        B.Exl3KvCache.from_tensors(torch.zeros((2, 1, 24, 64), dtype=torch.int8),
                                   torch.zeros((2, 1, 24, 64), dtype=torch.int8), s, s)
    with pytest.raises(ValueError):
        B.exl3_kv_plan(torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 3, 16,
                       torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros((2, 4), dtype=torch.int32))
