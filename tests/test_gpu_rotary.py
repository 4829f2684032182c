"""exl3_rotary on the GPU against float64.

The error allowed to an element: one rounding to binary16 (2^-11 of it, or half a
subnormal step, 2^-25); of the pair's |a| + |b|, times the factor: the angle as binary32
(2^-25 of half a turn, 2^-23.3 radians), cosine and sine (2 units of 2^-24), the factor, two
products and a sum (2^-24 each), in all under 2^-21; and position * 2^-50 for what
either side's 64-bit angle is off.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, x, position, radians, factor, interleaved):
    ref = BO.rotary(x, position, radians, factor, interleaved)
    got = got.double().cpu().numpy()
    half = len(radians)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    room = np.zeros(x.shape)
    room[..., a] = room[..., b] = np.abs(x[..., a].astype(np.float64)) + np.abs(x[..., b].astype(np.float64))
    room *= abs(factor) * (2.0 ** -21 + np.abs(np.asarray(position, np.float64))[:, None, None] * 2.0 ** -50)
    off = np.abs(got - ref)
    allowed = np.abs(ref) * 2.0 ** -11 + np.where(room > 0, 2.0 ** -25, 0) + room
    assert np.isfinite(got).all() and (off <= allowed).all(), f"{np.nanmax(off / np.maximum(allowed, 1e-300)):.3f} times what is allowed"
    untouched = np.arange(x.shape[-1]) >= 2 * half
    assert np.array_equal(got[..., untouched], x[..., untouched].astype(np.float64))


SHAPES = [(1, 1, 1, 64, 64), (5, 4, 2, 128, 128), (3, 7, 1, 64, 32), (33, 8, 8, 128, 32), (2, 5, 0, 96, 96), (64, 32, 8, 128, 64),
          (700, 3, 3, 64, 16), (1300, 1, 1, 64, 64), (4, 2, 1, 256, 256), (2, 1, 1, 512, 512), (9, 14, 2, 80, 48)]


@pytest.mark.parametrize("tokens,heads,kv_heads,dim,part", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling,scale", [("none", 1.0), ("yarn", 8.0)])
def test_rotary(tokens, heads, kv_heads, dim, part, interleaved, scaling, scale):
    rng = np.random.default_rng(tokens + heads + dim)
    q = rng.standard_normal((tokens, heads, dim)).astype(np.float16)
    k = rng.standard_normal((tokens, max(kv_heads, 1), dim)).astype(np.float16)
    position = rng.integers(0, 200000, tokens).astype(np.int32)
    position[0] = 0
    f = B.exl3_rotary_freqs(part, base=500000.0, scaling=scaling, scale=scale)
    radians, factor = BO.frequencies(part, 500000.0, scaling, scale)
    qo, ko = B.exl3_rotary(cuda(q), cuda(k) if kv_heads else None, cuda(position), f, interleaved=interleaved)
    check(qo, q, position, radians, factor, interleaved)
    if kv_heads:
        check(ko, k, position, radians, factor, interleaved)
    else:
        assert ko is None


@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_in_place_and_tokens_of_nobody(interleaved):
    """q and k as slices of a fused projection's output, turned where they lie; negative positions."""
    rng = np.random.default_rng(7)
    tokens, heads, kv, dim, part = 37, 6, 2, 64, 32
    wide = rng.standard_normal((tokens, heads + 2 * kv, dim)).astype(np.float16)
    position = rng.integers(0, 5000, tokens).astype(np.int32)
    position[[3, 20, 36]] = -1
    f = B.exl3_rotary_freqs(part)
    radians, factor = BO.frequencies(part, 10000.0)
    d = cuda(wide)
    q, k = d[:, :heads], d[:, heads:heads + kv]
    fresh = B.exl3_rotary(q, k, cuda(position), f, interleaved=interleaved)
    qo, ko = B.exl3_rotary(q, k, cuda(position), f, interleaved=interleaved, q_out=q, k_out=k)
    assert qo is q and ko is k and torch.equal(q, fresh[0]) and torch.equal(k, fresh[1])
    check(q, wide[:, :heads], position, radians, factor, interleaved)
    check(k, wide[:, heads:heads + kv], position, radians, factor, interleaved)
    assert np.array_equal(d[:, heads + kv:].cpu().numpy(), wide[:, heads + kv:])
    for t in (3, 20, 36):
        assert np.array_equal(d[t].cpu().numpy(), wide[t])


def test_far_positions():
    rng = np.random.default_rng(8)
    position = np.array([2 ** 31 - 1, 2 ** 24 + 1, 1000003, 131071, 1 << 30], np.int32)
    q = rng.standard_normal((5, 3, 128)).astype(np.float16)
    f = B.exl3_rotary_freqs(128, base=500000.0)
    qo, _ = B.exl3_rotary(cuda(q), None, cuda(position), f)
    check(qo, q, position, *BO.frequencies(128, 500000.0), False)


def test_what_is_not_finite_stays_in_its_pair():
    rng = np.random.default_rng(9)
    q = rng.standard_normal((4, 2, 64)).astype(np.float16)
    q[1, 0, 3], q[2, 1, 40] = np.inf, np.nan
    position = np.array([5, 6, 7, 8], np.int32)
    f = B.exl3_rotary_freqs(64)
    got, _ = B.exl3_rotary(cuda(q), None, cuda(position), f)
    bad = np.zeros(q.shape, bool)
    bad[1, 0, [3, 35]] = bad[2, 1, [8, 40]] = True
    assert np.array_equal(~np.isfinite(got.cpu().numpy()), bad)
    clean, _ = B.exl3_rotary(cuda(np.where(bad, np.float16(0), q)), None, cuda(position), f)
    assert np.array_equal(got.cpu().numpy()[~bad], clean.cpu().numpy()[~bad])


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(10)
    q, k = (cuda(rng.standard_normal((50, h, 128)).astype(np.float16)) for h in (8, 2))
    position = cuda(rng.integers(0, 9000, 50).astype(np.int32))
    f = B.exl3_rotary_freqs(128, scaling="llama3", scale=8.0)
    want = B.exl3_rotary(q, k, position, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = B.exl3_rotary(q, k, position, f)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.exl3_rotary(q, k, position, f)
    position.add_(1)
    graph.replay()
    want = B.exl3_rotary(q, k, position, f)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_no_tokens_and_shapes_that_do_not_fit():
    f = B.exl3_rotary_freqs(64)
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    assert B.exl3_rotary(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"), f)[0].shape == (0, 4, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: B.exl3_rotary(q, q[:1], pos, f), lambda: B.exl3_rotary(q, None, pos[:1], f),
                 lambda: B.exl3_rotary(q.transpose(0, 1), None, pos, f), lambda: B.exl3_rotary(q, None, pos, f, q_out=q[:, :2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        B.exl3_rotary(q.float(), None, pos, f)
    with pytest.raises(B.Exl3Error):
        B.exl3_rotary(q, None, pos, B.exl3_rotary_freqs(128))
