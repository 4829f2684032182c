"""exl3_attention where small terms make up the result.

Keys of one large score and many equal small ones, in closed form: with n - 1 keys
of score 0 and one whose score is g powers of two above, p = 2^g / (2^g + n - 1) for
that key.

The error allowed: the output to binary16 (2^-11 of it, or half a subnormal step);
a probability to 11 bits (2^-11 of sum p|v|) or, below binary16's normal range, to
2^-32 of the row's largest p v_scale (times |V|, summed over the keys); the exponent
of a score of g powers of two, 2^-22 g and as much again; sums over n keys in
binary32 (2^-23 for each of the 64 or so steps that partial sums go through, the
chains of up to n / 32 of them growing in equal steps: 2^-24 n / 32).
"""
import numpy as np
import pytest
import torch

from tests import test_gpu_attention as A
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def sink_call(heads, dim, page, keys, requests, sink, gaps):
    """Every request: key `sink` with score gaps[row], values 0; the others score 0 and hold 127 in the first half of the
    columns, 127 and -127 in turn and a few odd ones in the second.  One new token; (out, lse) and what they should be."""
    width = -(-keys // page)
    pages = width * requests
    k, v = (torch.zeros((pages, 1, page, dim), dtype=torch.int8, device="cuda") for _ in "kv")
    at = torch.arange(pages * page, device="cuda").view(pages, page) % (width * page)
    is_sink = at == sink
    k[:, 0, :, 0] = torch.where(is_sink, 100, 0)
    v[:, 0, :, :dim // 2] = 127
    v[:, 0, :, dim // 2:] = torch.where(at % 2 == 0, 127, torch.where(at % 7 == 1, 90, -127))[:, :, None].to(torch.int8)
    v[is_sink.nonzero(as_tuple=True)[0], 0, is_sink.nonzero(as_tuple=True)[1]] = 0
    ks, vs = torch.full((2, pages, 1), 1 / 64, device="cuda")
    scale = 0.125
    q = torch.zeros((requests, heads, dim), dtype=torch.float16, device="cuda")
    per = scale * 100 / 64 / np.log(2)                    # powers of two for q = 1
    q[:, :, 0] = torch.tensor([gaps[h % len(gaps)] / per for h in range(heads)], device="cuda").half()
    cache = B.Exl3KvCache.from_tensors(k, v, ks, vs)
    lens = torch.full((requests,), keys, dtype=torch.int32, device="cuda")
    got = B.exl3_attention(cache, q, torch.arange(requests + 1, dtype=torch.int32, device="cuda"), lens,
                           torch.arange(pages, dtype=torch.int32, device="cuda").view(requests, width), max_new=1, scale=scale, lse=True)
    g = q[0, :, 0].double().cpu().numpy() * per
    w = 2.0 ** g
    v64 = v[:width, 0].double().view(-1, dim)[:keys].cpu().numpy() / 64
    total = w + keys - 1
    out = v64.sum(0)[None] / total[:, None]
    spread = np.abs(v64).sum(0)[None] / total[:, None]
    largest = np.maximum(w, 1) / total
    score = 2 * 2.0 ** -22 * np.abs(g)
    chains = 64 * 2.0 ** -23 + keys / 32 * 2.0 ** -24
    allowed = (2.0 ** -11 * np.abs(out) + 2.0 ** -25 + spread * (2.0 ** -11 + 2 * score[:, None] + chains)
               + 2.0 ** -32 * largest[:, None] * np.abs(v64).sum(0)[None])
    lse, lse_allowed = np.log(total), score + chains + 2.0 ** -20 + 2.0 ** -22 * np.log(total)
    return got, out, allowed, lse, lse_allowed


GAPS = [-4.0, 3.0, 11.3, 17.6, 20.3, 22.9, 25.5, 30.1]


@pytest.mark.parametrize("heads,dim", [(8, 128), (16, 64), (64, 128), (72, 64)])
@pytest.mark.parametrize("keys,requests", [(500, 3), (3000, 40), (131072, 1)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_key_far_above_many(heads, dim, keys, requests, where):
    """An attention sink: one key outweighs each other by up to 2^30, its values are zero, and the others' sum is the result."""
    sink = {"first": 0, "middle": keys // 2 + 5, "last": keys - 1}[where]
    (got, got_lse), out, allowed, lse, lse_allowed = sink_call(heads, dim, 64, keys, requests, sink, GAPS)
    off = np.abs(got.double().cpu().numpy() - out[None])
    assert (off <= allowed).all(), f"{(off / allowed).max():.2f} times what is allowed, gap {GAPS[(off / allowed).max((0, 2)).argmax() % 8]}"
    off = np.abs(got_lse.double().cpu().numpy() - lse[None])
    assert (off <= lse_allowed).all(), f"lse: {(off / lse_allowed).max():.2f} times what is allowed"


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("tiny", [0.0, 1e-45, 1e-40, 2.0 ** -126, 1e-33, 2.0 ** -100, 2.0 ** -90, 2.0 ** -89, 1e-20])
def test_value_scales_next_to_zero(new, tiny):
    """Pages whose value scale is next to nothing, subnormal ones among them, beside others and alone: their values add
    nothing, their probabilities count."""
    x = A.make(np.random.default_rng(new), 4, 1, 128, 16, [700, new + 3, 40], [new, new, 1])
    x["v_scale"][x["block_table"][0, :43:3]] = tiny
    x["v_scale"][x["block_table"][1, :-(-(new + 3) // 16)]] = tiny
    A.check(x, A.run(x))


@pytest.mark.parametrize("heads,dim,new", [(8, 128, 1), (16, 64, 1), (4, 128, 100), (4, 64, 30)])
@pytest.mark.parametrize("size", [8, 16, 19, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 31, 34])
@pytest.mark.parametrize("spread", [12.0, 64.0])
def test_scores_as_large_as_the_types_allow(heads, dim, new, size, spread):
    """Scores around 2^size that differ by up to `spread` powers of two, or as far as binary32 tells them apart, in random
    order: whatever the weights are, equal values make an output of that value, to its own rounding (2^-11) and what the
    probabilities' rounding to binary16 (2^-11) and sums over n keys leave."""
    page, keys = 32, 3000
    g = torch.Generator(device="cuda").manual_seed(size)
    pages = -(-keys // page)
    k = torch.zeros((pages, 1, page, dim), dtype=torch.int8, device="cuda")
    k[..., 0] = 127
    k[..., 1] = torch.randint(0, 128, (pages, 1, page), generator=g, device="cuda").to(torch.int8)
    big = 2.0 ** min(size - 7, 15)
    unit = 2.0 ** size / (127 * big)                           # powers of two for a product of one
    small = spread / (127 * unit)
    q = torch.zeros((new, heads, dim), dtype=torch.float16, device="cuda")
    q[:, :, 0] = big
    q[:, :, 1] = small * (0.5 + torch.rand((new, heads), generator=g, device="cuda"))
    cache = B.Exl3KvCache.from_tensors(k, torch.full_like(k, 100), torch.full((pages, 1), unit, device="cuda"),
                                       torch.full((pages, 1), 1 / 64, device="cuda"))
    out, lse = B.exl3_attention(cache, q, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                torch.tensor([keys], dtype=torch.int32, device="cuda"),
                                torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1), max_new=new, scale=float(np.log(2)), lse=True)
    off = float((out.double() - 100 / 64).abs().max())
    assert off <= 100 / 64 * (2.0 ** -10 + (keys + 64) * 2.0 ** -23), off
    assert bool(torch.isfinite(lse).all())
