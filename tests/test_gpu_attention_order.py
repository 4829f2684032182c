"""exl3_attention where its roles hand over to one another in unusual orders:
items of one and of two MMA tiles, tiles of few rows behind full ones, the range
prelude's memory under the first queries.  Against 64 bits on the GPU.

Every probability is a power of two that binary16 holds, so that a unit read with
another's scales or a row of another item stands out against little: a query picks
one element of the keys (which one depends on token and head), the scores are whole
powers of two from 0 to -12, the value scales 2^-7 to 2^-4.  What is left of the
kernels' rounding: the output to binary16 (2^-11 of it, or half a subnormal step);
scale * log2(e) within 3 * 2^-24 of 1, so a score of 12 is off by 25 * 2^-24 in the
exponent, in numerator and denominator, with the exponentials and logarithms of
2^-22 each: 2^-17 of sum p|v|; binary32 sums over n keys, 2^-23 each.
"""
import numpy as np
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


LN2 = float(np.log(2.0))


def build(seed, heads, kv_heads, dim, page, seq, new):
    """Everything on the GPU; requests share a pool of a few hundred random pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = 300

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)

    k, v = ints(-6, 0, pages, kv_heads, page, dim).to(torch.int8), ints(-127, 127, pages, kv_heads, page, dim).to(torch.int8)
    ks, vs = ints(0, 1, pages, kv_heads).float().exp2(), ints(-7, -4, pages, kv_heads).float().exp2()
    table = ints(0, pages - 1, len(seq), -(-max(seq) // page))
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    pick = ints(0, dim - 1, sum(new), heads)
    q = (torch.arange(dim, device="cuda") == pick[:, :, None]).half()
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, start=start, seq=torch.tensor(seq, dtype=torch.int32, device="cuda"), q=q,
                lens=(seq, new))


def call(x, workspace=None):
    cache = B.Exl3KvCache.from_tensors(x["k"], x["v"], x["ks"], x["vs"])
    return B.exl3_attention(cache, x["q"], x["start"], x["seq"], x["table"], max_new=max(x["lens"][1]), scale=LN2, lse=True,
                            workspace=workspace)


def reference(x):
    """(out, lse, allowed error of out, of lse), float64."""
    kvh, page, dim = x["k"].shape[1:]
    tokens, heads, _ = x["q"].shape
    group = heads // kvh
    out, allowed = torch.zeros((2, tokens, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, heads), -np.inf, dtype=torch.float64, device="cuda")
    lse_allowed = torch.zeros_like(lse)
    at = 0
    for b, (n, m) in enumerate(zip(*x["lens"])):
        own = x["table"][b, :-(-n // page)].long()
        kk, vv = ((x[c][own].double() * x[c + "s"][own].double()[:, :, None, None]).transpose(0, 1).reshape(kvh, -1, dim)[:, :n] for c in "kv")
        q = x["q"][at:at + m].double().view(m, kvh, group, dim).permute(1, 0, 2, 3)
        sees = torch.arange(n, device="cuda")[None, :] <= torch.arange(n - m, n, device="cuda")[:, None]
        z = torch.einsum("hmgd,hjd->hmgj", q, kk) * LN2
        z.masked_fill_(~sees[None, :, None, :], -np.inf)
        w = torch.softmax(z, -1).nan_to_num(0.0)
        o, spread = (torch.einsum("hmgj,hjd->hmgd", w, t) for t in (vv, vv.abs()))
        s = torch.logsumexp(z, -1)
        rows = slice(at, at + m)
        for t, r in ((out, o), (allowed, 2.0 ** -11 * o.abs() + 2.0 ** -25 + spread * (2.0 ** -17 + (n + 64) * 2.0 ** -23))):
            t[rows] = r.permute(1, 0, 2, 3).reshape(m, heads, dim)
        for t, r in ((lse, s), (lse_allowed, 2.0 ** -17 + (n + 64) * 2.0 ** -24 + s.abs().nan_to_num(0, 0, 0) * 2.0 ** -22)):
            t[rows] = r.permute(1, 0, 2).reshape(m, heads)
        at += m
    return out, lse, allowed, lse_allowed


def check(x, got):
    out, lse, allowed, lse_allowed = reference(x)
    off = (got[0].double() - out).abs()
    assert bool((off <= allowed).all()), f"{float((off / allowed).nan_to_num(1e9).max()):.2f} times what is allowed"
    seen = torch.isfinite(lse)
    assert torch.equal(seen, torch.isfinite(got[1])) and bool((got[1][~seen] == -np.inf).all())
    off = (got[1].double() - lse).abs()[seen]
    assert bool((off <= lse_allowed[seen]).all()), f"lse: {float((off / lse_allowed[seen]).max()):.2f} times what is allowed"


def repeat(x, times=4):
    """Checked, and the same bits every time."""
    kvh, _, dim = x["k"].shape[1:]
    ws = B.alloc_attention_workspace(x["q"].shape[1], kvh, dim, max(x["lens"][1]), "cuda")
    first = [t.clone() for t in call(x, ws)]
    check(x, first)
    for _ in range(times):
        assert all(torch.equal(a, b) for a, b in zip(first, call(x, ws)))
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 128, 16), (8, 2, 64, 64), (14, 2, 128, 32)])
@pytest.mark.parametrize("small,keys", [(20, 1000), (32, 640), (15, 1500), (13, 300)])
def test_items_of_one_tile_before_items_of_two(heads, kv_heads, dim, page, small, keys):
    """Every block gets several items: some of at most 128 rows, of 3 to 12 units that the second tile's warps skip, then
    some of more."""
    rng = np.random.default_rng(small)
    requests = 240
    seq = [int(keys + rng.integers(0, 128)) for _ in range(requests)]
    new = [int(rng.integers(40, 64)) if i % 3 == 2 else small for i in range(requests)]
    repeat(build(small, heads, kv_heads, dim, page, seq, new))


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("keys", [260, 100, 900])
def test_tiles_of_few_rows_behind_full_ones(heads, kv_heads, dim, keys):
    """Many items a block, full tiles and tiles of 1 to 96 rows in turn: warps that have rows in one item and none in the
    next."""
    group = heads // kv_heads
    rng = np.random.default_rng(keys)
    rows = [256 if i % 2 == 0 else int(rng.choice([52, 64, 72, 96, 132, 160, 192, 224])) for i in range(400)]
    new = [max(r // group, 1) for r in rows]
    repeat(build(keys, heads, kv_heads, dim, 32, [max(keys, n) + i % 5 for i, n in enumerate(new)], new))


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("requests", [700, 2500])
def test_first_queries_where_the_prelude_wrote(heads, kv_heads, dim, requests):
    """The requests' table of the range prelude lies where the first items' queries are copied to."""
    rng = np.random.default_rng(requests)
    new = [13 if i % 2 else int(rng.integers(13, 40)) for i in range(requests)]
    repeat(build(requests, heads, kv_heads, dim, 64, [n + int(rng.integers(0, 90)) for n in new], new))
