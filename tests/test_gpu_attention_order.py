"""exl3_attention where its roles hand over to one another in unusual orders:
items of one and of two MMA tiles, tiles of few rows behind full ones, the range
prelude's memory under the first queries.  Against 64 bits on the GPU.

The error allowed, from what the kernels round: the output to binary16 (2^-11 of
it, or half a subnormal step); each probability to binary16 (2^-11 of sum p|v|);
binary32 scores (dim + 8 roundings of 2^-24 of the largest sum |q k| scale, in
numerator and denominator); binary32 sums over n keys (2^-23 each).  Scales differ
by e^0.5 and more from page to page, keys and values are random: a unit read with
another's scales, or a row of another item, is off by far more.
"""
import numpy as np
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def build(seed, heads, kv_heads, dim, page, seq, new):
    """Everything on the GPU; requests share a pool of a few hundred random pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = 300
    k, v = (torch.randn((pages, kv_heads, page, dim), generator=g, device="cuda").mul_(40).round_().clamp_(-127, 127).to(torch.int8)
            for _ in "kv")
    ks, vs = (0.025 * torch.exp(0.7 * torch.randn((pages, kv_heads), generator=g, device="cuda")) for _ in "kv")
    width = -(-max(seq) // page)
    table = torch.randint(0, pages, (len(seq), width), generator=g, device="cuda", dtype=torch.int32)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    q = torch.randn((sum(new), heads, dim), generator=g, device="cuda").half()
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, start=start, seq=torch.tensor(seq, dtype=torch.int32, device="cuda"), q=q,
                lens=(seq, new))


def call(x, workspace=None, scale=None):
    cache = B.Exl3KvCache.from_tensors(x["k"], x["v"], x["ks"], x["vs"])
    return B.exl3_attention(cache, x["q"], x["start"], x["seq"], x["table"], max_new=max(x["lens"][1]), scale=scale, lse=True,
                            workspace=workspace)


def reference(x, scale=None):
    """(out, lse, allowed error of out, of lse), float64."""
    kvh, page, dim = x["k"].shape[1:]
    tokens, heads, _ = x["q"].shape
    group = heads // kvh
    scale = dim ** -0.5 if scale is None else scale
    out, allowed = torch.zeros((2, tokens, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, heads), -np.inf, dtype=torch.float64, device="cuda")
    lse_allowed = torch.zeros_like(lse)
    at = 0
    for b, (n, m) in enumerate(zip(*x["lens"])):
        own = x["table"][b, :-(-n // page)].long()
        kk, vv = ((x[c][own].double() * x[c + "s"][own].double()[:, :, None, None]).transpose(0, 1).reshape(kvh, -1, dim)[:, :n] for c in "kv")
        q = x["q"][at:at + m].double().view(m, kvh, group, dim).permute(1, 0, 2, 3)
        sees = torch.arange(n, device="cuda")[None, :] <= torch.arange(n - m, n, device="cuda")[:, None]
        z = torch.einsum("hmgd,hjd->hmgj", q, kk) * scale
        z.masked_fill_(~sees[None, :, None, :], -np.inf)
        size = torch.einsum("hmgd,hjd->hmgj", q.abs(), kk.abs()).masked_fill_(~sees[None, :, None, :], 0).amax(-1) * abs(scale)
        w = torch.softmax(z, -1).nan_to_num(0.0)
        o, spread = (torch.einsum("hmgj,hjd->hmgd", w, t) for t in (vv, vv.abs()))
        score = (dim + 8) * 2.0 ** -24 * size
        a = 2.0 ** -11 * o.abs() + 2.0 ** -25 + spread * (2.0 ** -11 + 2 * score[..., None] + (n + 64) * 2.0 ** -23)
        s = torch.logsumexp(z, -1)
        sa = score + (n + 64) * 2.0 ** -24 + 2.0 ** -20 + s.abs().nan_to_num(0, 0, 0) * 2.0 ** -22
        rows = slice(at, at + m)
        for t, r in ((out, o), (allowed, a)):
            t[rows] = r.permute(1, 0, 2, 3).reshape(m, heads, dim)
        for t, r in ((lse, s), (lse_allowed, sa)):
            t[rows] = r.permute(1, 0, 2).reshape(m, heads)
        at += m
    return out, lse, allowed, lse_allowed


def check(x, got, scale=None):
    out, lse, allowed, lse_allowed = reference(x, scale)
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
