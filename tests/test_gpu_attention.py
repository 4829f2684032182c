"""exl3_attention on the GPU against the 64-bit oracle.

The error allowed to an element, from what the kernels round: the output to
binary16 (2^-11 of it, or half a subnormal step); every probability to binary16
(2^-11 of sum p|v|, and 2^-25 of the row's largest p v for what falls below
binary16's range); binary32 scores (dim + 8 roundings of 2^-24 of the largest
sum |q k| scale, twice, in numerator and denominator); binary32 sums over n keys
(2^-23 each, also for sums that the tensor cores cut instead of rounding).
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def cuda(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).cuda()


def make(rng, heads, kv_heads, dim, page, seq, new, extra=0, sharp=1.0, width=0):
    """Inputs as numpy.  Pages of nobody hold NaN scales, the tokens past a request's end the type's lowest value,
    table entries past its pages a number that is no page."""
    need = [-(-s // page) for s in seq]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(seq), max(max(need), 1, width)), 2 ** 30, np.int32)
    k, v = (np.clip(np.rint(40 * rng.standard_normal((pages, kv_heads, page, dim))), -127, 127).astype(np.int8) for _ in "kv")
    ks, vs = (np.full((pages, kv_heads), np.nan, np.float32) for _ in "kv")
    at = 0
    for b, n in enumerate(need):
        own = order[at:at + n]
        at += n
        table[b, :n] = own
        ks[own] = 0.025 * np.exp(0.5 * rng.standard_normal((n, kv_heads)))
        vs[own] = 0.025 * np.exp(1.0 * rng.standard_normal((n, kv_heads)))
        if n and seq[b] % page:
            k[own[-1], :, seq[b] % page:] = -128
            v[own[-1], :, seq[b] % page:] = -128
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = (sharp * rng.standard_normal((int(starts[-1]) + extra, heads, dim))).astype(np.float16)
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, q=q, q_start=starts, seq_len=np.array(seq, np.int32), block_table=table,
                scale=dim ** -0.5)


def run(x, max_new=None, workspace=None, out=None):
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    if max_new is None:
        max_new = max(int(np.diff(x["q_start"]).max()), 1)
    q = x["q"] if isinstance(x["q"], torch.Tensor) else cuda(x["q"])
    return B.exl3_attention(cache, q, cuda(x["q_start"]), cuda(x["seq_len"]), cuda(x["block_table"]), max_new=max_new,
                            scale=x["scale"], out=out, lse=True, workspace=workspace)


def check(x, got, rows=None):
    """Every row, or the requests' rows `rows` (the oracle is slow)."""
    out, lse = (t.double().cpu().numpy() for t in got)
    y = dict(x)
    y["q"] = x["q"].cpu().numpy() if isinstance(x["q"], torch.Tensor) else x["q"]
    ref, ref_lse, b = KO.attention(**y)
    n = int(x["q_start"][-1])
    dim = ref.shape[2]
    keys = float(x["seq_len"].max(initial=0))
    ref, ref_lse, spread, size = ref[:n], ref_lse[:n], b["spread"][:n], b["size"][:n, :, None]
    score = (dim + 8) * 2.0 ** -24 * size
    top = spread.max(-1, keepdims=True) * 4
    allowed = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + spread * (2.0 ** -11 + 2 * score + (keys + 64) * 2.0 ** -23) + keys * 2.0 ** -25 * top
    off = np.abs(out[:n] - ref)
    assert np.isfinite(out[:n]).all()
    assert (off <= allowed).all(), f"{(off / allowed).max():.2f} times what is allowed, at {np.unravel_index((off / allowed).argmax(), off.shape)}"
    seen = np.isfinite(ref_lse)
    assert np.array_equal(seen, np.isfinite(lse[:n])) and (lse[:n][~seen] == -np.inf).all()
    assert (out[:n][~seen] == 0).all()
    off = np.abs(lse[:n] - ref_lse)[seen]
    allowed = (score[..., 0] + (keys + 64) * 2.0 ** -24 + 2.0 ** -20 + np.abs(ref_lse) * 2.0 ** -22)[seen]
    assert (off <= allowed).all(), f"lse: {(off / allowed).max():.2f} times what is allowed"


HEADS = [(8, 8, 64), (4, 1, 128), (14, 2, 64), (16, 2, 128), (24, 2, 128), (5, 1, 64), (40, 1, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(heads, kv_heads, dim, page):
    """One new token; lengths around the pages and the tiles, and a place of the batch that holds nothing."""
    seq = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 257, 300]
    x = make(np.random.default_rng(heads + page), heads, kv_heads, dim, page, seq, [1] * len(seq))
    check(x, run(x))


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (14, 2, 64), (3, 3, 128)])
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("new", [2, 3, 5, 9])
def test_a_few_tokens(heads, kv_heads, dim, page, new):
    """Drafted tokens: causal among themselves; a request whose rows outnumber its tokens, and one without new tokens."""
    seq = [new, new + 1, 40, 130, 1, 31, 0, 77]
    news = [new, new, new, 1, new, 0, new, new - 1]
    x = make(np.random.default_rng(new + page), heads, kv_heads, dim, page, seq, news)
    check(x, run(x))


@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (4, 1, 128, 16), (4, 1, 64, 64), (7, 1, 64, 32), (6, 2, 128, 128), (1, 1, 128, 64), (12, 1, 128, 32)])
@pytest.mark.parametrize("seq,new", [
    ([33], [33]), ([128], [128]), ([129], [129]), ([300, 1, 200], [40, 1, 200]), ([257, 70, 0, 20], [150, 70, 1, 30]),
    ([513], [64])])
def test_prompts(heads, kv_heads, dim, page, seq, new):
    """Prompts and chunks of prompts beside single tokens."""
    x = make(np.random.default_rng(sum(seq) + heads), heads, kv_heads, dim, page, seq, new)
    check(x, run(x))


@pytest.mark.parametrize("max_new", [1, 2, 4, 8, 64, 4096])
def test_max_new_only_picks_kernels(max_new):
    """Requests with more new tokens than max_new says are computed all the same."""
    x = make(np.random.default_rng(9), 8, 2, 64, 32, [90, 1, 200, 17, 400], [1, 1, 50, 17, 3])
    check(x, run(x, max_new=max_new))


@pytest.mark.parametrize("new", [1, 100])
def test_long_context(new):
    x = make(np.random.default_rng(new), 2, 1, 128, 64, [9000, 100], [new, 1], sharp=3.0)
    check(x, run(x))


@pytest.mark.parametrize("new", [1, 6, 150])
def test_sharp_and_flat_scores(new):
    """Scores over a range of hundreds; a negative scale; a scale of zero (a plain mean)."""
    rng = np.random.default_rng(new)
    for sharp, scale in ((40.0, None), (1.0, -0.3), (1.0, 0.0)):
        x = make(rng, 4, 2, 64, 16, [new + 200, new], [new, new], sharp=sharp)
        x["scale"] = x["scale"] if scale is None else scale
        check(x, run(x))


@pytest.mark.parametrize("new", [1, 40])
def test_pages_of_very_different_scale(new):
    """Values a million times larger in some pages, and pages of zeros (scale 0) that still count in the sum."""
    rng = np.random.default_rng(new + 5)
    x = make(rng, 4, 1, 128, 16, [300, new], [new, new])
    x["v_scale"][np.isfinite(x["v_scale"])] *= 10.0 ** rng.integers(-6, 3, np.isfinite(x["v_scale"]).sum())
    own = x["block_table"][0, :19]
    x["v_scale"][own[::5]] = 0
    x["v"][own[::5]] = 0
    x["k_scale"][own[::4]] = 0
    check(x, run(x))


@pytest.mark.parametrize("new", [1, 33])
def test_rows_that_are_not_finite_stay_alone(new):
    """NaN or infinite queries spoil their own row and head only; a spoilt page its own request and head."""
    rng = np.random.default_rng(new + 6)
    x = make(rng, 8, 2, 64, 32, [200, 90], [new, 1])
    clean = [t.clone() for t in run(x)]
    x["q"][0, 1, 5], x["q"][new, 4, 0] = np.nan, np.inf
    out, lse = run(x)
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 1] = keep[new, 4] = False
    assert torch.isnan(out[~keep]).all() and torch.isnan(lse[~keep]).all()
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    y = dict(x, q=np.nan_to_num(x["q"], nan=0, posinf=0), k_scale=x["k_scale"].copy())
    y["k_scale"][y["block_table"][0, 1], 1] = np.nan
    out, _ = run(y)
    assert torch.isnan(out[:new, 4:]).all() and torch.isfinite(out[:new, :4]).all() and torch.isfinite(out[new:]).all()


@pytest.mark.parametrize("new", [1, 20])
def test_strides_and_rows_of_nobody(new):
    """q and out as slices of wider tensors; tokens after the last request's are left alone."""
    rng = np.random.default_rng(new + 7)
    x = make(rng, 6, 3, 64, 16, [new + 9, 50], [new, new], extra=4)
    wide = torch.zeros((x["q"].shape[0], 10, 64), dtype=torch.float16, device="cuda")
    wide[:, 2:8] = cuda(x["q"])
    room = torch.full((x["q"].shape[0], 9, 64), 7.0, dtype=torch.float16, device="cuda")
    x["q"] = wide[:, 2:8]
    out, lse = run(x, out=room[:, 1:7])
    check(x, (out, lse))
    assert (room[:, 0] == 7).all() and (room[:, 7:] == 7).all() and (room[2 * new:] == 7).all()


@pytest.mark.parametrize("new", [1, 5, 70])
def test_same_bits_and_clean_workspace(new):
    """Calls of different shapes with one workspace: equal bits every time, and counters that are zero after each."""
    rng = np.random.default_rng(new + 8)
    xs = [make(rng, 8, 2, 128, 64, seq, n) for seq, n in (([3000, 5, 400], [new, 1, new]), ([70 + new], [new]), ([1, 900], [1, new]))]
    ws = B.alloc_attention_workspace(8, 2, 128, new, "cuda")
    first = [[t.clone() for t in run(x, max_new=new, workspace=ws)] for x in xs]
    for _ in range(3):
        for x, a in zip(xs, first):
            b = run(x, max_new=new, workspace=ws)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, a in zip(xs, first):
        check(x, a)


def test_pages_shared_between_requests_and_other_stream():
    """Two requests over the same pages (a shared prompt), on a stream of their own."""
    rng = np.random.default_rng(11)
    x = make(rng, 8, 2, 64, 16, [100, 100], [1, 1])
    x["block_table"][1] = x["block_table"][0]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        got = run(x)
    stream.synchronize()
    check(x, got)


def test_page_numbers_outside_the_pool_read_as_zeros():
    x = make(np.random.default_rng(12), 4, 2, 64, 32, [100, 64], [1, 40])
    x["block_table"][0, 1], x["block_table"][1, 0] = -3, 2 ** 30
    got = run(x)
    y = {n: (np.concatenate([a, np.zeros_like(a[:1])]) if n in ("k", "v", "k_scale", "v_scale") else a) for n, a in x.items()}
    y["block_table"] = x["block_table"].copy()
    y["block_table"][0, 1] = y["block_table"][1, 0] = len(x["k"])
    check(y, got)


def test_lengths_past_the_table_are_cut():
    x = make(np.random.default_rng(13), 4, 2, 64, 16, [48, 32], [1, 1], width=3)
    x["seq_len"] = np.array([1000, 32], np.int32)
    got = run(x)
    x["seq_len"] = np.array([48, 32], np.int32)
    check(x, got)


@pytest.mark.parametrize("new", [1, 130])
def test_cache_past_four_gigabytes(new):
    page, kvh, dim = 128, 8, 128
    pages = (5 << 30) // (page * kvh * dim)
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free memory")
    x = make(np.random.default_rng(14), 8, kvh, dim, page, [200, 3 + new], [new, new])
    n = len(x["k"])
    big = [torch.empty((pages, kvh, page, dim), dtype=torch.int8, device="cuda") for _ in "kv"]
    scales = [torch.full((pages, kvh), float("nan"), device="cuda") for _ in "kv"]
    for t, name in zip(big + scales, ("k", "v", "k_scale", "v_scale")):
        t[-n:] = cuda(x[name])
    table = np.where(x["block_table"] < n, x["block_table"] + pages - n, x["block_table"]).astype(np.int32)
    got = B.exl3_attention(B.Exl3KvCache.from_tensors(*big, *scales), cuda(x["q"]), cuda(x["q_start"]), cuda(x["seq_len"]),
                           cuda(table), max_new=new, scale=x["scale"], lse=True)
    check(x, got)


def test_nothing_to_do():
    x = make(np.random.default_rng(15), 4, 2, 64, 16, [20], [1])
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = B.exl3_attention(cache, cuda(x["q"])[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), none,
                           torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)
    with pytest.raises(ValueError):
        B.exl3_attention(cache, cuda(x["q"]).transpose(0, 1), cuda(x["q_start"]), cuda(x["seq_len"]), cuda(x["block_table"]))
    with pytest.raises(TypeError):
        B.exl3_attention(cache, cuda(x["q"]).float(), cuda(x["q_start"]), cuda(x["seq_len"]), cuda(x["block_table"]))


@pytest.mark.parametrize("requests,new", [(33, 1), (100, 1), (300, 1), (65, 2), (40, 20)])
def test_many_requests(requests, new):
    """More requests than a warp has lanes, than a block has threads; some bring nothing; long ranges for every block."""
    rng = np.random.default_rng(requests + new)
    seq = rng.integers(0, 9000 // (new + requests // 20), requests)
    news = np.where(rng.random(requests) < 0.1, 0, new)
    x = make(rng, 8, 4, 64, 64, [int(s) for s in np.maximum(seq, news)], [int(n) for n in news])
    check(x, run(x))


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (7, 1, 64), (40, 1, 64)])
@pytest.mark.parametrize("seq,new", [([1200, 2, 3000], [40, 1, 65]), ([2600], [30]), ([1025, 1024, 1153, 900], [16, 16, 20, 64])])
def test_items_spread_over_many_blocks(heads, kv_heads, dim, seq, new):
    """Few rows over long contexts: every tile's keys are split between many thread blocks."""
    x = make(np.random.default_rng(sum(seq) + heads), heads, kv_heads, dim, 128, seq, new)
    check(x, run(x))


def test_in_a_graph_with_lengths_that_change():
    """A captured call reads lengths, tables and queries from device memory at every replay."""
    rng = np.random.default_rng(21)
    x = make(rng, 8, 2, 64, 32, [700, 333, 90], [1, 1, 1])
    y = dict(x, seq_len=np.array([650, 1, 64], np.int32), q=np.roll(x["q"], 1, 0))
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    q, start, seq, table = cuda(x["q"]), cuda(x["q_start"]), cuda(x["seq_len"]), cuda(x["block_table"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = B.alloc_attention_workspace(8, 2, 64, 1, "cuda")

    def call():
        B.exl3_attention(cache, q, start, seq, table, max_new=1, scale=x["scale"], out=out, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for z in (y, x, y):
        q.copy_(cuda(z["q"]))
        seq.copy_(cuda(z["seq_len"]))
        graph.replay()
        check(z, (out, lse))


@pytest.mark.parametrize("heads,dim", [(8, 128), (16, 128), (5, 64), (12, 64)])
@pytest.mark.parametrize("seq", [[4500], [17000], [68000], [9000, 30, 5200], [3000, 2999, 3, 1, 8000]])
def test_long_requests_over_many_blocks(heads, dim, seq):
    """One key/value head: an item's partial results come from up to a few hundred blocks, joined in one step or two.
    Twice from one workspace with the same bits, the counters left zero."""
    x = make(np.random.default_rng(len(seq) + seq[0]), heads, 1, dim, 64, seq, [1] * len(seq))
    ws = B.alloc_attention_workspace(heads, 1, dim, 1, "cuda")
    first = run(x, workspace=ws)
    check(x, first)
    second = run(x, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    head = ws[:256 + 4 * 3 * 640].view(torch.int32)   # the status word, the arrival counters
    assert int(head.abs().sum()) == 0


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (14, 2, 64)])
def test_prompts_beside_single_tokens(heads, kv_heads, dim):
    """A call that takes both kernels, the second beginning where the first's blocks end: three times from one workspace
    with the same bits."""
    seq = [900, 1, 64, 2100, 333, 0, 700, 1500, 80, 128, 3000, 17]
    new = [1, 1, 30, 1, 120, 0, 1, 65, 1, 3, 1, 17]
    x = make(np.random.default_rng(dim), heads, kv_heads, dim, 32, seq, new)
    ws = B.alloc_attention_workspace(heads, kv_heads, dim, max(new), "cuda")
    first = run(x, workspace=ws)
    check(x, first)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, run(x, workspace=ws)))
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("top", [12.0, 40.0, 130.0, -130.0])
def test_scores_that_climb(new, top):
    """Scores that rise (or fall) along the keys by up to 16 powers of two in 128 keys: the running maximum lags behind
    them, is passed within its room, and moves again and again."""
    heads, kv_heads, dim, page, seq = 4, 1, 128, 32, 1500
    x = make(np.random.default_rng(new), heads, kv_heads, dim, page, [seq], [new])
    for i, pg in enumerate(x["block_table"][0, :-(-seq // page)]):
        at = np.arange(i * page, (i + 1) * page)
        x["k"][pg] = np.rint(120 * np.minimum(at / seq, 1.0))[None, :, None].astype(np.int8) + (x["k"][pg] // 64)
        x["k_scale"][pg] = 0.01
    q = top / (120 * 0.01 * dim * x["scale"])
    x["q"] = (q * (1 + 0.1 * np.random.default_rng(5).standard_normal(x["q"].shape))).astype(np.float16)
    check(x, run(x))
