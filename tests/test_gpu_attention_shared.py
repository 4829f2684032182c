"""exl3_attention_shared on the GPU against the 64-bit oracle of exl3_attention, which
knows nothing of prefixes: the result is the one of every request over its own pages.
The error allowed is exl3_attention's (the two parts of a row are put together in
binary32: three more roundings of 2^-24)."""
import numpy as np
import pytest
import torch

from tests import test_gpu_attention as A
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu

cuda, check = A.cuda, A.check


def make(rng, heads, kv_heads, dim, page, groups, extra=0, sharp=1.0):
    """groups: (prefix, [(own cached and new tokens, new tokens), ...]); an own of None: the request holds nothing, or with
    a number below zero that many tokens less than the prefix.  Full pages of a prefix are shared; the page in which it
    ends is every request's own, with the same values up to there.  Nobody's pages hold NaN scales."""
    seq, new, start, prefix, of = [], [], [0], [], []
    for g, (p, members) in enumerate(groups):
        prefix.append(p)
        for own, n in members:
            seq.append(0 if own is None else p + own)
            new.append(n)
            of.append(g)
        start.append(len(seq))
    x = A.make(rng, heads, kv_heads, dim, page, seq, new, extra=extra, sharp=sharp)
    lead = {}
    for b, g in enumerate(of):
        p = prefix[g]
        if seq[b] == 0:
            continue
        if g not in lead or seq[lead[g]] < p <= seq[b]:
            lead.setdefault(g, b)
            if seq[b] >= p:
                lead[g] = b
    for b, g in enumerate(of):
        p = min(prefix[g], seq[b])
        if seq[b] == 0 or lead[g] == b or seq[lead[g]] < prefix[g]:
            continue
        table, full = x["block_table"], p // page
        table[b, :full] = table[lead[g], :full]
        if p % page:
            at, to = table[lead[g], full], table[b, full]
            for name in "kv":
                x[name][to, :, :p % page] = x[name][at, :, :p % page]
                x[name + "_scale"][to] = x[name + "_scale"][at]
    return x, np.array(start, np.int32), np.array(prefix, np.int32)


def widened(x):
    """The table with columns that no request reaches: what it could hold is worth sharing, so that the kernels for that run."""
    n, width = x["block_table"].shape
    page_bytes = 2 * x["k"][0].size
    wide = np.full((n, max(width, -(-200_000_000 // (n * page_bytes)))), 2 ** 30, np.int32)
    wide[:, :width] = x["block_table"]
    return wide


def run(x, start, prefix, max_new=None, max_group=None, workspace=None, out=None, wide=True):
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    if max_new is None:
        max_new = max(int(np.diff(x["q_start"]).max()), 1)
    if max_group is None:
        max_group = max([int(x["q_start"][e] - x["q_start"][a]) for a, e in zip(start[:-1], start[1:])] + [1])
    q = x["q"] if isinstance(x["q"], torch.Tensor) else cuda(x["q"])
    return B.exl3_attention_shared(cache, q, cuda(x["q_start"]), cuda(x["seq_len"]), cuda(widened(x) if wide else x["block_table"]),
                                   cuda(start), cuda(prefix), max_new=max_new, max_group=max_group, scale=x["scale"], out=out, lse=True, workspace=workspace)


HEADS = [(8, 8, 64), (4, 1, 128), (14, 2, 64), (16, 2, 128), (5, 1, 64)]


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("prefix", [1, 31, 64, 130, 517])
def test_samples_of_one_prompt(heads, kv_heads, dim, page, prefix):
    own = [1, 2, 15, 33, 64, 100, 7]
    x = make(np.random.default_rng(heads + page + prefix), heads, kv_heads, dim, page, [(prefix, [(k, 1) for k in own])])
    check(x[0], run(*x))


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("new", [1, 2, 5])
def test_groups_of_every_kind(heads, kv_heads, dim, page, new):
    """Groups of one, without a prefix, whose first request holds nothing or less than the prefix; requests without new tokens."""
    groups = [(100, [(new, new)]), (300, [(None, 1), (9, new), (new, new), (70, 1), (-20, 1), (40, 0)]), (0, [(5, new), (60, new)]),
              (64, [(None, 1), (None, 0)]), (129, [(-1, new), (-100, 1), (-5, 1)]), (40, [(200, new), (17, new), (new, new), (90, new)])]
    x = make(np.random.default_rng(heads + new), heads, kv_heads, dim, page, groups)
    check(x[0], run(*x))


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 128, 16), (8, 1, 64, 64), (7, 1, 128, 32), (6, 3, 64, 128)])
@pytest.mark.parametrize("requests,new", [(13, 1), (40, 1), (70, 2), (6, 4)])
def test_many_rows_behind_a_prefix(heads, kv_heads, dim, page, requests, new):
    """More than 48, 128 and 256 rows of a group: the prefix by the other kernel than the rest."""
    rng = np.random.default_rng(requests + heads)
    members = [(int(rng.integers(new, 90)), new) for _ in range(requests)]
    members[1] = (None, 1)
    x = make(rng, heads, kv_heads, dim, page, [(700, members), (333, [(5, new), (200, new)])])
    check(x[0], run(*x))


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 1, 128, 16), (8, 2, 64, 64), (7, 1, 64, 32)])
def test_chunks_of_prompts_behind_a_prefix(heads, kv_heads, dim, page):
    """Requests that bring many tokens: their own keys by the many-rows kernel too, beside single tokens."""
    groups = [(333, [(150, 150), (70, 40), (9, 1), (200, 13)]), (1000, [(300, 300), (1, 1)]), (50, [(100, 100), (90, 1)])]
    x = make(np.random.default_rng(heads), heads, kv_heads, dim, page, groups)
    check(x[0], run(*x))


@pytest.mark.parametrize("max_new,max_group", [(1, 1), (1, 100), (50, 1), (4096, 4096), (2, 3)])
def test_hints_only_pick_kernels(max_new, max_group):
    groups = [(300, [(40, 1), (50, 50), (3, 3)]), (100, [(1, 1), (60, 17)]), (64, [(5, 1)] * 30)]
    x = make(np.random.default_rng(9), 8, 2, 64, 32, groups)
    check(x[0], run(*x, max_new=max_new, max_group=max_group))


@pytest.mark.parametrize("requests,groups", [(33, 2), (100, 30), (300, 300), (64, 64)])
def test_many_requests_and_groups(requests, groups):
    rng = np.random.default_rng(requests)
    cuts = np.sort(rng.choice(np.arange(1, requests), groups - 1, replace=False)).tolist() if groups < requests else list(range(1, requests))
    x = make(rng, 8, 4, 64, 64, [(int(rng.integers(0, 400)), [(int(rng.integers(1, 200)), 1) for _ in range(e - a)])
                                 for a, e in zip([0] + cuts, cuts + [requests])])
    check(x[0], run(*x))


@pytest.mark.parametrize("groups,each,chunk", [(36, 25, 1), (41, 25, 1), (3, 4, 40), (9, 5, 60)])
def test_many_row_tiles(groups, each, chunk):
    """More row tiles than a warp has lanes, more requests and groups than are kept in shared memory; prefixes of one call on
    both sides of what either kernel takes."""
    rng = np.random.default_rng(groups)
    x = make(rng, 4, 2, 64, 32, [(int(rng.integers(64, 200)), [(int(rng.integers(chunk, chunk + 40)), chunk) for _ in range(each - g % 3)])
                                 for g in range(groups)])
    check(x[0], run(*x))


@pytest.mark.parametrize("requests", [8, 40])
def test_long_prefix(requests):
    """A prefix split between many blocks, in both kernels; twice from one workspace with the same bits, the counters left zero."""
    x, start, prefix = make(np.random.default_rng(requests), 4, 1, 128, 64, [(9001, [(5 + i, 1) for i in range(requests)])])
    ws = B.alloc_attention_shared_workspace(4, 1, 128, 1, requests, requests, "cuda")
    first = run(x, start, prefix, workspace=ws)
    check(x, first)
    second = run(x, start, prefix, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    assert not ws[:256 + 4 * 3 * 640].any()


@pytest.mark.parametrize("requests", [6, 30])
def test_sharp_scores_and_scales_far_apart(requests):
    """The prefix outweighs the own keys, or they it, by far; a negative scale; pages of very different scale."""
    rng = np.random.default_rng(requests)
    for sharp, scale in ((40.0, None), (1.0, -0.3), (1.0, 0.0)):
        x, start, prefix = make(rng, 8, 2, 64, 16, [(300, [(60, 1)] * requests)], sharp=sharp)
        x["scale"] = x["scale"] if scale is None else scale
        seen = np.isfinite(x["v_scale"])
        x["v_scale"][seen] *= 10.0 ** rng.integers(-5, 2, seen.sum())
        at = x["block_table"][:, 300 // 16]            # the page in which the prefix ends: the same in all requests
        x["v_scale"][at] = x["v_scale"][at[0]]
        check(x, run(x, start, prefix))


@pytest.mark.parametrize("requests", [5, 40])
def test_rows_that_are_not_finite_stay_alone(requests):
    rng = np.random.default_rng(requests)
    x, start, prefix = make(rng, 8, 2, 64, 32, [(200, [(50, 1)] * requests)])
    clean = [t.clone() for t in run(x, start, prefix)]
    x["q"][0, 1, 5], x["q"][2, 4, 0] = np.nan, np.inf
    out, lse = run(x, start, prefix)
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 1] = keep[2, 4] = False
    assert torch.isnan(out[~keep]).all() and torch.isnan(lse[~keep]).all()
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    y = dict(x, q=np.nan_to_num(x["q"], nan=0, posinf=0), k_scale=x["k_scale"].copy())
    y["k_scale"][y["block_table"][1, 7], 1] = np.nan   # a request's own page
    out, _ = run(y, start, prefix)
    bad = torch.zeros_like(lse, dtype=torch.bool)
    bad[1, 4:] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    y["k_scale"][y["block_table"][1, 1], 0] = np.nan   # a shared one
    out, _ = run(y, start, prefix)
    assert torch.isnan(out[:, :4]).all()


@pytest.mark.parametrize("requests", [5, 40])
def test_strides_rows_of_nobody_and_requests_outside_all_groups(requests):
    rng = np.random.default_rng(requests)
    x, start, prefix = make(rng, 6, 3, 64, 16, [(100, [(9, 1)] * 3), (300, [(50, 1)] * requests), (77, [(9, 1)] * 3)], extra=4)
    start, prefix = start[1:3], prefix[1:2]            # the first and the last three belong to no group
    wide = torch.zeros((x["q"].shape[0], 10, 64), dtype=torch.float16, device="cuda")
    wide[:, 2:8] = cuda(x["q"])
    room = torch.full((x["q"].shape[0], 9, 64), 7.0, dtype=torch.float16, device="cuda")
    x["q"] = wide[:, 2:8]
    out, lse = run(x, start, prefix, out=room[:, 1:7])
    check(x, (out, lse))
    n = int(x["q_start"][-1])
    assert (room[:, 0] == 7).all() and (room[:, 7:] == 7).all() and (room[n:] == 7).all()


@pytest.mark.parametrize("requests,new", [(7, 1), (3, 40)])
def test_little_to_read(requests, new):
    """Tables that hold too little for a look at what is shared: the bits of the call without prefixes."""
    x, start, prefix = make(np.random.default_rng(new), 8, 2, 64, 32, [(200, [(50 + new, new)] * requests)])
    got = run(x, start, prefix, wide=False)
    check(x, got)
    assert all(torch.equal(a, b) for a, b in zip(got, A.run(x)))


def test_no_groups_at_all():
    x, _, _ = make(np.random.default_rng(3), 4, 2, 64, 16, [(0, [(90, 1), (33, 2), (None, 1)])])
    check(x, run(x, np.zeros(1, np.int32), np.zeros(0, np.int32)))
    check(x, run(x, np.array([0, 2], np.int32), np.array([-5], np.int32)))


def test_in_a_graph_with_lengths_that_change():
    x, start, prefix = make(np.random.default_rng(21), 8, 2, 64, 32, [(333, [(70, 1), (40, 1), (9, 1)]), (64, [(200, 1)] * 20)])
    y = dict(x, seq_len=np.where(np.arange(23) % 3 == 1, 0, x["seq_len"] - 5).astype(np.int32), q=np.roll(x["q"], 1, 0))
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    q, starts, seq, table, gs, pl = (cuda(a) for a in (x["q"], x["q_start"], x["seq_len"], widened(x), start, prefix))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = B.alloc_attention_shared_workspace(8, 2, 64, 1, 20, 23, "cuda")

    def call():
        B.exl3_attention_shared(cache, q, starts, seq, table, gs, pl, max_new=1, max_group=20, scale=x["scale"], out=out, lse=lse,
                                workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    check(x, (out, lse))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for z, p in ((y, prefix), (x, prefix), (x, prefix // 2), (y, 0 * prefix)):
        q.copy_(cuda(z["q"]))
        seq.copy_(cuda(z["seq_len"]))
        pl.copy_(cuda(p))
        graph.replay()
        check(z, (out, lse))


def test_default_sizes_and_refusals():
    x, start, prefix = make(np.random.default_rng(4), 4, 2, 64, 16, [(40, [(5, 1), (7, 2)])])
    cache = B.Exl3KvCache.from_tensors(cuda(x["k"]), cuda(x["v"]), cuda(x["k_scale"]), cuda(x["v_scale"]))
    args = [cuda(x[n]) for n in ("q", "q_start", "seq_len", "block_table")]
    out = B.exl3_attention_shared(cache, *args, cuda(start), cuda(prefix))
    assert torch.equal(out, run(x, start, prefix, max_new=3, max_group=3, wide=False)[0])
    small = B.alloc_attention_shared_workspace(4, 2, 64, 3, 3, 2, "cuda")
    with pytest.raises(B.Exl3Error):
        B.exl3_attention_shared(cache, *args, cuda(start), cuda(prefix), max_new=3, max_group=3, workspace=small)
    with pytest.raises(ValueError):
        B.exl3_attention_shared(cache, *args, cuda(start), cuda(np.zeros(2, np.int32)))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    empty = B.exl3_attention_shared(cache, args[0][:0], torch.zeros(1, dtype=torch.int32, device="cuda"), none, args[3][:0],
                                    torch.zeros(1, dtype=torch.int32, device="cuda"), none)
    assert empty.shape == (0, 4, 64)


@pytest.mark.parametrize("heads,kv_heads,dim,groups", [
    (8, 2, 128, [(3000, [(300, 1), (9, 1), (200, 1)])]), (8, 2, 64, [(4000, [(200, 1)] * 40), (300, [(150, 1), (9, 1)])]),
    (4, 1, 128, [(700, [(200, 150), (300, 1)])])])
def test_rows_that_could_not_be_finished_are_nan(heads, kv_heads, dim, groups):
    """Waits that run out, without a GPU fault (the hook posts a range's first keys only): no row holds a plausible number."""
    x, start, prefix = make(np.random.default_rng(dim), heads, kv_heads, dim, 32, groups)
    new, most = int(np.diff(x["q_start"]).max()), int(x["q_start"][-1])
    ws = B.alloc_attention_shared_workspace(heads, kv_heads, dim, new, most, most, "cuda")
    B.exl3_debug_stall_tensor_wait(True)
    try:
        out, lse = run(x, start, prefix, max_group=most, workspace=ws, out=torch.full_like(cuda(x["q"]), 5.0))
        torch.cuda.synchronize()
    finally:
        B.exl3_debug_stall_tensor_wait(False)
    assert B.exl3_device_status(ws, 0) == 9            # EXL3_ERR_DEVICE_CHECK
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    ws.zero_()
    check(x, run(x, start, prefix, max_group=most, workspace=ws))
    assert B.exl3_device_status(ws, 0) == 0
