"""exl3_kv_fork and exl3_kv_copy on the GPU against the oracle: whole numbers and
moved bytes, equal bit for bit."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def cuda(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).cuda()


def make(rng, requests, page, most, spare, share=0.4, extra_width=0, extra_ring=0):
    """Tables whose requests share leading pages with the one before them now and then; the ring's head anywhere."""
    ctx = rng.integers(0, most + 1, requests)
    need = -(-ctx // page)
    width = max(int(need.max(initial=1)), 1) + extra_width
    pages = int(need.sum()) + spare + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((requests, width), -7, np.int32)
    at = 0
    for b in range(requests):
        same = min(ctx[b] // page, ctx[b - 1] // page) if b and rng.random() < share else 0
        table[b, :same] = table[b - 1, :same]
        table[b, same:need[b]] = order[at:at + need[b] - same]
        at += need[b] - same
    cap = pages + extra_ring
    ring = np.full(cap, -1, np.int32)
    head = int(rng.integers(0, cap))
    ring[(head + np.arange(spare)) % cap] = order[at:at + spare]
    return dict(ctx_len=ctx, page_size=page, pages=pages, free_pages=ring, free_state=[head, spare], block_table=table)


def run(x, parent, workspace=None, out=None):
    ring = cuda(x["free_pages"])
    f = B.exl3_kv_fork(cuda(parent, np.int32), cuda(x["ctx_len"], np.int32), x["page_size"], x["pages"], ring,
                       cuda(x["free_state"], np.int32), cuda(x["block_table"]), workspace=workspace, out=out)
    return dict(ctx_len=f.ctx_len, block_table=f.block_table, copy_from=f.copy_from, copy_to=f.copy_to, copy_tokens=f.copy_tokens,
                free_state=f.free_state, free_pages=ring)


def check(x, parent, workspace=None):
    want = BO.fork(parent, **x)
    got = run(x, parent, workspace)
    for name, ref in want.items():
        assert np.array_equal(got[name].cpu().numpy(), ref), name
    return want


@pytest.mark.parametrize("requests,rows,page,most,spare", [
    (1, 1, 16, 0, 0), (1, 1, 16, 40, 0), (1, 8, 64, 100, 9), (1, 500, 32, 5000, 600), (16, 64, 16, 2000, 80), (7, 3, 128, 1000, 4),
    (500, 509, 64, 8000, 520), (33, 1025, 16, 30, 1100), (1025, 33, 16, 30, 40), (8192, 8192, 16, 20, 8200), (300, 2000, 16, 16000, 2000)])
def test_fork(requests, rows, page, most, spare):
    rng = np.random.default_rng(requests + rows)
    x = make(rng, requests, page, most, spare)
    alive = rng.permutation(requests)[:max(1, requests // 3)]
    parent = rng.choice(alive, rows)
    parent[rng.random(rows) < 0.1] = -1
    ws = B.alloc_kv_fork_workspace(x["pages"], "cuda")
    check(x, parent, ws)
    assert not ws.any()
    check(x, rng.integers(0, requests, rows), ws)
    check(x, np.arange(rows) % requests, ws)          # each in its place, then once more


@pytest.mark.parametrize("spare", [0, 1, 5, 19])
def test_fork_without_enough_pages(spare):
    rng = np.random.default_rng(spare)
    x = make(rng, 6, 16, 100, spare)
    want = check(x, rng.integers(0, 6, 40))
    assert want["free_state"][2] > 0


def test_fork_of_nothing_and_into_nothing():
    rng = np.random.default_rng(2)
    x = make(rng, 9, 32, 300, 4)
    check(x, np.zeros(0, np.int32))                    # all requests end
    check(x, np.full(5, -1))
    check(x, np.array([9, 100, -5, 2]))                # parents that are no requests
    y = dict(x, ctx_len=np.zeros(0, np.int64), block_table=np.zeros((0, 4), np.int32))
    check(y, np.zeros(0, np.int32))
    check(y, np.array([0, 1]))
    check(dict(x, ctx_len=np.zeros(9, np.int64)), np.arange(9))


def test_fork_cuts_lengths_and_keeps_odd_entries():
    """Lengths beyond the table's rows, negative ones; page numbers outside the pool are carried along and never returned;
    a ring too small for what comes back; counts out of range."""
    rng = np.random.default_rng(3)
    x = make(rng, 12, 16, 200, 6)
    x["ctx_len"][[1, 5]] = [10 ** 6, -4]
    x["block_table"][2, 0], x["block_table"][4, 0] = 2 ** 30, -3
    parent = np.array([0, 1, 1, 2, 2, 5, 8])
    check(x, parent)
    small = dict(x, free_pages=x["free_pages"][:8].copy(), free_state=[3, 2])
    small["free_pages"][[3, 4]] = [x["pages"] - 1, x["pages"] - 2]
    check(small, parent)
    check(dict(small, free_pages=np.zeros(0, np.int32), free_state=[0, 0]), parent)
    check(dict(x, free_state=[-5, 10 ** 6]), np.arange(12))


def test_fork_of_wide_tables():
    """Rows of 8000 pages: many clusters."""
    rng = np.random.default_rng(4)
    x = make(rng, 40, 16, 128000, 90)
    check(x, rng.integers(0, 30, 100))


def test_fork_captured_and_into_given_outputs():
    rng = np.random.default_rng(5)
    x = make(rng, 20, 16, 400, 60)
    parent = cuda(rng.integers(0, 15, 40), np.int32)
    ring, ctx, state, table = cuda(x["free_pages"]), cuda(x["ctx_len"], np.int32), cuda(x["free_state"], np.int32), cuda(x["block_table"])
    ws = B.alloc_kv_fork_workspace(x["pages"], "cuda")
    out = B.Exl3KvFork(40, table.shape[1], torch.device("cuda", torch.cuda.current_device()))
    B.exl3_kv_fork(parent, ctx, 16, x["pages"], ring, state, table, workspace=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = B.exl3_kv_fork(parent, ctx, 16, x["pages"], ring, state, table, workspace=ws, out=out)
    assert f is out
    for seed in range(3):
        p = np.random.default_rng(seed).integers(-1, 20, 40)
        parent.copy_(cuda(p, np.int32))
        ring.copy_(cuda(x["free_pages"]))
        graph.replay()
        want = BO.fork(p, **x)
        for name in ("ctx_len", "block_table", "copy_from", "copy_to", "copy_tokens", "free_state"):
            assert np.array_equal(getattr(f, name).cpu().numpy(), want[name]), name
        assert np.array_equal(ring.cpu().numpy(), want["free_pages"])
    with pytest.raises(ValueError):
        B.exl3_kv_fork(parent, ctx, 16, x["pages"], ring, state, table, workspace=ws, out=B.Exl3KvFork(39, table.shape[1], table.device))
    for args in ((f.ctx_len[:20], state, table), (ctx, f.free_state, table), (ctx, state, f.block_table)):
        with pytest.raises(ValueError):                # its own results as inputs
            B.exl3_kv_fork(parent, args[0], 16, x["pages"], ring, *args[1:], workspace=ws, out=f)


# ---- copy ----------------------------------------------------------------------------

def check_copy(rng, layers, pages, heads, page, dim, src, dst, tokens):
    q = rng.integers(-128, 128, (2, layers, pages, heads, page, dim)).astype(np.int8)
    s = rng.standard_normal((2, layers, pages, heads)).astype(np.float32)
    s[0, 0, 0, 0] = np.nan
    caches = [B.Exl3KvCache.from_tensors(cuda(q[0, i]), cuda(q[1, i]), cuda(s[0, i]), cuda(s[1, i])) for i in range(layers)]
    B.exl3_kv_copy(B.Exl3KvCacheGroup(caches), cuda(src, np.int32), cuda(dst, np.int32), cuda(tokens, np.int32))
    for i, c in enumerate(caches):
        for j, (got, got_scale) in enumerate(((c.k, c.k_scale), (c.v, c.v_scale))):
            ref, ref_scale = BO.copy(q[j, i], s[j, i], src, dst, tokens)
            assert np.array_equal(got.cpu().numpy(), ref) and np.array_equal(got_scale.cpu().numpy(), ref_scale, equal_nan=True), (i, j)


@pytest.mark.parametrize("layers,heads,page,dim", [(1, 1, 16, 64), (3, 2, 64, 128), (64, 1, 16, 64), (65, 1, 16, 64), (2, 8, 128, 128),
                                                   (2, 5, 32, 64), (300, 1, 16, 64)])
def test_copy(layers, heads, page, dim):
    rng = np.random.default_rng(layers + heads)
    pages, pairs = 24, 9
    order = rng.permutation(pages)
    tokens = rng.integers(1, page + 1, pairs)
    tokens[:4] = [1, page, page - 1, min(17, page)]
    check_copy(rng, layers, pages, heads, page, dim, order[:pairs], order[pairs:2 * pairs], tokens)


def test_copy_skips_and_cuts():
    rng = np.random.default_rng(3)
    check_copy(rng, 2, 12, 2, 16, 64, [0, -1, 3, 4, 99, 5, 0], [6, 7, -1, 8, 9, 12, 10], [5, 6, 7, 99, 3, 2, 0])


def test_copy_from_one_page_to_many_past_four_gigabytes():
    page, heads, dim = 128, 8, 128
    pages = (5 << 30) // (page * heads * dim)
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free memory")
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    k[0] = torch.randint(-127, 128, k[0].shape, device="cuda", dtype=torch.int8)
    v[0] = torch.randint(-127, 128, v[0].shape, device="cuda", dtype=torch.int8)
    s = torch.rand((2, pages, heads), device="cuda")
    cache = B.Exl3KvCacheGroup([B.Exl3KvCache.from_tensors(k, v, s[0], s[1])])
    to = cuda([pages - 1, pages // 2, 5], np.int32)
    B.exl3_kv_copy(cache, torch.zeros(3, dtype=torch.int32, device="cuda"), to, cuda([100, 128, 3], np.int32))
    for p, n in ((pages - 1, 100), (pages // 2, 128), (5, 3)):
        assert torch.equal(k[p, :, :n], k[0, :, :n]) and torch.equal(v[p, :, :n], v[0, :, :n]) and not k[p, :, n:].any()
        assert torch.equal(s[:, p], s[:, 0])
