"""exl3_kv_plan and exl3_kv_append on the GPU against the oracle: whole numbers
and scales are equal, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def cuda(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).cuda()


# ---- plan --------------------------------------------------------------------------

def plan_inputs(rng, requests, page, most_ctx, most_new, width, spare, done=0.1, none=0.1):
    ctx = rng.integers(0, most_ctx + 1, requests)
    new = rng.integers(1, most_new + 1, requests)
    new[rng.random(requests) < none] = 0
    new[rng.random(requests) < done] = -1
    have = -(-ctx // page)
    width = max(width, int(have.max(initial=0)), 1)
    total = int(have.sum()) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((requests, width), -1, np.int32)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    ring = np.full(total, -1, np.int32)
    head = int(rng.integers(0, max(total, 1)))
    ring[(head + np.arange(spare)) % max(total, 1)] = order[at:]
    return ctx, new, ring, [head, spare], table


def check_plan(ctx, new, ring, state, table, page, tokens):
    want = KO.plan(ctx, new, tokens, page, ring, state, table)
    d_table, d_ring = cuda(table), cuda(ring)
    got = B.exl3_kv_plan(cuda(ctx, np.int32), cuda(new, np.int32), tokens, page, d_ring, cuda(state, np.int32), d_table)
    got = dict(zip(("seq_len", "q_start", "slot", "position", "free_state"), got), block_table=d_table, free_pages=d_ring)
    for name, ref in want.items():
        assert np.array_equal(got[name].cpu().numpy(), ref), name


@pytest.mark.parametrize("requests,page,most_ctx,most_new,width,spare", [
    (1, 16, 0, 1, 4, 2), (1, 64, 100, 1, 8, 3), (7, 32, 50, 40, 9, 40), (64, 64, 3000, 1, 60, 64),
    (255, 16, 100, 3, 20, 300), (257, 128, 1000, 200, 16, 600), (1025, 16, 40, 20, 8, 2000), (8192, 16, 30, 1, 4, 9000),
    (3, 16, 10, 5000, 400, 2000),
])
def test_plan(requests, page, most_ctx, most_new, width, spare):
    rng = np.random.default_rng(requests + page)
    ctx, new, ring, state, table = plan_inputs(rng, requests, page, most_ctx, most_new, width, spare)
    check_plan(ctx, new, ring, state, table, page, int(np.maximum(new, 0).sum()) + 5)  # five tokens of nobody


@pytest.mark.parametrize("spare", [0, 1, 7, 30])
def test_plan_refuses_for_pages(spare):
    rng = np.random.default_rng(spare)
    ctx, new, ring, state, table = plan_inputs(rng, 40, 16, 60, 50, 12, spare)
    check_plan(ctx, new, ring, state, table, 16, int(np.maximum(new, 0).sum()))


def test_plan_refuses_for_the_table_and_for_tokens():
    rng = np.random.default_rng(3)
    ctx, new, ring, state, table = plan_inputs(rng, 30, 16, 64, 40, 4, 200)   # rows of 4 pages: 64 tokens
    total = int(np.maximum(new, 0).sum())
    check_plan(ctx, new, ring, state, table, 16, total)
    check_plan(ctx, new, ring, state, table, 16, total // 2)


def test_plan_of_nothing():
    state = cuda([3, 2, 9], np.int32)
    out = B.exl3_kv_plan(cuda([], np.int32), cuda([], np.int32), 0, 16, cuda(np.arange(5), np.int32), state,
                         torch.zeros((0, 4), dtype=torch.int32, device="cuda"))
    assert out[1].tolist() == [0] and out[4].tolist() == [3, 2, 0]
    check_plan([5, 0], [0, 0], np.zeros(0, np.int32), [0, 0], np.full((2, 2), 4, np.int32), 16, 0)


# ---- append --------------------------------------------------------------------------

def slots_of(table, ctx, new, page):
    return np.array([int(table[b][(c + i) // page]) * page + (c + i) % page
                     for b, (c, n) in enumerate(zip(ctx, new)) for i in range(n)], np.int64)


def check_append(rng, heads, dim, page, ctx, new, edit=None, pad=0, spread=0.5):
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n])
        at += n
    q8 = rng.integers(-127, 128, (2, pages, heads, page, dim)).astype(np.int8)
    scale = (0.01 * np.exp(spread * rng.standard_normal((2, pages, heads)))).astype(np.float32)
    tokens = sum(new)
    x = (np.exp(spread * rng.standard_normal((2, tokens, 1, 1))) * rng.standard_normal((2, tokens, heads, dim))).astype(np.float16)
    slot = slots_of(table, ctx, new, page)
    if edit:
        edit(q8, scale, x, slot)
    cache = B.Exl3KvCache.from_tensors(cuda(q8[0]), cuda(q8[1]), cuda(scale[0]), cuda(scale[1]))
    wide = torch.zeros((tokens, 2 * heads + pad, dim), dtype=torch.float16, device="cuda")  # a fused projection's output
    wide[:, :heads], wide[:, heads + pad:] = cuda(x[0]), cuda(x[1])
    for call in range(2):  # the second call finds its own results and changes nothing
        B.exl3_kv_append(cache, wide[:, :heads], wide[:, heads + pad:], cuda(slot))
        for i, (got, got_scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
            ref, ref_scale = KO.append(q8[i], scale[i], x[i], slot)
            assert np.array_equal(got_scale.cpu().numpy(), ref_scale, equal_nan=True), (call, i)
            assert np.array_equal(got.cpu().numpy(), ref), (call, i)


@pytest.mark.parametrize("heads,dim,page,ctx,new", [
    (1, 64, 16, [0], [1]), (1, 128, 128, [127], [1]), (8, 128, 64, [0, 63, 64, 65, 200], [1, 1, 1, 1, 1]),
    (2, 64, 32, [5, 31, 0], [100, 2, 33]), (3, 128, 16, [7, 16], [250, 16]), (5, 64, 128, [1, 0, 300], [127, 129, 1]),
    (8, 128, 64, [10, 0, 130, 64], [700, 64, 1, 190]), (1, 128, 32, [0] * 130, [1] * 130),
])
def test_append(heads, dim, page, ctx, new):
    check_append(np.random.default_rng(heads * dim + page), heads, dim, page, ctx, new)


def test_append_from_a_strided_projection_and_skips():
    def skip(q8, scale, x, slot):
        slot[3:20] = -1                        # a refused request's tokens
        slot[40] = 10 ** 12                    # a slot outside the cache
    check_append(np.random.default_rng(1), 2, 128, 32, [3, 0, 50], [10, 30, 64], edit=skip, pad=3)


def test_append_zeros_ties_and_extremes():
    def edit(q8, scale, x, slot):
        x[:, 0] = 0                            # opens a page with zeros: scale 0
        x[:, 1:33, :, :] = 0
        x[:, 1:33, :, 0] = 127                 # scale 1: halves are ties
        x[:, 1:33, :, 1:40] = np.arange(39) * 0.5 - 9.5
        x[:, 33:40] = np.float16(6e-8)         # the smallest subnormal
        x[:, 40:50] = np.float16(65504)
    check_append(np.random.default_rng(2), 2, 64, 16, [0, 0, 0, 0], [1, 32, 7, 10], edit=edit)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_append_of_what_is_not_finite(bad):
    def edit(q8, scale, x, slot):
        x[0, 4, 1, 9] = bad
    check_append(np.random.default_rng(5), 3, 64, 32, [9, 3], [12, 5], edit=edit)

    def poisoned(q8, scale, x, slot):          # a page that was spoilt before stays so
        scale[0, int(slot[0]) // 32] = np.nan
    check_append(np.random.default_rng(6), 3, 64, 32, [9, 3], [2, 5], edit=poisoned)


def test_append_past_four_gigabytes():
    page, heads, dim = 128, 8, 128
    pages = (5 << 30) // (page * heads * dim)
    free = torch.cuda.mem_get_info()[0]
    if free < 12 << 30:
        pytest.skip("needs 12 GB of free memory")
    k = torch.empty((pages, heads, page, dim), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    scale = torch.zeros((2, pages, heads), device="cuda")
    cache = B.Exl3KvCache.from_tensors(k, v, scale[0], scale[1])
    x = torch.randn((3, heads, dim), device="cuda").half()
    last = pages * page - 128
    slot = torch.tensor([last, last + 1, last + 2], device="cuda")
    B.exl3_kv_append(cache, x, x, slot)
    q, s = KO.append(np.zeros((1, heads, page, dim), np.int8), np.zeros((1, heads), np.float32), x.cpu().numpy(), [0, 1, 2])
    assert np.array_equal(k[-1, :, :3].cpu().numpy(), q[0, :, :3]) and np.array_equal(v[-1, :, :3].cpu().numpy(), q[0, :, :3])
    assert np.array_equal(scale[:, -1].cpu().numpy(), np.stack([s[0], s[0]]))
