"""Rings that are full, and rings and tables whose places are numbered near 2^31: exl3_kv_fork and
exl3_kv_plan.  Whole numbers, worked out by hand."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def fork(parent, ctx, page, pages, ring, state, table):
    f = B.exl3_kv_fork(ints(parent), ints(ctx), page, pages, ring, ints(state), table)
    return f, f.free_state.tolist()


@pytest.mark.parametrize("rows,state,ring", [(5, [2, 4, 0], [2, 5, 0, 1]), (3, [0, 4, 0], [8, 9, 0, 1]), (4, [1, 4, 0], [2, 9, 0, 1]),
                                             (1, [2, 4, 0], [8, 9, 6, 7]), (7, [2, 4, 2], [2, 5, 0, 1])])
def test_a_full_ring_takes_back_as_many_pages_as_it_gave(rows, state, ring):
    pages = ints([8, 9, 6, 7])
    f, got = fork([0] * rows, [20, 64], 16, 10, pages, [2, 4], ints([[3, 4, -1, -1], [0, 1, 2, 5]]))
    assert got == state and pages.tolist() == ring
    assert f.block_table.tolist() == [[3, p, -1, -1] for p in (4, 6, 7, 8, 9)][:rows] + [[-1] * 4] * max(rows - 5, 0)


def test_many_rows_of_a_full_ring():
    """More pages than a block appends at once, from several clusters."""
    rng = np.random.default_rng(1)
    page, requests, rows = 16, 700, 900
    ctx = rng.integers(1, 400, requests)
    need = -(-ctx // page)
    table = np.full((requests, int(need.max())), -1, np.int32)
    pages = int(need.sum()) + rows
    order = rng.permutation(pages).astype(np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    for cap in (rows, rows + 50, rows + 5000):
        ring = np.full(cap, -1, np.int32)
        head = int(rng.integers(0, cap))
        ring[(head + np.arange(rows)) % cap] = order[at:at + rows]
        x = dict(ctx_len=ctx, page_size=page, pages=pages, free_pages=ring, free_state=[head, rows], block_table=table)
        parent = rng.integers(0, 200, rows)
        want = BO.fork(parent, **x)
        got_ring = ints(ring)
        f, state = fork(parent, ctx, page, pages, got_ring, [head, rows], ints(table))
        assert state == want["free_state"].tolist() and np.array_equal(got_ring.cpu().numpy(), want["free_pages"])
        assert np.array_equal(f.block_table.cpu().numpy(), want["block_table"])


def room_for(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free memory")


@pytest.mark.parametrize("head", [-2, 2 ** 30 + 6])
def test_ring_of_more_than_a_billion_places(head):
    """Head near the end: places and their sums pass 2^31 before they come round."""
    room_for(6)
    cap = 2 ** 30 + 8
    ring = torch.empty(cap, dtype=torch.int32, device="cuda")
    at = torch.tensor([cap - 2, cap - 1, 0, 1, 2, 3, 4], device="cuda")
    ring[at] = ints([6, 7, 8, 9, -1, -1, -1])
    f, state = fork([0] * 4, [20, 32], 16, 10, ring, [head, 4], ints([[3, 4], [1, 2]]))
    assert state == [1, 3, 0] and f.block_table.tolist() == [[3, 4], [3, 6], [3, 7], [3, 8]]
    assert ring[at].tolist() == [6, 7, 8, 9, 1, 2, -1]
    ring[at] = ints([6, 7, 8, 9, -1, -1, -1])
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    table[1, :2] = ints([1, 2])
    seq_len, _, slot, position, out = B.exl3_kv_plan(ints([0, 32]), ints([60, -1]), 60, 16, ring, ints([head, 4, 0]), table)
    assert seq_len.tolist() == [60, 0] and table[0].tolist() == [6, 7, 8, 9] and out.tolist() == [2, 2, 0]
    assert slot.tolist() == [16 * (6 + i // 16) + i % 16 for i in range(60)] and position.tolist() == list(range(60))
    assert ring[at].tolist() == [6, 7, 8, 9, 1, 2, -1]
    del ring
    torch.cuda.empty_cache()


def test_request_of_all_tokens_that_have_a_number():
    """2^31 - 1 tokens: its pages go back when it ends, and go on when it does."""
    width, pages = 1 << 24, 1010
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(width, dtype=torch.int32, device="cuda") % 1000
    table[1, 0] = 1005
    ctx = [2 ** 31 - 1, 20]
    ring = torch.full((2000,), -1, dtype=torch.int32, device="cuda")
    f, state = fork([1], ctx, 128, pages, ring, [7, 0], table)
    assert state == [7, 1000, 0] and ring[7:1007].tolist() == list(range(1000)) and bool((ring[1007:] == -1).all())
    assert f.ctx_len.tolist() == [20] and f.block_table[0, :2].tolist() == [1005, -1]
    ring[7] = 1007
    f, state = fork([0, 0], ctx, 128, pages, ring, [7, 1], table)
    assert state == [8, 1, 0] and ring[8] == 1005      # the second request ends
    assert f.ctx_len.tolist() == [2 ** 31 - 1] * 2 and f.copy_tokens.tolist() == [0, 127]
    assert f.copy_from.tolist() == [-1, (width - 1) % 1000] and f.copy_to.tolist() == [-1, 1007]
    assert torch.equal(f.block_table[0], table[0]) and torch.equal(f.block_table[1, :-1], table[0, :-1]) and f.block_table[1, -1] == 1007
