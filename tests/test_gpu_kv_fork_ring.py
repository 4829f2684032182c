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
