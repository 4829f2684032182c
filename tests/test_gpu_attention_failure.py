"""Waits of the attention kernels that run out, without a GPU fault: with the test
hook on, a block's producer posts the first keys of its range and nothing after.
The call ends by itself, the status word is set, rows whose keys were not all read
are NaN (also where blocks join their partial results) and none holds a plausible
number, and the next call on a cleared workspace is right.
"""
import time

import numpy as np
import pytest
import torch

from tests import test_gpu_attention as A
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads,dim,seq,new", [
    (8, 2, 128, [300, 200, 0, 20000, 8], [1, 1, 1, 1, 0]),          # few rows: whole items, split ones, a row that sees nothing
    (16, 1, 64, [70000], [1]),                                      # joined in two steps
    (4, 2, 128, [300, 700, 30], [150, 70, 30]),                     # many rows
    (4, 1, 64, [20000, 4000], [100, 60]),                           # many rows, split
    (8, 2, 64, [900, 1, 3000, 2500], [200, 1, 3, 1]),               # both kernels
])
def test_rows_that_could_not_be_finished_are_nan(heads, kv_heads, dim, seq, new):
    x = A.make(np.random.default_rng(dim), heads, kv_heads, dim, 32, seq, new)
    ws = B.alloc_attention_workspace(heads, kv_heads, dim, max(new), "cuda")
    B.exl3_debug_stall_tensor_wait(True)
    try:
        t0 = time.perf_counter()
        out, lse = A.run(x, workspace=ws, out=torch.full_like(A.cuda(x["q"]), 5.0))
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        B.exl3_debug_stall_tensor_wait(False)
    print(f"stalled call returned after {elapsed:.3f} s")
    assert elapsed < 60.0
    assert B.exl3_device_status(ws, 0) == 9     # EXL3_ERR_DEVICE_CHECK
    at = 0
    for n, m in zip(seq, new):
        rows = slice(at, at + m)
        if n == 0:
            assert bool((out[rows] == 0).all()) and bool((lse[rows] == -np.inf).all())
        elif n > 128:                           # more than one unit of keys, whatever the range
            assert bool(torch.isnan(lse[rows][-1]).all()) and bool(torch.isnan(out[rows][-1]).all()), (n, m)
            assert bool((torch.isnan(lse[rows]) == torch.isnan(out[rows]).all(-1)).all())
        at += m
    ws.zero_()
    A.check(x, A.run(x, workspace=ws))
    assert B.exl3_device_status(ws, 0) == 0
