"""Calls on two streams at once, and in two branches of one graph, each with a workspace of its own: the bits
of the same calls one at a time."""
import numpy as np
import pytest
import torch

from tests import test_gpu_attention_shared as S
from trellis_decode_gemv_gb300 import binding as B

pytestmark = pytest.mark.gpu


def shared_call(seed, heads, kv_heads, dim, groups):
    x, start, prefix = S.make(np.random.default_rng(seed), heads, kv_heads, dim, 32, groups)
    cache = B.Exl3KvCache.from_tensors(*(S.cuda(x[n]) for n in ("k", "v", "k_scale", "v_scale")))
    args = [S.cuda(t) for t in (x["q"], x["q_start"], x["seq_len"], S.widened(x), start, prefix)]
    new = int(np.diff(x["q_start"]).max())
    most = max(int(x["q_start"][e] - x["q_start"][a]) for a, e in zip(start[:-1], start[1:]))
    ws = B.alloc_attention_shared_workspace(heads, kv_heads, dim, new, most, len(x["q"]), "cuda")
    return lambda: B.exl3_attention_shared(cache, *args, max_new=new, max_group=most, scale=x["scale"], lse=True, workspace=ws)


def test_at_once():
    one = shared_call(1, 8, 2, 64, [(900, [(50, 1)] * 40), (64, [(9, 2)] * 3)])         # both kernels
    other = shared_call(2, 8, 2, 128, [(2000, [(100, 1), (7, 2), (30, 1)]), (300, [(40, 1)] * 4)])   # the few-rows kernel
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn((700, 4096), generator=g, device="cuda").half() for _ in range(2))
    w = (1 + 0.2 * torch.randn(4096, generator=g, device="cuda")).half()
    sign = torch.where(torch.randn(4096, generator=g, device="cuda") < 0, -1.0, 1.0).half()

    def left():
        return *one(), *B.exl3_rms_norm(x, w, 1e-5, residual=r)

    def right():
        return *B.exl3_rms_norm_i8(x, w, 1e-5, [sign, None], residual=r), *other()

    want = [t.clone() for t in (*left(), *right())]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(50):
        with torch.cuda.stream(a):
            mine = left()
        with torch.cuda.stream(b):
            got.append((*mine, *right()))
    torch.cuda.synchronize()
    assert all(torch.equal(t, u) for call in got for t, u in zip(call, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        a.wait_stream(now)
        with torch.cuda.stream(a):
            mine = left()
        rest = right()
        now.wait_stream(a)
        y, h = B.exl3_rms_norm(mine[2], w, 1e-5, residual=rest[2])                      # behind both branches
    last = B.exl3_rms_norm(want[2], w, 1e-5, residual=want[6])
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip((*mine, *rest, y, h), (*want, *last)))
