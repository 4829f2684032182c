"""Calls behind one another without a pause: kernels that begin where the blocks of the one
before end read nothing of it too early and write nothing it still reads.  Each chain
is compared with the same calls one at a time; buffers are written over again and again."""
import pytest
import torch

from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import upload

pytestmark = pytest.mark.gpu

N = 4096


def test_norms_rotary_and_copies_in_a_row():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.empty((3000, N), dtype=torch.float16, device="cuda") for _ in range(2))
    w = (1 + 0.2 * torch.randn(N, generator=g, device="cuda")).half()
    sign = torch.where(torch.randn(N, generator=g, device="cuda") < 0, -1.0, 1.0).half()
    position = torch.randint(0, 50000, (3000,), generator=g, device="cuda", dtype=torch.int32)
    f = B.exl3_rotary_freqs(128, base=500000.0)
    sources = [torch.randn((2, 3000, N), generator=g, device="cuda").half() for _ in range(4)]

    def chain(source, wait):
        x.copy_(source[0])
        r.copy_(source[1])
        wait()
        y, h = B.exl3_rms_norm(x, w, 1e-5, residual=r)
        wait()
        z, h2 = B.exl3_rms_norm(y, w, 1e-5, residual=h, h=r)       # over the first call's residual
        wait()
        q, s, _ = B.exl3_rms_norm_i8(z, w, 1e-5, [sign, None], residual=r, h=x)   # over the first call's x
        wait()
        B.exl3_rotary(z.view(3000, 32, 128), None, position, f, q_out=z.view(3000, 32, 128))
        wait()
        few, _ = B.exl3_rms_norm(z[:5], w, 1e-5, residual=x[:5])   # a few blocks behind many
        wait()
        x.zero_()
        return y, h, z, q, s, r.clone(), few

    want = [chain(s, torch.cuda.synchronize) for s in sources]
    for _ in range(3):
        got = [chain(s, lambda: None) for s in sources]
        assert all(torch.equal(a, b) for one, other in zip(got, want) for a, b in zip(one, other))


@pytest.mark.parametrize("M", [1, 2, 7, 40])
def test_projections_between_norms(M):
    """The projections' kernels begin early too: norm, layer, norm, int8 layer, over and over with the same buffers."""
    m, n, K = 512, 512, 3
    layers = [upload({k: v for k, v in synth.layer_inputs(m, n, K, 1, config=94, index=i).items() if k != "x"}) for i in range(2)]
    first, second = (B.Exl3Linear(t["codes"], K, B.CB_1MAD, m, n, t["s_in"], t["s_out"], t["scales"], max_batch=M) for t in layers)
    ws = torch.zeros(max(B.exl3_gemm_i8_workspace_bytes(m, n, min(M, 32)), 1), dtype=torch.uint8, device="cuda")
    w = torch.ones(n, device="cuda").half()
    g = torch.Generator(device="cuda").manual_seed(M)
    sources = [torch.randn((M, n), generator=g, device="cuda").half() for _ in range(12)]
    x, a, b = (torch.empty((M, n), dtype=torch.float16, device="cuda") for _ in range(3))

    def chain(source, wait):
        x.copy_(source)
        wait()
        y, _ = B.exl3_rms_norm(x, w, 1e-5, out=a)
        wait()
        first(y, b)
        wait()
        y, h = B.exl3_rms_norm(b, w, 1e-5, residual=x, out=a, h=x)
        wait()
        second(y, b)
        wait()
        out, _ = B.exl3_rms_norm(b, w, 1e-5, residual=h)
        if M <= 32:
            q, s, _ = B.exl3_rms_norm_i8(out, w, 1e-5, [layers[0]["s_in"]])
            wait()
            out = B.exl3_gemm_i8(layers[0]["codes"], K, B.CB_1MAD, m, n, layers[0]["s_out"], layers[0]["scales"], q[0], s[0], workspace=ws)
        wait()
        return out

    want = [chain(s, torch.cuda.synchronize) for s in sources]
    for _ in range(5):
        got = [chain(s, lambda: None) for s in sources]
        # binary16 results of layers in between may differ by a rounding each, the int8 step by its own: 1/127 of a block's largest
        for one, other in zip(got, want):
            assert bool(torch.isfinite(one).all())
            assert float((one.float() - other.float()).norm()) <= 2e-2 * float(other.float().norm())


def test_forks_and_copies_in_a_row():
    """Fork after fork and the copies of each, in graphs of many and one at a time."""
    g = torch.Generator(device="cuda").manual_seed(3)
    page, pages, layers = 16, 400, 6
    caches = [B.Exl3KvCache(pages, 4, page, 64) for _ in range(layers)]
    group = B.Exl3KvCacheGroup(caches)
    ws = B.alloc_kv_fork_workspace(pages, "cuda")
    start = [torch.randint(-127, 128, (2, pages, 4, page, 64), generator=g, device="cuda", dtype=torch.int8) for _ in range(layers)]
    parents = [torch.randint(-1, 20, (20,), generator=g, device="cuda", dtype=torch.int32) for _ in range(8)]
    ctx0 = torch.randint(1, 100, (20,), generator=g, device="cuda", dtype=torch.int32)
    table0 = torch.full((20, 7), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(ctx0.tolist()):
        k = -(-c // page)
        table0[b, :k] = torch.arange(at, at + k, dtype=torch.int32, device="cuda")
        at += k
    ring0 = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring0[:pages - at] = torch.arange(at, pages, dtype=torch.int32, device="cuda")
    state0 = torch.tensor([0, pages - at, 0], dtype=torch.int32, device="cuda")

    def chain(wait):
        for c, s in zip(caches, start):
            c.k.copy_(s[0])
            c.v.copy_(s[1])
        ctx, table, ring, state = ctx0.clone(), table0.clone(), ring0.clone(), state0.clone()
        for p in parents:
            wait()
            f = B.exl3_kv_fork(p, ctx, page, pages, ring, state, table, workspace=ws)
            wait()
            B.exl3_kv_copy(group, f.copy_from, f.copy_to, f.copy_tokens)
            ctx, table, state = f.ctx_len, f.block_table, f.free_state
        wait()
        return [ctx, table, ring, state] + [t.clone() for c in caches for t in (c.k, c.v)]

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, chain(lambda: None)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
