"""Norm, projections, rotary positions, cache, attention and output projection together,
over prompts, single tokens, forks of the requests and steps behind their shared
prompts, against the float64 oracles.

Tolerance: as of the attention block (2e-2 relative L2: projections of 5e-3 behind one
another, cache values next to a rounding boundary); the norm and the rotary positions
add roundings of 2^-11 before the projections.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from oracle import exl3_oracle as O
from oracle import kv_oracle as KO
from trellis_decode_gemv_gb300 import attention_block as AB
from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import upload

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE, PAGES = 256, 8, 2, 64, 16, 60
EPS, BASE = 1e-5, 10000.0


def cuda(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).cuda()


class Reference:
    """The same in numpy: one block and its pool."""

    def __init__(self, host, shapes, weight, requests, width, part):
        self.host, self.shapes, self.weight = host, shapes, weight
        self.k8 = np.zeros((2, PAGES, KV, PAGE, DIM), np.int8)
        self.scale = np.zeros((2, PAGES, KV), np.float32)
        self.ctx, self.ring, self.state = np.zeros(requests, np.int32), np.arange(PAGES, dtype=np.int32), [0, PAGES]
        self.table = np.full((requests, width), -1, np.int32)
        self.radians, self.factor = BO.frequencies(part, BASE)

    def linear(self, n, x):
        m, c = self.shapes[n]
        w = self.host[n]
        return O.layer_forward(w["codes"], 4, 1, m, c, w["s_in"], w["s_out"], w["scales"], x)

    def step(self, x, add, new, tokens):
        p = KO.plan(self.ctx, new, tokens, PAGE, self.ring, self.state, self.table)
        self.ring, self.state, self.table, self.ctx = p["free_pages"], p["free_state"], p["block_table"], p["seq_len"]
        y, h = BO.rms_norm(x, self.weight, EPS, add)
        q, k, v = (self.linear(n, y.astype(np.float16)).astype(np.float16).reshape(tokens, -1, DIM) for n in "qkv")
        q, k = (BO.rotary(t, p["position"], self.radians, self.factor).astype(np.float16) for t in (q, k))
        for i, t in enumerate((k, v)):
            self.k8[i], self.scale[i] = KO.append(self.k8[i], self.scale[i], t, p["slot"])
        out, _, _ = KO.attention(self.k8[0], self.k8[1], self.scale[0], self.scale[1], q, p["q_start"], p["seq_len"], self.table, DIM ** -0.5)
        return h, self.linear("o", out.reshape(tokens, -1).astype(np.float16))

    def fork(self, parent):
        f = BO.fork(parent, self.ctx, PAGE, PAGES, self.ring, self.state, self.table)
        self.ring, self.state, self.table, self.ctx = f["free_pages"], f["free_state"], f["block_table"], f["ctx_len"]
        for i in range(2):
            self.k8[i], self.scale[i] = BO.copy(self.k8[i], self.scale[i], f["copy_from"], f["copy_to"], f["copy_tokens"])


@pytest.mark.parametrize("part,width", [(64, 10), (32, 1700)])
def test_block_with_forks_against_oracle(part, width):
    """width 1700: tables that could hold enough for the kernels that look for shared keys."""
    shapes = dict(q=(HEADS * DIM, HIDDEN), k=(KV * DIM, HIDDEN), v=(KV * DIM, HIDDEN), o=(HIDDEN, HEADS * DIM))
    host = {n: synth.layer_inputs(m, c, 4, 1, config=92, index=i) for i, (n, (m, c)) in enumerate(shapes.items())}
    dev = {}
    for n, (m, c) in shapes.items():
        host[n]["scales"] = (host[n]["scales"].astype(np.float32) * 4).astype(np.float16)
        dev[n] = dict({k: t for k, t in upload(host[n]).items() if k != "x"}, K=4, cb=1, m=m, n=c)
    rng = np.random.default_rng(6)
    weight = (1 + 0.2 * rng.standard_normal(HIDDEN)).astype(np.float16)
    block = AB.AttentionBlock(dev, HEADS, KV, DIM, PAGES, PAGE, 160, norm=(cuda(weight), EPS), rotary=B.exl3_rotary_freqs(part, base=BASE),
                              max_shared=12)
    pool = AB.PagePool(3, PAGES, PAGE, width)
    caches = B.Exl3KvCacheGroup([block.cache])
    ref = Reference(host, shapes, weight, 3, width, part)

    def step(new, shared=None):
        tokens = sum(max(n, 0) for n in new)
        x, add = (rng.standard_normal((tokens, HIDDEN)).astype(np.float16) for _ in range(2))
        h, y = block(cuda(x), pool.step(cuda(new, np.int32), tokens), max(new), cuda(add),
                     None if shared is None else (cuda(shared[0], np.int32), cuda(shared[1], np.int32), shared[2]))
        h_ref, y_ref = ref.step(x, add, new, tokens)
        assert np.array_equal(pool.table.cpu().numpy(), ref.table) and np.array_equal(pool.ctx_len.cpu().numpy(), ref.ctx)
        assert np.abs(h.double().cpu().numpy() - h_ref).max() <= np.abs(h_ref).max() * 2.0 ** -10
        y = y.double().cpu().numpy()
        rel = np.linalg.norm(y - y_ref) / np.linalg.norm(y_ref)
        assert np.isfinite(y).all() and rel <= 2e-2, (new, rel)

    def fork(parent):
        pool.fork(cuda(parent, np.int32), caches)
        ref.fork(parent)
        assert np.array_equal(pool.ring.cpu().numpy(), ref.ring) and pool.state.tolist() == list(ref.state)

    step([70, 33, 5])
    step([1, 1, 1])
    fork([0, 0, 1, 0, 1, 0, 1])                       # four rows of the first, three of the second, the third ends
    order = [0, 1, 3, 5, 2, 4, 6]
    fork(order)                                       # groups beside one another
    groups = ([0, 4, 7], [71, 34])
    step([1] * 7, groups + (4,))
    step([1, 2, 1, 1, 0, 1, 3], groups + (5,))
    fork([0, 1, -1, 3, 4, 5, 6])                      # one ends, its place stays
    step([1, 1, 0, 1, 1, 1, 1], groups + (4,))
    fork([0, 1, 3, 3, -1, 6])
    step([1, 1, 1, 1, 0, 1], ([0, 4], [71], 4))       # the last belongs to no group
    step([1, 1, 1, 1, 0, 1])


def test_example_command_with_samples(capsys):
    assert AB.main(["--layers", "2", "--requests", "3", "--prompt", "40", "--steps", "3", "--hidden", "256", "--heads", "4x2x64",
                    "--page", "16", "--samples", "3"]) == 0
    assert "of 9 rows" in capsys.readouterr().out


def test_block_says_what_it_was_made_without():
    block = AB.AttentionBlock(AB.random_weights(256, 4, 2, 64, 3, B.CB_3INST, 1), 4, 2, 64, 8, 16, 8)
    pool = AB.PagePool(2, 8, 16, 4)
    one = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        block(torch.zeros((2, 256), dtype=torch.float16, device="cuda"), pool.step(torch.ones(2, dtype=torch.int32, device="cuda"), 2), 1,
              shared=(one, one[:1], 2))
