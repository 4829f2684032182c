"""The attention block (projections, plan, append, attention, output projection)
against the float64 oracle, over prompts, a chunk, single tokens, a request that
ends and one that takes its pages.

Tolerance: every projection is within 5e-3 relative L2 of its oracle; three of them
lie one behind the other (k or v, o; q in the exponent), and a value next to a
rounding boundary of the cache may fall to the other side (one step of 1/127 of a
page's largest value, for few values): 2e-2 relative L2.
"""
import numpy as np
import pytest
import torch

from oracle import exl3_oracle as O
from oracle import kv_oracle as KO
from trellis_decode_gemv_gb300 import attention_block as AB
from trellis_decode_gemv_gb300 import binding as B
from trellis_decode_gemv_gb300 import synth
from tests.gpu_helpers import upload

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE, PAGES, WIDTH = 256, 4, 2, 64, 16, 24, 12


def test_block_against_oracle():
    shapes = dict(q=(HEADS * DIM, HIDDEN), k=(KV * DIM, HIDDEN), v=(KV * DIM, HIDDEN), o=(HIDDEN, HEADS * DIM))
    host = {n: synth.layer_inputs(m, c, 4, 1, config=90, index=i) for i, (n, (m, c)) in enumerate(shapes.items())}
    dev = {}
    for n, (m, c) in shapes.items():
        host[n]["scales"] = (host[n]["scales"].astype(np.float32) * 4).astype(np.float16)   # outputs of about 1
        dev[n] = dict({k: t for k, t in upload(host[n]).items() if k != "x"}, K=4, cb=1, m=m, n=c)
    block = AB.AttentionBlock(dev, HEADS, KV, DIM, PAGES, PAGE, 160)
    pool = AB.PagePool(3, PAGES, PAGE, WIDTH)

    def linear(n, x):
        m, c = shapes[n]
        w = host[n]
        return O.layer_forward(w["codes"], 4, 1, m, c, w["s_in"], w["s_out"], w["scales"], x)

    k8 = np.zeros((2, PAGES, KV, PAGE, DIM), np.int8)
    scale = np.zeros((2, PAGES, KV), np.float32)
    ctx, ring, state, table = np.zeros(3, np.int32), np.arange(PAGES, dtype=np.int32), [0, PAGES], np.full((3, WIDTH), -1, np.int32)
    rng = np.random.default_rng(4)
    for new in ([70, 33, 5], [1, 20, 1], [1, 1, 1], [-1, 1, 1], [40, 1, 1], [1, 1, 1]):
        tokens = sum(max(n, 0) for n in new)
        x = rng.standard_normal((tokens, HIDDEN)).astype(np.float16)
        step = pool.step(torch.tensor(new, dtype=torch.int32, device="cuda"), tokens)
        y = block(torch.from_numpy(x).cuda(), step, max(new)).double().cpu().numpy()

        p = KO.plan(ctx, new, tokens, PAGE, ring, state, table)
        ring, state, table = p["free_pages"], p["free_state"], p["block_table"]
        assert np.array_equal(step.seq_len.cpu().numpy(), p["seq_len"]) and np.array_equal(step.slot.cpu().numpy(), p["slot"])
        q, k, v = (linear(n, x).astype(np.float16).reshape(tokens, -1, DIM) for n in "qkv")
        for i, t in enumerate((k, v)):
            k8[i], scale[i] = KO.append(k8[i], scale[i], t, p["slot"])
        out, _, _ = KO.attention(k8[0], k8[1], scale[0], scale[1], q, p["q_start"], p["seq_len"], table, DIM ** -0.5)
        ref = linear("o", out.reshape(tokens, -1).astype(np.float16))
        rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
        assert np.isfinite(y).all() and rel <= 2e-2, (new, rel)
        ctx = p["seq_len"]


def test_example_command(capsys):
    assert AB.main(["--layers", "2", "--requests", "3", "--prompt", "40", "--steps", "3", "--hidden", "256", "--heads", "4x2x64",
                    "--page", "16"]) == 0
    assert "ms a step" in capsys.readouterr().out
