"""The attention part of a decoder on quantized projections: q, k and v by
exl3_gemm, new keys and values into a paged 8-bit cache, attention over it, the
output projection.  Shows the cache operators as a server uses them:

    pool = PagePool(requests, pages, page_size, width)
    for every step:                              # prompts, chunks of prompts, single tokens
        step = pool.step(new_len, tokens)        # one launch, no word to the host
        for block in blocks:
            x = x + block(x, step, max_new)      # x [tokens, hidden] halves
    pool.step with -1 new tokens gives a finished request's pages back.

    python -m trellis_decode_gemv_gb300.attention_block --layers 4 --requests 8 --prompt 500 --steps 32

Position encodings are the model's business: step.position holds every token's
position, and whatever rotates q and k goes between the projections and the cache.
"""
from __future__ import annotations

import argparse
from types import SimpleNamespace

import torch

from . import binding as B


class PagePool:
    """Pages, block tables and lengths of up to `requests` running requests, all in
    device memory and shared by the caches of all layers."""

    def __init__(self, requests, pages, page_size, width, device="cuda"):
        self.page_size = page_size
        self.ctx_len = torch.zeros(requests, dtype=torch.int32, device=device)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=device)
        self.ring = torch.arange(pages, dtype=torch.int32, device=device)
        self.state = torch.tensor([0, pages, 0], dtype=torch.int32, device=device)

    def step(self, new_len, tokens):
        """Pages and slots for new_len [requests] int32 new tokens (`tokens` of them
        in all; -1: the request is finished).  step.state[2] counts pages that were
        lacking; requests that got none keep their length."""
        seq_len, q_start, slot, position, self.state = B.exl3_kv_plan(
            self.ctx_len, new_len, tokens, self.page_size, self.ring, self.state, self.table)
        self.ctx_len = seq_len
        return SimpleNamespace(seq_len=seq_len, q_start=q_start, slot=slot, position=position, state=self.state,
                               table=self.table)


class AttentionBlock:
    """One layer.  weights: q, k, v, o as dicts of codes, K, cb, m, n, s_in, s_out,
    scales (the arguments of Exl3Linear)."""

    def __init__(self, weights, heads, kv_heads, head_dim, pages, page_size, max_tokens, device="cuda"):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.proj = {name: B.Exl3Linear(w["codes"], w["K"], w["cb"], w["m"], w["n"], w["s_in"], w["s_out"], w["scales"],
                                        max_batch=max_tokens) for name, w in weights.items()}
        self.cache = B.Exl3KvCache(pages, kv_heads, page_size, head_dim, device)
        self.workspace = B.alloc_attention_workspace(heads, kv_heads, head_dim, max_tokens, device)

    def __call__(self, x, step, max_new):
        """x [tokens, hidden] halves -> the block's output (no residual)."""
        tokens = x.shape[0]
        q = self.proj["q"](x).view(tokens, self.heads, self.head_dim)
        k = self.proj["k"](x).view(tokens, self.kv_heads, self.head_dim)
        v = self.proj["v"](x).view(tokens, self.kv_heads, self.head_dim)
        B.exl3_kv_append(self.cache, k, v, step.slot)
        out = B.exl3_attention(self.cache, q, step.q_start, step.seq_len, step.table, max_new=max_new,
                               workspace=self.workspace)
        return self.proj["o"](out.view(tokens, -1))


def random_weights(hidden, heads, kv_heads, head_dim, K, cb, seed, device="cuda"):
    """Random projections of the right shapes (uniform code words are legal streams)."""
    from .profcase import _layer
    shapes = dict(q=(heads * head_dim, hidden), k=(kv_heads * head_dim, hidden), v=(kv_heads * head_dim, hidden),
                  o=(hidden, heads * head_dim))
    return {name: dict(_layer(m, n, K, 1, seed + 10 * i, device), K=K, cb=cb) for i, (name, (m, n)) in enumerate(shapes.items())}


def main(argv=None):
    ap = argparse.ArgumentParser(description="prompts, then single tokens, through quantized attention blocks")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", default="32x8x128", help="query heads x key/value heads x head dimension")
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args(argv)
    heads, kv_heads, dim = map(int, a.heads.split("x"))
    dev = torch.device("cuda", torch.cuda.current_device())
    width = -(-(a.prompt + a.steps) // a.page)
    pages, most = a.requests * width, a.requests * a.prompt
    pool = PagePool(a.requests, pages, a.page, width, dev)
    blocks = [AttentionBlock(random_weights(a.hidden, heads, kv_heads, dim, 3, B.CB_3INST, 1000 * i, dev), heads, kv_heads, dim,
                             pages, a.page, most, dev) for i in range(a.layers)]

    def run(x, new):
        step = pool.step(torch.full((a.requests,), new, dtype=torch.int32, device=dev), a.requests * new)
        for block in blocks:
            x = x + block(x, step, new)
        return x

    events = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    x = torch.randn((most, a.hidden), device=dev).half()
    events[0].record()
    x = run(x, a.prompt).view(a.requests, a.prompt, -1)[:, -1].contiguous()
    events[1].record()
    for _ in range(a.steps):
        x = run(x, 1)
    events[2].record()
    torch.cuda.synchronize()
    assert pool.ctx_len.tolist() == [a.prompt + a.steps] * a.requests and int(pool.state[2]) == 0
    print(f"{a.layers} blocks, {a.requests} requests: prompts of {a.prompt} tokens {events[0].elapsed_time(events[1]):.2f} ms, "
          f"then {events[1].elapsed_time(events[2]) / a.steps:.3f} ms a step over {a.steps} steps")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
