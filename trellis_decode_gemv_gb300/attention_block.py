"""The attention part of a decoder on quantized projections: norm, q, k and v, rotary
positions, new keys and values into a paged 8-bit cache, attention over it, the
output projection.  Shows the operators around the projections as a server uses them:

    pool = PagePool(requests, pages, page_size, width)
    for every step:                              # prompts, chunks of prompts, single tokens
        step = pool.step(new_len, tokens)        # one launch, no word to the host
        add = None                               # what the block before adds to x
        for block in blocks:
            x, add = block(x, step, max_new, add)    # x [tokens, hidden] halves
    pool.step with -1 new tokens gives a finished request's pages back, if it shares none.
    pool.fork(parent) goes on with rows of other requests (samples of one prompt, beams): their
    pages are shared but for the last one, and rows that are not gone on with end; with shared=(group_start, prefix_len, max_group)
    the blocks then read the keys that a group's requests have in common once.

    python -m trellis_decode_gemv_gb300.attention_block --layers 4 --requests 8 --prompt 500 --steps 32 --samples 4

A block without norm and rotary frequencies (norm=None, rotary=None) leaves both to the
model, as it leaves the residual's addition: block(x, step, max_new) is its output alone.
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
        self.fork_workspace = B.alloc_kv_fork_workspace(pages, device)

    def step(self, new_len, tokens):
        """Pages and slots for new_len [requests] int32 new tokens (`tokens` of them
        in all; -1: the request is finished, and none of its pages is another's).  step.state[2] counts pages that were
        lacking; requests that got none keep their length."""
        seq_len, q_start, slot, position, self.state = B.exl3_kv_plan(
            self.ctx_len, new_len, tokens, self.page_size, self.ring, self.state, self.table)
        self.ctx_len = seq_len
        return SimpleNamespace(seq_len=seq_len, q_start=q_start, slot=slot, position=position, state=self.state,
                               table=self.table)


    def fork(self, parent, caches):
        """Go on with rows that continue the requests parent [rows] int32 (-1: an empty row), in
        any order, a request several times or not at all; `caches` the Exl3KvCacheGroup of all
        layers.  state[2] counts rows for which no page was left (they are empty)."""
        f = B.exl3_kv_fork(parent, self.ctx_len, self.page_size, self.ring.numel(), self.ring, self.state, self.table,
                           workspace=self.fork_workspace)
        B.exl3_kv_copy(caches, f.copy_from, f.copy_to, f.copy_tokens)
        self.ctx_len, self.table, self.state = f.ctx_len, f.block_table, f.free_state


class AttentionBlock:
    """One layer.  weights: q, k, v, o as dicts of codes, K, cb, m, n, s_in, s_out,
    scales (the arguments of Exl3Linear).  norm: (weight [hidden] halves, eps) of the norm
    before the projections, rotary: an Exl3RotaryFreqs; None: the model sees to them.
    max_shared: the most tokens of a call with shared prefixes (0: there is none)."""

    def __init__(self, weights, heads, kv_heads, head_dim, pages, page_size, max_tokens, device="cuda", norm=None, rotary=None,
                 interleaved=False, max_shared=0):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.norm, self.rotary, self.interleaved = norm, rotary, interleaved
        self.proj = {name: B.Exl3Linear(w["codes"], w["K"], w["cb"], w["m"], w["n"], w["s_in"], w["s_out"], w["scales"],
                                        max_batch=max_tokens) for name, w in weights.items()}
        self.cache = B.Exl3KvCache(pages, kv_heads, page_size, head_dim, device)
        self.workspace = B.alloc_attention_workspace(heads, kv_heads, head_dim, max_tokens, device)
        self.shared_workspace = None if max_shared == 0 else B.alloc_attention_shared_workspace(
            heads, kv_heads, head_dim, max_shared, max_shared, max_shared, device)

    def __call__(self, x, step, max_new, add=None, shared=None):
        """x [tokens, hidden] halves -> the block's output (no residual); with a norm: (x +
        add, the block's output), the sum made on the way to the norm.  shared: (group_start,
        prefix_len, max_group) of exl3_attention_shared."""
        tokens = x.shape[0]
        y = x
        if self.norm is not None:
            y, x = B.exl3_rms_norm(x, *self.norm, residual=add)
        q = self.proj["q"](y).view(tokens, self.heads, self.head_dim)
        k = self.proj["k"](y).view(tokens, self.kv_heads, self.head_dim)
        v = self.proj["v"](y).view(tokens, self.kv_heads, self.head_dim)
        if self.rotary is not None:
            B.exl3_rotary(q, k, step.position, self.rotary, interleaved=self.interleaved, q_out=q, k_out=k)
        B.exl3_kv_append(self.cache, k, v, step.slot)
        if shared is None:
            out = B.exl3_attention(self.cache, q, step.q_start, step.seq_len, step.table, max_new=max_new,
                                   workspace=self.workspace)
        else:
            if self.shared_workspace is None:
                raise ValueError("the block was made without max_shared")
            group_start, prefix_len, max_group = shared
            out = B.exl3_attention_shared(self.cache, q, step.q_start, step.seq_len, step.table, group_start, prefix_len,
                                          max_new=max_new, max_group=max_group, workspace=self.shared_workspace)
        out = self.proj["o"](out.view(tokens, -1))
        return out if self.norm is None else (x, out)


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
    ap.add_argument("--samples", type=int, default=1, help="rows that go on from each prompt")
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", default="32x8x128", help="query heads x key/value heads x head dimension")
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args(argv)
    heads, kv_heads, dim = map(int, a.heads.split("x"))
    dev = torch.device("cuda", torch.cuda.current_device())
    width = -(-(a.prompt + a.steps) // a.page)
    rows = a.requests * a.samples
    pages, most = rows * width, max(a.requests * a.prompt, rows)
    pool = PagePool(a.requests, pages, a.page, width, dev)
    rotary = B.exl3_rotary_freqs(dim, device=dev)
    blocks = [AttentionBlock(random_weights(a.hidden, heads, kv_heads, dim, 3, B.CB_3INST, 1000 * i, dev), heads, kv_heads, dim,
                             pages, a.page, most, dev, norm=(torch.ones(a.hidden, device=dev).half(), 1e-5), rotary=rotary,
                             max_shared=rows if a.samples > 1 else 0)
              for i in range(a.layers)]
    caches = B.Exl3KvCacheGroup([block.cache for block in blocks])

    def run(x, requests, new, shared=None):
        step = pool.step(torch.full((requests,), new, dtype=torch.int32, device=dev), requests * new)
        add = None
        for block in blocks:
            x, add = block(x, step, new, add, shared)
        return x + add

    events = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    x = torch.randn((a.requests * a.prompt, a.hidden), device=dev).half()
    events[0].record()
    x = run(x, a.requests, a.prompt).view(a.requests, a.prompt, -1)[:, -1]
    events[1].record()
    shared = None
    if a.samples > 1:
        parent = torch.arange(a.requests, dtype=torch.int32, device=dev).repeat_interleave(a.samples)
        pool.fork(parent, caches)
        shared = (torch.arange(0, rows + 1, a.samples, dtype=torch.int32, device=dev),
                  torch.full((a.requests,), a.prompt // a.page * a.page, dtype=torch.int32, device=dev), a.samples)
    x = x.repeat_interleave(a.samples, 0).contiguous()
    for _ in range(a.steps):
        x = run(x, rows, 1, shared)
    events[2].record()
    torch.cuda.synchronize()
    assert pool.ctx_len.tolist() == [a.prompt + a.steps] * rows and int(pool.state[2]) == 0
    print(f"{a.layers} blocks, {a.requests} requests: prompts of {a.prompt} tokens {events[0].elapsed_time(events[1]):.2f} ms, "
          f"then {events[1].elapsed_time(events[2]) / a.steps:.3f} ms a step of {rows} rows over {a.steps} steps")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
