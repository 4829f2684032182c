"""CPU definition (numpy, 64-bit) of the paged 8-bit cache and the attention over it.

Test infrastructure: shares nothing with the CUDA side.  Rounding decisions of
the cache (which int8 a value becomes) are taken on binary32 quotients, as the
interface defines them; everything else is float64.
"""
from __future__ import annotations

import math

import numpy as np

f32 = np.float32


def plan(ctx_len, new_len, tokens, page_size, free_pages, free_state, block_table):
    """One request after the other; returns dict of the outputs (copies)."""
    table, ring = np.array(block_table), np.array(free_pages)
    n, cap = len(ctx_len), len(ring)
    head, count = int(free_state[0]), int(free_state[1])
    asked = taken = lacking = 0
    seq, starts = np.zeros(n, np.int32), np.zeros(n + 1, np.int32)
    slot, position = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int32)
    at = 0
    pushed = []
    for b in range(n):
        c, k = int(ctx_len[b]), int(new_len[b])
        starts[b] = min(at, tokens)
        have = math.ceil(c / page_size)
        if k < 0:
            pushed += [int(table[b, j]) for j in range(have)]
            continue
        want = math.ceil((c + k) / page_size)
        seq[b] = c
        ok = want <= table.shape[1] and at + k <= tokens
        if ok:
            need = want - have
            if need == 0 or asked + need <= count:
                for j in range(need):
                    table[b, have + j] = ring[(head + asked + j) % cap]
                taken += need
                seq[b] = c + k
            else:
                lacking += need
                ok = False
            asked += need
        for i in range(k):
            if at + i < tokens:
                position[at + i] = c + i
                if ok:
                    slot[at + i] = int(table[b, (c + i) // page_size]) * page_size + (c + i) % page_size
        at += k
    starts[n] = min(at, tokens)
    for j, page in enumerate(pushed[:max(0, cap - count)]):
        ring[(head + count + j) % cap] = page
    state = [(head + taken) % cap if cap else 0, count - taken + min(len(pushed), cap - count), lacking]
    return dict(seq_len=seq, q_start=starts, slot=slot, position=position, free_state=np.array(state, np.int32),
                block_table=table, free_pages=ring)


def append(q, scale, x, slot):
    """New values x [tokens][heads][dim] (binary16) into the pages q [pages][heads]
    [page_size][dim] int8 with scale [pages][heads]; returns copies."""
    q, scale = np.array(q), np.array(scale, f32)
    size = q.shape[2]
    order = {}
    for t, s in enumerate(slot):
        if 0 <= s < q.shape[0] * size:
            order.setdefault(int(s) // size, []).append((int(s) % size, t))
    for page, items in order.items():
        first = items[0][0]
        for h in range(q.shape[1]):
            xs = np.stack([x[t, h] for _, t in items]).astype(f32)
            old = f32(scale[page, h]) if first > 0 else f32(0)
            if not np.isfinite(xs).all() or np.isnan(old):
                scale[page, h] = np.nan
                q[page, h, :first + len(items)] = 0
                continue
            new = max(old, f32(np.abs(xs).max()) / f32(127))
            if new != old:
                ratio = f32(old) / f32(new)
                q[page, h, :first] = np.rint(q[page, h, :first].astype(f32) * ratio).astype(np.int8)
            scale[page, h] = new
            for (off, _), row in zip(items, xs):
                q[page, h, off] = np.rint(row / new).astype(np.int8) if new > 0 else 0
    return q, scale


def gather(q, scale, table_row, length, head):
    """The first `length` tokens of a request, one head, as float64 [length][dim]."""
    size = q.shape[2]
    pages = [int(p) for p in table_row[:math.ceil(length / size)]]
    if not pages:
        return np.zeros((0, q.shape[3]))
    return np.concatenate([q[p, head].astype(np.float64) * float(scale[p, head]) for p in pages])[:length]


def attention(k, v, k_scale, v_scale, q, q_start, seq_len, block_table, scale):
    """(out, lse, spread): float64 [tokens][heads][dim], [tokens][heads], and the
    pieces of an error bound per row: `spread` sum_j p_j |v_j| and `size` the
    largest sum_d |scale q_d k_jd|."""
    tokens, heads, dim = q.shape
    group = heads // k.shape[1]
    out, spread = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads, dim))
    lse, size = np.full((tokens, heads), -np.inf), np.zeros((tokens, heads))
    for b in range(len(seq_len)):
        n = int(q_start[b + 1] - q_start[b])
        length = min(int(seq_len[b]), block_table.shape[1] * k.shape[2])
        for h in range(k.shape[1]):
            if length <= 0:
                continue
            kk = gather(k, k_scale, block_table[b], length, h)
            vv = gather(v, v_scale, block_table[b], length, h)
            for i in range(n):
                see = length - n + i + 1
                if see <= 0:
                    continue
                t = int(q_start[b]) + i
                for g in range(h * group, (h + 1) * group):
                    row = q[t, g].astype(np.float64)
                    s = scale * (kk[:see] @ row)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[t, g], spread[t, g] = p @ vv[:see], p @ np.abs(vv[:see])
                    lse[t, g] = s.max() + math.log(e.sum())
                    size[t, g] = (abs(scale) * (np.abs(kk[:see]) @ np.abs(row))).max()
    return out, lse, dict(spread=spread, size=size)
