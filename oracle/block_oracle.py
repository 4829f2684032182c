"""CPU definition (numpy, 64-bit) of the operators around a decoder's quantized
projections: norms, rotary positions, forks of requests over the paged cache.

Test infrastructure: shares nothing with the CUDA side.
"""
from __future__ import annotations

import math

import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """(y, h) in float64, h before any rounding."""
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight.astype(np.float64), h


def hadamard():
    h = np.ones((1, 1))
    while len(h) < 128:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(128)


def rotate(y, signs):
    """Blocks of 128 of y after the signs and the transform (y itself without signs)."""
    if signs is None:
        return y
    return ((y * signs.astype(np.float64)).reshape(*y.shape[:-1], -1, 128) @ hadamard()).reshape(y.shape)


def frequencies(dim, base, scaling="none", scale=1.0, original=8192, low=1.0, high=4.0, fast=32.0, slow=1.0):
    """Radians a position of each pair, and the factor on cosine and sine."""
    if scaling == "ntk":
        base *= scale ** (dim / (dim - 2))
    out, factor = [], 1.0
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        if scaling == "linear":
            f /= scale
        if scaling == "llama3":
            wave = 2 * math.pi / f
            if wave > original / low:
                f /= scale
            elif wave >= original / high:
                mix = (original / wave - low) / (high - low)
                f = (1 - mix) * f / scale + mix * f
        if scaling == "yarn":
            first = max(math.floor(dim * math.log(original / (fast * 2 * math.pi)) / (2 * math.log(base))), 0)
            last = min(math.ceil(dim * math.log(original / (slow * 2 * math.pi)) / (2 * math.log(base))), dim - 1)
            ramp = min(max((i - first) / max(last - first, 1e-3), 0), 1)
            f = f / scale * ramp + f * (1 - ramp)
            factor = 0.1 * math.log(scale) + 1
        out.append(f)
    return np.array(out), factor


def rotary(x, position, radians, factor=1.0, interleaved=False):
    """x [tokens, heads, dim] in float64; tokens of negative position as they are."""
    y = x.astype(np.float64)
    half = len(radians)
    angle = np.asarray(position, np.float64)[:, None] * radians
    c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, w = y[..., a], y[..., b]
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    keep = np.asarray(position) < 0
    y[keep] = x[keep].astype(np.float64)
    return y


def fork(parent, ctx_len, page_size, pages, free_pages, free_state, block_table):
    """One row after the other; returns dict of the outputs (copies)."""
    table, ring = np.array(block_table), np.array(free_pages)
    requests, width = len(ctx_len), table.shape[1]
    cap = len(ring)
    head, count = (int(free_state[0]) % cap if cap else 0), min(max(int(free_state[1]), 0), cap)
    rows = len(parent)
    tokens = [min(max(int(c), 0), width * page_size) for c in ctx_len]
    new = np.full((rows, width), -1, np.int32)
    ctx = np.zeros(rows, np.int32)
    src, dst, part_of = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
    continued, taken, lacking = set(), 0, 0
    for i, b in enumerate(map(int, parent)):
        if not 0 <= b < requests:
            continue
        full, part = divmod(tokens[b], page_size)
        again = b in continued
        continued.add(b)
        if again and part:
            if taken == count:
                lacking += 1
                continue
            src[i], dst[i], part_of[i] = table[b, full], ring[(head + taken) % cap], part
            new[i, full] = dst[i]
            taken += 1
        elif part:
            new[i, full] = table[b, full]
        new[i, :full] = table[b, :full]
        ctx[i] = tokens[b]
    held = [set(int(p) for p in table[b, :-(-tokens[b] // page_size)]) for b in range(requests)]
    before = set().union(*[held[b] for b in range(requests) if b not in continued] or [set()])
    after = set().union(*[held[b] for b in continued] or [set()]) | {int(p) for p in dst}
    back = sorted(p for p in before - after if 0 <= p < pages)[:cap - count + taken]
    for j, p in enumerate(back):
        ring[(head + count + j) % cap] = p
    state = [(head + taken) % cap if cap else 0, count - taken + len(back), lacking]
    return dict(ctx_len=ctx, block_table=new, copy_from=src, copy_to=dst, copy_tokens=part_of,
                free_state=np.array(state, np.int32), free_pages=ring)


def copy(q, scale, src, dst, tokens):
    """Pages q [pages][heads][page_size][dim] and scale [pages][heads] after the copies."""
    q, scale = np.array(q), np.array(scale)
    was, was_scale = q.copy(), scale.copy()
    for a, b, n in zip(src, dst, tokens):
        if 0 <= a < len(q) and 0 <= b < len(q):
            n = min(max(int(n), 0), q.shape[2])
            q[b, :, :n] = was[a, :, :n]
            scale[b] = was_scale[a]
    return q, scale
