"""Partial results of attention, none lost: every 32 keys of a request count.

All keys of a row have the same score (another one in every row), and the values of
the 32-key unit u are one number in column u mod D and 0 elsewhere.  A row that sees
n keys is then, in column d, that number times the share of the n keys in the units
of column d, and its log-sum is the score plus log n.  A unit is at least 6% of its
column for 68000 keys and D = 128, and 1 / 2125 of the sum.

The error allowed: the output to binary16 (2^-11 of it).  The score x is a binary32
number of up to 16 in magnitude, so x - m is off by at most 2^-20, the same for every
key: 2^-18 with the exponential.  The products' sums are whole numbers of less than
24 bits; the sum l has at most n / 32 additions of 2^-24 each behind one another and
64 more in the joins.  The log-sum: the same, and 2^-20 for the logarithms, 2^-22 of
itself.
"""
import numpy as np
import pytest

UNIT = 32
CASES = [  # heads, kv_heads, dim, requests' lengths, new tokens
    (8, 1, 128, [68000], [1]), (16, 1, 128, [68000], [1]), (5, 1, 64, [68000], [1]), (12, 1, 64, [68000], [1]),
    (40, 1, 128, [68000], [1]), (8, 2, 128, [17000], [1]), (16, 2, 64, [9000, 30, 5200], [1, 1, 1]),
    (24, 1, 128, [3000, 2999, 3, 1, 8000], [1, 2, 1, 1, 2]),
    (56, 1, 128, [68000], [1]), (100, 1, 64, [30000], [1]), (4, 1, 128, [2600], [30]), (8, 2, 64, [1200, 2, 3000], [40, 1, 65]),
    (7, 1, 64, [20000, 900], [60, 20]),
]


def value(b, head):
    return 127 - 40 * head - 13 * (b % 3)


def score(t, h):
    return ((7 * t + 3 * h) % 16) - 8.0    # as q holds it; times 1/2


def expected(heads, kv_heads, dim, seq, new, lost=None):
    """(out, lse) in 64 bits; `lost`: (request, unit) whose keys do not count."""
    tokens = sum(new)
    out, lse = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads))
    t = 0
    for b, (length, m) in enumerate(zip(seq, new)):
        key = np.arange(length)
        keep = np.ones(length, bool)
        if lost is not None and lost[0] == b:
            keep[lost[1] * UNIT:(lost[1] + 1) * UNIT] = False
        for i in range(m):
            mine = key[:length - m + i + 1][keep[:length - m + i + 1]]
            share = np.bincount(mine // UNIT % dim, minlength=dim) / len(mine)
            for h in range(heads):
                out[t, h] = share * value(b, h // (heads // kv_heads)) / 64
                lse[t, h] = score(t, h) / 2 + np.log(len(mine))
            t += 1
    return out, lse


def check(got, got_lse, case):
    out, lse = expected(*case)
    off = np.abs(np.asarray(got, np.float64) - out)
    steps = (max(case[3]) / UNIT + 64) * 2.0 ** -24
    allowed = np.abs(out) * (2.0 ** -11 + 2.0 ** -18 + steps) + 2.0 ** -25
    assert (off <= allowed).all(), f"{(off / allowed).max():.2f} times what is allowed"
    off = np.abs(np.asarray(got_lse, np.float64) - lse)
    allowed = 2.0 ** -18 + steps + 2.0 ** -20 + np.abs(lse) * 2.0 ** -22
    assert (off <= allowed).all(), f"lse: {(off / allowed).max():.2f} times what is allowed"


@pytest.mark.parametrize("case", CASES)
def test_a_lost_unit_is_seen(case):
    """The check itself: it passes what is expected, rounded, and fails wherever 32 keys are missing, in the values and in
    the log-sums alike."""
    out, lse = expected(*case)
    check(out.astype(np.float16), lse.astype(np.float32), case)
    for b, length in enumerate(case[3]):
        units = -(-length // UNIT)
        for u in sorted({0, 1, units // 3, units // 2, units - 2, units - 1} & set(range(1 if units == 1 else units))):
            if (u + 1) * UNIT >= length and u * UNIT <= length - case[4][b]:
                continue   # some row would see nothing else, or not this unit
            less, less_lse = expected(*case, lost=(b, u))
            with pytest.raises(AssertionError, match="^[0-9]"):
                check(less.astype(np.float16), lse, case)
            with pytest.raises(AssertionError, match="^lse"):
                check(out.astype(np.float16), less_lse, case)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", CASES)
def test_every_unit_counts(case, page):
    """Three times from one workspace, between calls of other lengths, so that no slot's old contents would do."""
    import torch

    from trellis_decode_gemv_gb300 import binding as B

    heads, kv_heads, dim, seq, new = case
    ws = B.alloc_attention_workspace(heads, kv_heads, dim, max(new), "cuda")
    for shift in (0, 37, 0):
        lens = [n + shift for n in seq]
        need = [-(-n // page) for n in lens]
        pages, tokens = sum(need), sum(new)
        order = np.random.default_rng(pages).permutation(pages)
        table = np.full((len(seq), max(need)), -1, np.int32)
        k, v = (np.zeros((pages, kv_heads, page, dim), np.int8) for _ in "kv")
        k[..., 0] = 1
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
            key = np.arange(n * page)
            for h in range(kv_heads):
                rows = np.zeros((n * page, dim), np.int8)
                rows[key, key // UNIT % dim] = value(b, h)
                v[table[b, :n], h] = rows.reshape(n, page, dim)
        q = np.zeros((tokens, heads, dim), np.float16)
        q[:, :, 0] = [[score(t, h) for h in range(heads)] for t in range(tokens)]
        one = np.ones((pages, kv_heads), np.float32)
        up = [torch.from_numpy(a).cuda() for a in (k, v, one, one / 64, q, np.concatenate([[0], np.cumsum(new)]).astype(np.int32),
                                                   np.array(lens, np.int32), table)]
        out, lse = B.exl3_attention(B.Exl3KvCache.from_tensors(*up[:4]), *up[4:], max_new=max(new), scale=0.5, lse=True, workspace=ws)
        check(out.cpu().numpy(), lse.cpu().numpy(), (heads, kv_heads, dim, lens, new))
