"""The operators of a decoder's block around its quantized projections and its paged 8-bit cache: what is timed, in plain torch and
through the library.

  norm    the residual's addition and the root-mean-square norm; binary16 out, or int8 with a scale for each 128 values, turned by the
          signs and Hadamard blocks of the projections that read it
  rotary  rotary positions on queries and keys, in the two layouts, on all or a part of a head, scaled for long contexts
  fork    rows of a block table from parent rows: full pages shared, the last one copied, pages that nobody continues given back
  copy    the pages that forks have to copy, in the caches of all layers
  share   attention of requests that share a long prefix, whose scores are computed for all of them at once

`own` chooses the side: false, the elementary torch operations below; true, the calls of this repository's package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's residual and norm before the projections of a layer of 4096: latency is all
        dict(name="norm_step", op="norm", rows=1, n=4096, residual=True, outs=0, rotate=False),
        # a chunk of prompt through the norm of a layer of 8192
        dict(name="norm_prompt", op="norm", rows=4095, n=8192, residual=True, outs=0, rotate=False),
        # a decoding batch before the q, k and v projections on int8 activations
        dict(name="norm_int8", op="norm", rows=16, n=4096, residual=True, outs=3, rotate=True),
        # a decoding step's queries and keys, slices of one projection's output, far positions
        dict(name="rotary_step", op="rotary", tokens=64, heads=32, kv_heads=8, dim=128, part=128, interleaved=False, scaling="llama3",
             scale=8.0, reach=131071),
        # a chunk of prompt: half of each head, neighbours as pairs
        dict(name="rotary_prompt", op="rotary", tokens=8191, heads=64, kv_heads=8, dim=128, part=64, interleaved=True, scaling="yarn",
             scale=4.0, reach=32767),
        # four samples of each of 16 prompts
        dict(name="fork_step", op="fork", requests=16, rows=64, ctx=2000, alive=16, page=16, lens=1),
        # a wide tick: many rows, a third of the requests go, the others are continued once or several times
        dict(name="fork_many", op="fork", requests=500, rows=509, ctx=8000, alive=333, page=64, lens=2),
        # the last pages of a few forks in the caches of a small model's layers
        dict(name="copy_few", op="copy", layers=24, pairs=7, kv_heads=2, dim=64, page=32, lens=3),
        # the last pages of 61 samples in 32 layers' caches of 8 heads of 128
        dict(name="copy_many", op="copy", layers=32, pairs=61, kv_heads=8, dim=128, page=64, lens=4),
        # eight samples of one prompt
        dict(name="share_samples", op="share", requests=8, groups=1, prefix=2011, ctx=300, new=1, heads=32, kv_heads=8, dim=128, page=16, lens=5),
        # a busy server's step: 64 requests behind one long document, one unused place of the batch among them
        dict(name="share_document", op="share", requests=64, groups=1, prefix=32000, ctx=1000, new=1, heads=32, kv_heads=8, dim=128, page=64, lens=6),
        # four drafted tokens of 40 requests behind five system prompts
        dict(name="share_draft", op="share", requests=40, groups=5, prefix=6000, ctx=700, new=4, heads=64, kv_heads=8, dim=128, page=32, lens=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rotary", "fork", "copy", "share", "share"])
    lens = rng.randrange(1 << 20)
    if op == "norm":
        outs = rng.choice([0, 0, 1, 2, 3])
        n = 128 * _log(rng, 1, 128) if outs else 8 * _log(rng, 4, 2048)
        return dict(op=op, rows=_log(rng, 1, min(8192, 30000000 // (n * max(outs, 1)))), n=n, residual=rng.random() < 0.7, outs=outs,
                    rotate=outs > 0 and rng.random() < 0.7)
    if op == "rotary":
        kv_heads, dim = rng.choice([1, 2, 3, 8]), rng.choice([64, 128])
        heads = kv_heads * rng.choice([1, 4, 5, 7, 8])
        scaling = rng.choice(["none", "linear", "ntk", "llama3", "yarn"])
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=heads, kv_heads=kv_heads, dim=dim, part=rng.choice([dim, dim, dim // 2, dim // 4]),
                    interleaved=rng.random() < 0.5, scaling=scaling, scale=1.0 if scaling == "none" else rng.choice([2.0, 3.5, 8.0, 32.0]),
                    reach=_log(rng, 100, 1000000))
    page = rng.choice([16, 32, 64, 128])
    if op == "fork":
        requests, rows = _log(rng, 1, 500), _log(rng, 1, 500)
        return dict(op=op, requests=requests, rows=rows, ctx=_log(rng, 1, 8000), alive=rng.randint(1, requests), page=page, lens=lens)
    kv_heads, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128])
    if op == "copy":
        return dict(op=op, layers=rng.randint(1, 40), pairs=_log(rng, 1, 60), kv_heads=kv_heads, dim=dim, page=page, lens=lens)
    requests, new = _log(rng, 2, 64), rng.choice([1, 1, 1, 2, 5])
    return dict(op=op, requests=requests, groups=rng.randint(1, min(requests, 6)), prefix=_log(rng, 100, 400000 // (requests * new)),
                ctx=_log(rng, 1, 1000), new=new, heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv_heads, dim=dim, page=page, lens=lens)


def _forks(case):
    """Tokens of each request and the parent of each row: parents among the first `alive` of a shuffled list, some rows without one;
    a third of the requests share their leading pages with the request before them."""
    r = random.Random(case["lens"])
    n = case["requests"]
    ctx = [r.randint(0, case["ctx"]) for _ in range(n)]
    ctx[0] = case["ctx"]
    order = list(range(n))
    r.shuffle(order)
    parent = [r.choice(order[:case["alive"]]) if r.random() < 0.95 else -1 for _ in range(case["rows"])]
    shared = [i > 0 and r.random() < 0.33 for i in range(n)]
    return ctx, parent, shared


def _groups(case):
    """First request of each group (and their number), each group's shared tokens, each request's own cached and new tokens."""
    r = random.Random(case["lens"])
    n, g = case["requests"], case["groups"]
    start = [0] + sorted(r.sample(range(1, n), g - 1)) + [n]
    prefix = [case["prefix"] if i == 0 else r.randint(case["prefix"] // 4, case["prefix"]) for i in range(g)]
    ctx = [case["ctx"] if i == 0 else r.randint(0, case["ctx"]) for i in range(n)]
    new = [case["new"] if i == 0 else r.randint((case["new"] + 1) // 2, case["new"]) for i in range(n)]
    empty = [i == n - 1 and n >= 4 and case["new"] == 1 for i in range(n)]  # an unused place of a padded batch: one query, no keys at all
    return start, prefix, ctx, new, empty


def _copies(case):
    r = random.Random(case["lens"])
    return [r.randint(1, case["page"]) for _ in range(case["pairs"])]


def _frequencies(part, scaling, scale, base=500000.0, original=8192):
    """Radians a position of each pair, in 64 bits, and the factor on cosine and sine."""
    i = torch.arange(part // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * scale ** (part / (part - 2))
    f = base ** (-2 * i / part)
    factor = 1.0
    if scaling == "linear":
        f = f / scale
    elif scaling == "llama3":
        turns = original * f / (2 * math.pi)  # within the original context
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f / scale * (1 - keep) + f * keep
    elif scaling == "yarn":
        def pair(turns):
            return part * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), part - 1)
        drop = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / scale * drop + f * (1 - drop)
        factor = 0.1 * math.log(scale) + 1.0
    return f, factor


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(DEV)


def _hadamard(dtype):
    h = torch.ones((1, 1), dtype=dtype, device=DEV)
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(128)


def _bytes8(shape, g):
    x = torch.empty(shape, dtype=torch.int8, device=DEV)
    for part in x.split(max(1, (1 << 27) // (x[0].numel() or 1))):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(36).round_().clamp_(-127, 127))
    return x


def _scales(shape, g):
    return torch.exp(0.3 * torch.randn(shape, generator=g, device=DEV)) * 0.03


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    s = dict(case=case)
    op = case["op"]
    if op == "norm":
        rows, n = case["rows"], case["n"]
        # a residual stream some of whose channels are large, as trained ones are
        s |= dict(x=(randn(rows, n) * 0.7).half(), weight=(1 + 0.2 * randn(n)).half(), eps=EPS,
                  residual=(randn(rows, n) * torch.exp(0.5 * randn(n))).half() if case["residual"] else None)
        s["signs"] = [torch.where(randn(n) < 0, -1.0, 1.0).half() if case["rotate"] else None for _ in range(case["outs"])]
        s["hadamard"] = _hadamard(torch.float32)
        return s
    if op == "rotary":
        t, heads, kvh, dim = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        qkv = randn(t, (heads + 2 * kvh) * dim).half()
        q, k, _ = qkv.split([heads * dim, kvh * dim, kvh * dim], 1)
        f, factor = _frequencies(case["part"], case["scaling"], case["scale"])
        s |= dict(q=q.view(t, heads, dim), k=k.view(t, kvh, dim), freqs=f.to(DEV), factor=factor,
                  position=torch.randint(0, case["reach"] + 1, (t,), generator=g, device=DEV, dtype=torch.int32))
        if own:  # what a server keeps: the frequencies as the library takes them
            from trellis_decode_gemv_gb300 import binding as B
            s["plan"] = B.exl3_rotary_freqs(case["part"], base=500000.0, scaling=case["scaling"], scale=case["scale"],
                                            original=8192, device=DEV)
        return s
    page = case["page"]
    if op == "fork":
        ctx, parent, shared = _forks(case)
        n = case["requests"]
        need = [-(-c // page) for c in ctx]
        width = max(max(need), 1)
        pages = sum(need) + case["rows"] + 5
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((n, width), -1, dtype=torch.int32)
        at = 0
        for i, k in enumerate(need):
            same = min(ctx[i] // page, ctx[i - 1] // page) if shared[i] else 0
            table[i, :same] = table[i - 1, :same]
            table[i, same:k] = order[at:at + k - same]
            at += k - same
        count = pages - at
        free = torch.full((pages,), -1, dtype=torch.int32)
        head = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
        free[(head + torch.arange(count)) % pages] = order[at:]
        s |= dict(page=page, pages=pages, ctx_len=_ints(ctx), parent=_ints(parent), table=table.to(DEV), free_pages=free.to(DEV),
                  free_state=_ints([head, count]))
        if own:
            from trellis_decode_gemv_gb300 import binding as B
            s["workspace"] = B.alloc_kv_fork_workspace(pages, DEV)
        return s
    kvh, dim = case["kv_heads"], case["dim"]
    if op == "copy":
        tokens, layers = _copies(case), case["layers"]
        pages = 4 * len(tokens) + 4
        order = torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32)  # the last page belongs to nobody
        pairs = len(tokens)
        s |= dict(k=list(_bytes8((layers * pages, kvh, page, dim), g).split(pages)), v=list(_bytes8((layers * pages, kvh, page, dim), g).split(pages)),
                  k_scale=list(_scales((layers * pages, kvh), g).split(pages)), v_scale=list(_scales((layers * pages, kvh), g).split(pages)),
                  tokens=_ints(tokens), copy_from=order[:pairs].clone(), copy_to=order[pairs:2 * pairs].clone())
        if pairs >= 4:  # a row that needs no copy
            s["copy_from"][1] = -1
            s["copy_to"][1] = -1
        if own:
            from trellis_decode_gemv_gb300 import binding as B
            s["caches"] = B.Exl3KvCacheGroup([B.Exl3KvCache.from_tensors(*c) for c in zip(s["k"], s["v"], s["k_scale"], s["v_scale"])])
        return s
    start, prefix, ctx, new, empty = _groups(case)
    n = case["requests"]
    of = [max(i for i in range(len(prefix)) if start[i] <= b) for b in range(n)]
    seq = [0 if empty[b] else prefix[of[b]] + ctx[b] + new[b] for b in range(n)]
    full = [p // page for p in prefix]
    need = [0 if empty[b] else -(-seq[b] // page) - full[of[b]] for b in range(n)]
    pages = sum(full) + sum(need) + 3
    order = torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((n, max(full[of[b]] + need[b] for b in range(n))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(full):
        for b in range(start[i], start[i + 1]):
            if not empty[b]:
                table[b, :k] = order[at:at + k]
        at += k
    for b in range(n):
        table[b, full[of[b]]:full[of[b]] + need[b]] = order[at:at + need[b]]
        at += need[b]
    q_start = [sum(new[:b]) for b in range(n + 1)]
    shape = (pages, kvh, page, dim)
    s |= dict(page=page, k_cache=_bytes8(shape, g), v_cache=_bytes8(shape, g), k_scale=_scales(shape[:2], g), v_scale=_scales(shape[:2], g),
              q=(2 * randn(q_start[-1], case["heads"], dim)).half(), table=table.to(DEV), seq_len=_ints(seq), q_start=_ints(q_start),
              group_start=_ints(start), prefix_len=_ints(prefix), of=_ints(of, torch.int64), most_new=max(new),
              most_group=max(q_start[start[i + 1]] - q_start[start[i]] for i in range(len(prefix))),
              most_prefix=max(prefix), most_own=max(max(c + k for c, k in zip(ctx, new)), 1), scale=dim ** -0.5)
    # where a request's own part begins inside a page, that page holds the last tokens of the prefix: the same values for the whole group
    for i in range(len(prefix)):
        part, k = prefix[i] % page, full[i]
        rows = [b for b in range(start[i], start[i + 1]) if not empty[b]]
        if part and rows:
            at = table[rows, k].long().to(DEV)
            for name in ("k", "v"):
                cache = s[name + "_cache"]
                cache[at, :, :part] = cache[at[0], :, :part].clone()
                s[name + "_scale"][at] = s[name + "_scale"][at[0]].clone()
    if own:
        from trellis_decode_gemv_gb300 import binding as B
        s["cache"] = B.Exl3KvCache.from_tensors(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["workspace"] = B.alloc_attention_shared_workspace(case["heads"], kvh, dim, s["most_new"], s["most_group"], q_start[-1], DEV)
    return s


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from trellis_decode_gemv_gb300 import binding as B
        if op == "norm":
            if case["outs"]:
                q, scale, h = B.exl3_rms_norm_i8(s["x"], s["weight"], s["eps"], s["signs"], residual=s["residual"])
                got = dict(q=_values(q, scale), scale=scale)
            else:
                y, h = B.exl3_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"])
                got = dict(y=y)
            return got | dict(h=h) if case["residual"] else got
        if op == "rotary":
            q, k = B.exl3_rotary(s["q"], s["k"], s["position"], s["plan"], interleaved=case["interleaved"])
            return dict(q=q, k=k)
        if op == "fork":
            f = B.exl3_kv_fork(s["parent"], s["ctx_len"], s["page"], s["pages"], s["free_pages"], s["free_state"], s["table"],
                               workspace=s["workspace"])
            return dict(ctx_len=f.ctx_len, table=f.block_table, copy_from=f.copy_from, copy_to=f.copy_to, copy_tokens=f.copy_tokens,
                        free_state=f.free_state, free_pages=s["free_pages"])
        if op == "copy":
            B.exl3_kv_copy(s["caches"], s["copy_from"], s["copy_to"], s["tokens"])
            return _copied(s)
        out, lse = B.exl3_attention_shared(s["cache"], s["q"], s["q_start"], s["seq_len"], s["table"], s["group_start"], s["prefix_len"],
                                           max_new=s["most_new"], max_group=s["most_group"], scale=s["scale"], lse=True,
                                           workspace=s["workspace"])
        return dict(out=out, lse=lse)
    return dict(norm=_norm, rotary=_rotary, fork=_fork, copy=_copy, share=_share)[op](s)


# ---------------------------------------------------------------- plain forms

def _values(q, scale):
    """What int8 [outs, rows, n] and its scales [outs, rows, n / 128] stand for."""
    values = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    torch.mul(q.view(*scale.shape, 128), scale[..., None], out=values.view(*scale.shape, 128))
    return values


def _norm(s):
    h = s["x"].float()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        got["h"] = h.half()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if not s["signs"]:
        return dict(y=y.half(), **got)
    outs = len(s["signs"])
    if s["case"]["rotate"]:
        z = (y * torch.stack(s["signs"]).float()[:, None]).view(outs, len(y), -1, 128) @ s["hadamard"]
    else:
        z = y.expand(outs, -1, -1).reshape(outs, len(y), -1, 128)
    scale = z.abs().amax(-1) / 127.0
    q = torch.round(z / torch.where(scale > 0, scale, 1.0)[..., None]).to(torch.int8)
    return dict(q=_values(q.view(outs, *y.shape), scale), scale=scale, **got)


def _rotary(s):
    case = s["case"]
    part, half = case["part"], case["part"] // 2
    angle = s["position"].double()[:, None] * s["freqs"]  # far positions want 64 bits
    cos, sin = ((t(angle) * s["factor"]).float()[:, None, :] for t in (torch.cos, torch.sin))

    def turn(x):
        y = x.clone()
        a, b = (x[..., 0:part:2], x[..., 1:part:2]) if case["interleaved"] else (x[..., :half], x[..., half:part])
        a, b = a.float(), b.float()
        u, w = (a * cos - b * sin).half(), (b * cos + a * sin).half()
        y[..., :part] = torch.stack([u, w], -1).flatten(-2) if case["interleaved"] else torch.cat([u, w], -1)
        return y

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _fork(s):
    """Row i continues request parent[i]: the full pages are shared; a partly filled one stays with the first row of a parent, each further
    row takes a page from the ring's head and a copy; pages that no row holds any more go to the ring's end in ascending order."""
    page, pages, table, ring = s["page"], s["pages"], s["table"], s["free_pages"]
    n, width = table.shape
    parent = s["parent"].long()
    rows, capacity = parent.numel(), ring.numel()
    head, count = s["free_state"].long()
    live = (parent >= 0) & (parent < n)
    p = torch.where(live, parent, n)
    i = torch.arange(rows, device=DEV)
    first = torch.full((n + 1,), rows, device=DEV).scatter_reduce(0, p, i, "amin")
    ctx = s["ctx_len"].long().clamp(0, width * page)
    c = torch.where(live, ctx[p.clamp(max=n - 1)], 0)
    full, part = c // page, c % page
    need = live & (part > 0) & (first[p] != i)
    before = torch.cumsum(need, 0) - need.long()
    got = ~need | (before < count)
    fresh = ring[(head + before) % capacity]
    j = torch.arange(width, device=DEV)
    old = table[p.clamp(max=n - 1)]
    last = torch.where(need, fresh, old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0])
    keep = (live & got)[:, None]
    out = torch.where(keep & (j < full[:, None]), old, -1)
    out = torch.where(keep & (j == full[:, None]) & (part > 0)[:, None], last[:, None], out)
    copies = need & got
    # pages held before and not after
    held = (j < ((ctx + page - 1) // page)[:, None]) & (table >= 0) & (table < pages)
    was = torch.zeros(pages + 1, dtype=torch.bool, device=DEV)
    was[torch.where(held, table, pages).reshape(-1).long()] = True
    now = torch.zeros(pages + 1, dtype=torch.bool, device=DEV)
    now[torch.where((out >= 0) & (out < pages), out, pages).reshape(-1).long()] = True
    back = (was & ~now)[:pages]
    place = torch.where(back, (head + count + torch.cumsum(back, 0) - 1) % capacity, capacity)
    flat = torch.cat([ring, ring.new_zeros(1)])
    flat[place] = torch.arange(pages, dtype=torch.int32, device=DEV)
    ring.copy_(flat[:-1])
    taken = copies.sum()
    state = torch.stack([(head + taken) % capacity, count - taken + back.sum(), need.sum() - taken]).to(torch.int32)
    at = old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    return dict(ctx_len=torch.where(got, c, 0).to(torch.int32), table=out, copy_from=torch.where(copies, at, -1),
                copy_to=torch.where(copies, fresh, -1), copy_tokens=torch.where(copies, part, 0).to(torch.int32), free_state=state, free_pages=ring)


def _copied(s):
    """The pages that were written, in all layers (pages of no pair stay as they are)."""
    return dict(k=s["k"][0]._base, v=s["v"][0]._base, k_scale=s["k_scale"][0]._base, v_scale=s["v_scale"][0]._base)


def _copy(s):
    to, layers, pages = s["copy_to"].long(), s["case"]["layers"], s["k"][0].shape[0]
    live = (s["copy_from"] >= 0) & (to >= 0)
    at = torch.arange(layers, device=DEV)[:, None] * pages
    # a pair of nothing copies the last page onto itself
    src, dst = ((torch.where(live, x.long(), pages - 1) + at).view(-1) for x in (s["copy_from"], to))
    keep = torch.arange(s["case"]["page"], device=DEV) < s["tokens"][:, None]
    keep = (keep & live[:, None]).repeat(layers, 1)[:, None, :, None]
    got = _copied(s)
    for name in ("k", "v"):
        cache, scale = got[name], got[name + "_scale"]
        cache[dst] = torch.where(keep, cache[src], cache[dst])
        scale[dst] = scale[src]
    return got


def _share(s):
    """Scores of a group's rows with the shared keys as one product, those with a request's own keys apart, one softmax over both;
    a row that sees no key is 0, and its log-sum -inf."""
    case, page, q = s["case"], s["page"], s["q"].float()
    tokens, heads, dim = q.shape
    kvh, n, groups = case["kv_heads"], case["requests"], case["groups"]
    group = heads // kvh
    q_start, seq, start, prefix, of = s["q_start"].long(), s["seq_len"].long(), s["group_start"].long(), s["prefix_len"].long(), s["of"]
    new = q_start[1:] - q_start[:-1]

    def keys(name, pages, held):
        x = s[name + "_cache"][pages].float() * s[name + "_scale"][pages][:, :, :, None, None]  # [n, blocks, kvh, page, dim]
        return torch.where(held[:, None, :, None], x.transpose(1, 2).reshape(len(pages), kvh, -1, dim), 0.0)

    # the prefixes: rows of a group beside one another
    shared = s["table"][start[:-1], :-(-s["most_prefix"] // page)].long().clamp(min=0)
    j = torch.arange(shared.shape[1] * page, device=DEV)
    held = j < prefix[:, None]
    first = q_start[start]
    i = torch.arange(s["most_group"], device=DEV)
    at = (first[:-1, None] + i).clamp(max=tokens - 1)
    rows = q[at].view(groups, -1, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(groups, kvh, -1, dim)
    score = (rows @ keys("k", shared, held).transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~held[:, None, None], -math.inf)
    top_a = score.amax(-1)
    p = score.sub_(torch.where(top_a == -math.inf, 0.0, top_a)[..., None]).exp_()
    sum_a, out_a = p.sum(-1), p @ keys("v", shared, held)
    t = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(q_start[1:], t, right=True)
    sees = seq[b] > 0
    g = of[b]

    def by_token(x, where, row, depth):  # [where, kvh, group * depth, ...] -> [tokens, heads, ...]
        x = x.view(x.shape[0], kvh, group, depth, *x.shape[3:])[where, :, :, row]
        return x.reshape(tokens, heads, *x.shape[3:])

    parts = [by_token(x, g, t - first[g], len(i)) for x in (top_a, sum_a, out_a)]
    # each request's own keys
    block = prefix[of] // page
    j = torch.arange((s["most_own"] + 2 * page - 1) // page, device=DEV)
    pages = s["table"].gather(1, (block[:, None] + j).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    j = block[:, None] * page + torch.arange(pages.shape[1] * page, device=DEV)
    held = (j >= prefix[of][:, None]) & (j < seq[:, None])
    i = torch.arange(s["most_new"], device=DEV)
    at = (q_start[:-1, None] + i).clamp(max=tokens - 1)
    rows = q[at].view(n, -1, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kvh, -1, dim)
    seen = held[:, None, :] & (j[:, None, :] <= (seq - new)[:, None, None] + i[:, None])
    score = (rows @ keys("k", pages, held).transpose(-1, -2)).view(n, kvh, group, len(i), -1)
    score = score.mul_(s["scale"]).masked_fill_(~seen[:, None, None], -math.inf).view(n, kvh, group * len(i), -1)
    top_b = score.amax(-1)
    p = score.sub_(torch.where(top_b == -math.inf, 0.0, top_b)[..., None]).exp_()
    sum_b, out_b = p.sum(-1), p @ keys("v", pages, held)
    own_parts = [by_token(x, b, t - q_start[b], len(i)) for x in (top_b, sum_b, out_b)]
    # one softmax over both
    ta = torch.where(sees[:, None], parts[0], -math.inf)
    tb = own_parts[0]
    top = torch.maximum(ta, tb)
    base = torch.where(top == -math.inf, 0.0, top)
    fa, fb = torch.exp(ta - base), torch.exp(tb - base)
    total = parts[1] * fa + own_parts[1] * fb
    out = (parts[2] * fa[..., None] + own_parts[2] * fb[..., None]) / torch.where(total > 0, total, 1.0)[..., None]
    return dict(out=out.half(), lse=base + torch.log(total))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "norm":
        rows, n = case["rows"], case["n"]
        outs = case["outs"]
        out = outs * (n + n // 32) if outs else 2 * n
        return dict(bytes=rows * (2 * n + (4 * n if case["residual"] else 0) + out) + 2 * n * (1 + (outs if case["rotate"] else 0)),
                    flops=rows * n * (5 + outs * (9 if case["rotate"] else 2)))
    if op == "rotary":
        t, heads = case["tokens"], case["heads"] + case["kv_heads"]
        return dict(bytes=4 * t * heads * case["dim"] + 4 * t + 4 * case["part"], flops=3 * t * heads * case["part"])
    if op == "fork":
        ctx, parent, _ = _forks(case)
        page = case["page"]
        held = sum(-(-ctx[p] // page) for p in parent if p >= 0)
        old = sum(-(-ctx[p] // page) for p in set(parent) if p >= 0)
        width = max(-(-case["ctx"] // page), 1)
        gone = sum(-(-c // page) for b, c in enumerate(ctx) if b not in set(parent))
        return dict(bytes=4 * (old + case["rows"] * width + 2 * gone + 5 * case["rows"] + case["requests"]), flops=held)
    kvh, dim = case["kv_heads"], case["dim"]
    if op == "copy":
        tokens = [t for i, t in enumerate(_copies(case)) if case["pairs"] < 4 or i != 1]
        return dict(bytes=case["layers"] * (2 * 2 * sum(tokens) * kvh * dim + 16 * len(tokens) * kvh) + 12 * case["pairs"], flops=0)
    start, prefix, ctx, new, empty = _groups(case)
    heads, page = case["heads"], case["page"]
    keys = pairs = blocks = 0
    for g, p in enumerate(prefix):
        keys += p
        blocks += -(-p // page)
        for b in range(start[g], start[g + 1]):
            if not empty[b]:
                keys += ctx[b] + new[b]
                blocks += -(-(ctx[b] + new[b]) // page)
                pairs += new[b] * (p + ctx[b]) + new[b] * (new[b] + 1) // 2
    t = sum(new)
    return dict(bytes=2 * keys * kvh * dim + 8 * blocks * kvh + 4 * blocks + 4 * t * heads * dim + 4 * t * heads + 8 * case["requests"] + 8 * len(prefix),
                flops=4 * pairs * heads * dim)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("fork", "copy"):
        return None  # whole numbers, and scales that are moved as they are
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"].double()
        got = {}
        if s["residual"] is not None:
            h += s["residual"].double()
            got["h"] = h.clone()
        h /= torch.sqrt(h.square().sum(-1, keepdim=True) / case["n"] + s["eps"])
        h *= s["weight"].double()
        if not s["signs"]:
            return dict(y=h, **got)
        q, scales = [], []
        for sign in s["signs"]:
            z = h if sign is None else h * sign.double()
            z = z.reshape(-1, 128)
            if sign is not None:
                for k in range(7):  # the butterflies of the transform, one bit of the index after the other
                    a = z.view(-1, 128 >> (k + 1), 2, 1 << k)
                    z = torch.stack([a[:, :, 0] + a[:, :, 1], a[:, :, 0] - a[:, :, 1]], 2).reshape(-1, 128)
                z = z / math.sqrt(128)
            step = z.abs().amax(-1, keepdim=True) / 127
            q.append((torch.round(z / torch.where(step > 0, step, 1.0)) * step).view(h.shape))
            scales.append(step.view(h.shape[0], -1))
        return dict(q=torch.stack(q), scale=torch.stack(scales), **got)
    if op == "rotary":
        part = case["part"]
        pairs = torch.arange(part // 2, device=DEV)
        ia, ib = (2 * pairs, 2 * pairs + 1) if case["interleaved"] else (pairs, pairs + part // 2)
        turned = torch.polar(torch.full_like(s["freqs"], s["factor"])[None].expand(case["tokens"], -1).contiguous(), s["position"].double()[:, None] * s["freqs"])
        got = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            z = torch.complex(x[..., ia], x[..., ib]) * turned[:, None]
            x[..., ia], x[..., ib] = z.real, z.imag
            got[name] = x
        return got
    start, prefix, ctx, new, empty = _groups(case)
    page, kvh, heads, dim = case["page"], case["kv_heads"], case["heads"], case["dim"]
    group, q = heads // kvh, s["q"].double()
    out, lse = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for b, k in enumerate(new):
        n = 0 if empty[b] else prefix[max(g for g in range(len(prefix)) if start[g] <= b)] + ctx[b] + k
        if n:
            at = s["table"][b, :-(-n // page)].long()
            kk, vv = ((s[x + "_cache"][at].double() * s[x + "_scale"][at].double()[:, :, None, None]).transpose(0, 1).reshape(kvh, -1, dim)[:, :n] for x in "kv")
            z = torch.einsum("tkgd,kjd->kgtj", q[t:t + k].view(k, kvh, group, dim), kk) * dim ** -0.5
            late = torch.arange(n, device=DEV)[None, :] > torch.arange(n - k, n, device=DEV)[:, None]
            z.masked_fill_(late, -math.inf)
            lse[t:t + k] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(k, heads)
            out[t:t + k] = torch.einsum("kgtj,kjd->tkgd", torch.softmax(z, -1), vv).reshape(k, heads, dim)
        t += k
    return dict(out=out, lse=lse)
