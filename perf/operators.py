"""The serving operators around a paged key/value cache held in 8 bits: what is timed, in plain torch and through the library.

  plan    block tables and slot maps on the GPU, from the requests' lengths and a ring of free pages
  append  new keys and values into the cache: int8 with one binary32 scale for each page and head
  attend  attention of each request's newest tokens over its cached keys and values (grouped heads, causal)

`own` chooses the side: false, the elementary torch operations below; true, the calls of this repository's package.
A cache is k, v int8 [pages, kv_heads, page_size, head_dim] and k_scale, v_scale float32 [pages, kv_heads].
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the bookkeeping of one decoding step: 64 running requests, one new token each
        dict(name="plan_step", op="plan", requests=64, ctx=8192, new=1, chunks=0, done=0, page=64, lens=1),
        # a full scheduler tick: several hundred requests, many with a chunk of prompt, some finished
        dict(name="plan_mixed", op="plan", requests=509, ctx=4096, new=511, chunks=250, done=31, page=16, lens=2),
        # one token for each of 64 requests (8 heads of 128, as Llama-3-8B and 70B), most into pages that are partly filled
        dict(name="append_step", op="append", requests=64, ctx=4096, new=1, chunks=0, kv_heads=8, dim=128, page=64, lens=3),
        # prompts of odd lengths of several requests, and a few single tokens beside them
        dict(name="append_prompts", op="append", requests=11, ctx=700, new=4093, chunks=7, kv_heads=8, dim=128, page=32, lens=4),
        # one request, a short context: a single user's token, where latency is all
        dict(name="attend_single", op="attend", requests=1, ctx=517, new=1, chunks=0, heads=32, kv_heads=8, dim=128, page=16, lens=5),
        # a busy server's step: 64 requests of very different lengths, one unused place of the batch among them
        dict(name="attend_batch", op="attend", requests=64, ctx=8192, new=1, chunks=0, heads=32, kv_heads=8, dim=128, page=64, lens=6),
        # one request with a very long document (Llama-3-70B's heads)
        dict(name="attend_long", op="attend", requests=1, ctx=131070, new=1, chunks=0, heads=64, kv_heads=8, dim=128, page=128, lens=7),
        # checking four drafted tokens of 16 requests at once
        dict(name="attend_draft", op="attend", requests=16, ctx=4000, new=4, chunks=16, heads=64, kv_heads=8, dim=128, page=64, lens=8),
        # a small model with heads of 64 in groups of seven, odd lengths
        dict(name="attend_small", op="attend", requests=33, ctx=2011, new=1, chunks=0, heads=14, kv_heads=2, dim=64, page=32, lens=9),
        # chunked prefill: two chunks of prompt over long contexts beside single tokens of other requests
        dict(name="attend_chunk", op="attend", requests=13, ctx=8111, new=500, chunks=2, heads=32, kv_heads=8, dim=128, page=64, lens=10),
        # a chunk of a draft model's prompt: heads of 64
        dict(name="attend_chunk64", op="attend", requests=3, ctx=1000, new=1023, chunks=3, heads=14, kv_heads=2, dim=64, page=16, lens=11),
        # a whole prompt in one call
        dict(name="attend_prompt", op="attend", requests=1, ctx=0, new=8192, chunks=1, heads=32, kv_heads=8, dim=128, page=128, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "attend"])
    page, lens = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20)
    if op == "plan":
        requests = _log(rng, 1, 500)
        return dict(op=op, requests=requests, ctx=_log(rng, 16, 8192), new=_log(rng, 1, 500), chunks=rng.randint(0, requests // 2),
                    done=rng.randint(0, requests // 8), page=page, lens=lens)
    dim, kv_heads = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        requests = _log(rng, 1, 64)
        chunks = rng.randint(0, min(requests, 7))
        return dict(op=op, requests=requests, ctx=_log(rng, 1, 2048), new=_log(rng, 1, 4000) if chunks else 1, chunks=chunks,
                    kv_heads=kv_heads, dim=dim, page=page, lens=lens)
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    kind = rng.choice(["step", "step", "draft", "chunk", "prompt"])
    if kind == "step":
        requests = _log(rng, 1, 64)
        ctx, new, chunks = _log(rng, 1, min(131000, 500000 // requests)), 1, 0
    elif kind == "draft":
        requests = _log(rng, 1, 32)
        ctx, new, chunks = _log(rng, 16, 8192), rng.randint(2, 8), requests
    elif kind == "chunk":
        requests = _log(rng, 1, 6)
        ctx, new, chunks = _log(rng, 64, 8192), _log(rng, 16, 512), rng.randint(1, min(2, requests))
    else:
        requests, ctx, new, chunks = 1, 0, _log(rng, 16, 8000), 1
        heads = min(heads, 32 // kv_heads * kv_heads)
    return dict(op=op, requests=requests, ctx=ctx, new=new, chunks=chunks, heads=heads, kv_heads=kv_heads, dim=dim, page=page, lens=lens)


def _lengths(case):
    """Cached and new tokens of each request: the first `chunks` bring `new` tokens or somewhat fewer, the others one;
    contexts from the longest down to nothing. -1 new tokens: the request is done."""
    r = random.Random(case["lens"])
    n, chunks = case["requests"], case["chunks"]
    ctx = [case["ctx"] if i == 0 else r.randint(0, case["ctx"]) for i in range(n)]
    new = [(case["new"] if i == 0 else r.randint((case["new"] + 1) // 2, case["new"])) if i < chunks else 1 for i in range(n)]
    if case["op"] == "attend" and n >= 4 and case["new"] == 1:
        ctx[-1] = -1  # an unused place of a padded batch: one query, no keys at all
    for i in r.sample(range(n), case.get("done", 0)):
        new[i] = -1
    return ctx, new


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(DEV)


def _starts(counts):
    return [0] + np.cumsum(counts).tolist()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ctx, new = _lengths(case)
    page = case["page"]
    n = len(ctx)
    s = dict(case=case, page=page)
    if case["op"] == "plan":
        have = [-(-c // page) for c in ctx]
        want = [-(-(c + max(k, 0)) // page) for c, k in zip(ctx, new)]
        width = max(max(want), 1)
        total = sum(want) + 64
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((n, width), -1, dtype=torch.int32)
        at = 0
        for i, h in enumerate(have):
            table[i, :h] = order[at:at + h]
            at += h
        free = torch.full((total,), -1, dtype=torch.int32)
        head = int(torch.randint(0, total, (1,), generator=g, device=DEV))
        count = total - at
        free[(head + torch.arange(count)) % total] = order[at:]
        s |= dict(ctx_len=_ints(ctx), new_len=_ints(new), table=table.to(DEV), free_pages=free.to(DEV), free_state=_ints([head, count]),
                  tokens=sum(max(k, 0) for k in new))
        return s
    dim, kvh = case["dim"], case["kv_heads"]
    seq = [c + k for c, k in zip(ctx, new)]
    need = [-(-q // page) for q in seq]
    pages, width = sum(need) + 3, max(max(need), 1)
    order = torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32).cpu()  # the last page belongs to nobody
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    for i, h in enumerate(need):
        table[i, :h] = order[at:at + h]
        at += h
    shape = (pages, kvh, page, dim)

    def bytes8():
        x = torch.empty(shape, dtype=torch.int8, device=DEV)
        for part in x.split(max(1, (1 << 27) // (kvh * page * dim))):
            part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(36).round_().clamp_(-127, 127))
        return x

    def scales():
        return torch.exp(0.3 * torch.randn((pages, kvh), generator=g, device=DEV)) * 0.03

    s |= dict(k_cache=bytes8(), v_cache=bytes8(), k_scale=scales(), v_scale=scales())
    if case["op"] == "append":
        t = sum(new)
        slot = [int(table[i, (c + j) // page]) * page + (c + j) % page for i, (c, k) in enumerate(zip(ctx, new)) for j in range(k)]
        # the heads of a step's projections, of slightly different size from token to token, so that some pages' scales grow
        size = torch.exp(0.3 * torch.randn((t, 1, 1), generator=g, device=DEV))
        s |= dict(k=(torch.randn((t, kvh, dim), generator=g, device=DEV) * size).half(),
                  v=(torch.randn((t, kvh, dim), generator=g, device=DEV) * size).half(), slot=_ints(slot, torch.int64),
                  most_pages=min(t, t // page + 2 * n))
    else:
        t = sum(new)
        s |= dict(q=(2 * torch.randn((t, case["heads"], dim), generator=g, device=DEV)).half(), table=table.to(DEV), seq_len=_ints(seq),
                  q_start=_ints(_starts(new)), most_new=max(new), most_seq=max(max(seq), 1), scale=dim ** -0.5)
    if own:  # what a server keeps from step to step: the cache object, and the attention's workspace
        from trellis_decode_gemv_gb300 import binding as B
        s["cache"] = B.Exl3KvCache.from_tensors(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if case["op"] == "attend":
            s["workspace"] = B.alloc_attention_workspace(case["heads"], kvh, dim, s["most_new"], DEV)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        from trellis_decode_gemv_gb300 import binding as B
        if op == "plan":
            seq_len, q_start, slot, position, state = B.exl3_kv_plan(s["ctx_len"], s["new_len"], s["tokens"], s["page"], s["free_pages"],
                                                                     s["free_state"], s["table"])
            return dict(seq_len=seq_len, q_start=q_start, slot=slot, position=position, free_state=state, table=s["table"], free_pages=s["free_pages"])
        if op == "append":
            B.exl3_kv_append(s["cache"], s["k"], s["v"], s["slot"])
            return dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        out, lse = B.exl3_attention(s["cache"], s["q"], s["q_start"], s["seq_len"], s["table"], max_new=s["most_new"], scale=s["scale"],
                                    lse=True, workspace=s["workspace"])
        return dict(out=out, lse=lse)
    if op == "plan":
        return _plan(s)
    if op == "append":
        # int8 is a whole number in a page whose scale stands beside it: both are returned as they are held
        _append(s["k"], s["slot"], s["k_cache"], s["k_scale"], s["most_pages"])
        _append(s["v"], s["slot"], s["v_cache"], s["v_scale"], s["most_pages"])
        return dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _attend(s)


# ---------------------------------------------------------------- plain forms

def _plan(s):
    """Requests in order get the pages their new tokens need from the ring's head; one that does not fit gets none (slot -1)."""
    page, tokens, table, ring = s["page"], s["tokens"], s["table"], s["free_pages"]
    ctx, done = s["ctx_len"].long(), s["new_len"] < 0
    new = s["new_len"].long().clamp(min=0)
    head, count = s["free_state"].long()
    ring_size = ring.numel()
    ends = torch.cumsum(new, 0)
    have = (ctx + page - 1) // page
    want = (ctx + new + page - 1) // page
    need = torch.where(done | (want > table.shape[1]) | (ends > tokens), 0, want - have)
    fits = ~done & (want <= table.shape[1]) & (ends <= tokens)
    first = torch.cumsum(need, 0) - need
    got = fits & ((need == 0) | (first + need <= count))
    taken = torch.where(got, need, 0).sum()
    short = need.sum() - taken
    seq_len = torch.where(done, 0, torch.where(got, ctx + new, ctx))
    q_start = torch.cat([ends.new_zeros(1), ends]).clamp(max=tokens)
    # tokens
    t = torch.arange(tokens, device=ctx.device)
    b = torch.searchsorted(q_start[1:], t, right=True).clamp(max=ctx.numel() - 1)
    inside = t < q_start[-1]
    i = t - q_start[b]
    position = ctx[b] + i
    at = position // page
    old = table[b, at.clamp(max=table.shape[1] - 1)].long()
    fresh = ring[(head + first[b] + at - have[b]) % ring_size].long()
    where = torch.where(at < have[b], old, fresh)
    ok = inside & got[b]
    slot = torch.where(ok, where * page + position % page, -1)
    opens = ok & (at >= have[b])
    cell = torch.where(opens, b * table.shape[1] + at, table.numel())
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[cell] = where.to(torch.int32)
    table.copy_(flat[:-1].view_as(table))
    # pages of finished requests go to the ring's end
    back = torch.where(done, have, 0)
    to = torch.cumsum(back, 0) - back
    j = torch.arange(table.shape[1], device=ctx.device)
    gone = j[None, :] < back[:, None]
    place = torch.where(gone, (head + count + to[:, None] + j[None, :]) % ring_size, ring_size)
    flat = torch.cat([ring, ring.new_zeros(1)])
    flat[place.reshape(-1)] = table.reshape(-1)
    ring.copy_(flat[:-1])
    state = torch.stack([(head + taken) % ring_size, count - taken + back.sum(), short]).to(torch.int32)
    return dict(seq_len=seq_len.to(torch.int32), q_start=q_start.to(torch.int32), slot=slot,
                position=torch.where(inside, position, -1).to(torch.int32), free_state=state, table=table, free_pages=ring)


def _append(x, slot, cache, scale, most):
    """A page's scale is the largest |value| it has held over 127; earlier tokens of a page whose scale grows are rounded again."""
    size = cache.shape[2]
    page, off = slot // size, slot % size
    xf = x.float()
    token = xf.abs().amax(-1) / xf.new_full((), 127.0)                           # [t, heads]; a number here would be multiplied by its reciprocal
    opens = torch.ones_like(slot, dtype=torch.bool)                              # first new token of its page
    opens[1:] = (off[1:] == 0) | (slot[1:] != slot[:-1] + 1)
    run_of = torch.cumsum(opens, 0) - 1
    runs = torch.full((most + 1,), -1, dtype=torch.int64, device=slot.device)
    runs[torch.where(opens, run_of, most)] = torch.where(opens, slot, -1)
    runs = runs[:most]
    live, where, before = runs >= 0, (runs // size).clamp(min=0), runs % size
    grown = torch.zeros((most, scale.shape[1]), device=slot.device).scatter_reduce(0, run_of[:, None].expand_as(token), token, "amax")
    old = torch.where((before > 0)[:, None], scale[where], 0.0)
    fresh = torch.maximum(old, grown)
    ratio = torch.where(fresh > 0, old / fresh, 0.0)
    pages = cache[where].float()                                                 # [most, heads, size, dim]
    again = torch.round(pages * ratio[:, :, None, None]).to(torch.int8)
    earlier = (torch.arange(size, device=slot.device)[None, :] < before[:, None]) & live[:, None]
    again = torch.where(earlier[:, None, :, None], again, cache[where])
    last = torch.where(live, where, cache.shape[0] - 1)                          # what pads the list goes to a page of nobody
    keep = live[:, None, None, None]
    cache[last] = torch.where(keep, again, cache[last])
    scale[last] = torch.where(live[:, None], fresh, scale[last])
    by = scale[page][:, :, None]
    cache[page, :, off] = torch.where(by > 0, torch.round(xf / by), 0.0).clamp(-127, 127).to(torch.int8)


def _attend(s):
    """softmax(scale q k^T) v for the newest tokens of each request; a row that sees no key is 0, and its log-sum -inf."""
    size, q, q_start, seq = s["page"], s["q"].float(), s["q_start"].long(), s["seq_len"].long()
    tokens, heads, dim = q.shape
    kvh, n, most = s["k_cache"].shape[1], seq.numel(), s["most_seq"]
    group = heads // kvh
    pages = s["table"][:, :-(-most // size)].long().clamp(min=0)                  # [n, blocks]
    j = torch.arange(pages.shape[1] * size, device=q.device)
    held = (j[None, :] < seq[:, None])[:, None, :, None]                         # [n, 1, keys, 1]

    def keys(cache, scale):
        x = cache[pages].float() * scale[pages][:, :, :, None, None]              # [n, blocks, kvh, size, dim]
        return torch.where(held, x.transpose(1, 2).reshape(n, kvh, -1, dim), 0.0)

    i = torch.arange(s["most_new"], device=q.device)
    new = q_start[1:] - q_start[:-1]
    at = (q_start[:-1, None] + i[None, :]).clamp(max=tokens - 1)                  # [n, rows]
    rows = q[at].view(n, -1, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kvh, -1, dim)
    position = seq[:, None] - new[:, None] + i[None, :]                           # [n, rows]
    sees = (j[None, None, :] <= position[:, :, None]) & (j[None, None, :] < seq[:, None, None])
    score = (rows @ keys(s["k_cache"], s["k_scale"]).transpose(-1, -2)).view(n, kvh, group, len(i), -1)
    score.mul_(s["scale"]).masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    out = p.view(n, kvh, -1, p.shape[-1]) @ keys(s["v_cache"], s["v_scale"])
    out = out.view(n, kvh, group, len(i), dim) / torch.where(total > 0, total, 1.0)
    lse = base[..., 0] + torch.log(total[..., 0])
    out = out.permute(0, 3, 1, 2, 4).reshape(n, len(i), heads, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(n, len(i), heads)
    t = torch.arange(tokens, device=q.device)
    b = torch.searchsorted(q_start[1:], t, right=True)
    return dict(out=out[b, t - q_start[b]].half(), lse=lse[b, t - q_start[b]].contiguous())


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    ctx, new = _lengths(case)
    page, n = case["page"], case["requests"]
    if case["op"] == "plan":
        t = sum(max(k, 0) for k in new)
        fresh = sum(-(-(c + k) // page) - -(-c // page) for c, k in zip(ctx, new) if k >= 0)
        back = sum(-(-c // page) for c, k in zip(ctx, new) if k < 0)
        return dict(bytes=16 * n + 12 * t + 8 * fresh + 8 * back, flops=0)
    kvh, dim = case["kv_heads"], case["dim"]
    t = sum(new)
    if case["op"] == "append":
        touched = sum(-(-(c + k) // page) - c // page for c, k in zip(ctx, new))
        return dict(bytes=2 * t * kvh * dim * 3 + 8 * t + 16 * touched * kvh, flops=4 * t * kvh * dim)
    heads = case["heads"]
    seq = [c + k for c, k in zip(ctx, new)]
    blocks = sum(-(-q // page) for q in seq)
    pairs = sum(k * c + k * (k + 1) // 2 for c, k in zip(ctx, new) if c >= 0)
    return dict(bytes=2 * sum(seq) * kvh * dim + 8 * blocks * kvh + 4 * blocks + 4 * t * heads * dim + 4 * t * heads + 8 * n,
                flops=4 * pairs * heads * dim)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers only
    if case["op"] == "append":
        slot, out = s["slot"].cpu().numpy(), {"k": None, "v": None}  # whole numbers, decided by binary32 quotients
        for name in ("k", "v"):
            top = np.abs(s[name].cpu().numpy().astype(np.float64)).max(-1)
            scale = s[name + "_scale"].cpu().numpy().astype(np.float64)
            seen = set()
            for t, at in enumerate(slot.tolist()):
                p = at // case["page"]
                if p not in seen and at % case["page"] == 0:
                    scale[p] = 0
                seen.add(p)
                scale[p] = np.maximum(scale[p], top[t] / 127)
            out[name + "_scale"] = scale
        return out
    ctx, new = _lengths(case)
    page, kvh, heads, dim = case["page"], case["kv_heads"], case["heads"], case["dim"]
    group, q = heads // kvh, s["q"].double()
    out, lse = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start = 0
    for b, (c, k) in enumerate(zip(ctx, new)):
        if c + k > 0:
            at = s["table"][b, :-(-(c + k) // page)].long()
            for h in range(kvh):
                kk, vv = ((s[x + "_cache"][at, h].double() * s[x + "_scale"][at, h].double()[:, None, None]).reshape(-1, dim)[:c + k] for x in "kv")
                for lo in range(0, k, 1024):
                    hi = min(k, lo + 1024)
                    z = torch.einsum("tgd,jd->tgj", q[start + lo:start + hi, h * group:(h + 1) * group], kk[:c + hi]) * dim ** -0.5
                    late = torch.arange(c + hi, device=DEV)[None, :] > torch.arange(c + lo, c + hi, device=DEV)[:, None]
                    z.masked_fill_(late[:, None, :], -math.inf)
                    lse[start + lo:start + hi, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
                    out[start + lo:start + hi, h * group:(h + 1) * group] = torch.softmax(z, -1) @ vv[:c + hi]
        start += k
    return dict(out=out, lse=lse)
