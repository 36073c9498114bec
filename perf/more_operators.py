"""Attention over long paged contexts, measured one operator at a time.

Two ways of not reading all of every request's cache at every step, over the pool of K/V
blocks that many requests share (perf/operators.py has the pool's own operators):

  bounds  the smallest and largest key of every block that a step's tokens lie in, by
          dimension: what select goes by
  select  for each query token and K/V head, the pages of its request that may hold its
          largest scores: some first ones, some last ones, and the best by an upper bound of
          the sum of its queries' scores,
          sum_d max_d sum_h max(q_hd, 0) + min_d sum_h min(q_hd, 0)
  sparse  attention of each query token over the pages it is given for each K/V head
  prefix  attention of each query token over a prefix that its group of rows shares (a
          request of its own, read once for the group) and then over its own request

`run` computes them with elementary torch operations; with `own` set it calls the
framework's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one new token for each of 64 sessions: each block's bounds follow its last row
        dict(name="bounds_step_b64", op="bounds", requests=64, pad=0, kv_heads=8, head_dim=128,
             cache="bf16", block=16, max_len=9000, max_new=1, lens_seed=1),
        # the prompts of new requests: every block that they fill is read once
        dict(name="bounds_prompts", op="bounds", requests=24, pad=100, kv_heads=8, head_dim=128,
             cache="bf16", block=32, max_len=500, max_new=8192, lens_seed=2),
        # one request with a long context
        dict(name="select_b1_long", op="select", rows=1, pad=0, empty=0, heads=32, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=16, columns=8192, min_len=131071,
             max_len=131071, top=128, first=1, last=2, lens_seed=3),
        # a padded batch of contexts of different lengths, some of fewer pages than are asked for
        dict(name="select_b64", op="select", rows=64, pad=3, empty=1, heads=32, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=32, columns=2048, min_len=1000,
             max_len=65000, top=64, first=1, last=2, lens_seed=4),
        # one request: 2048 of its 131071 positions for each K/V head
        dict(name="sparse_b1_long", op="sparse", rows=1, pad=0, empty=0, heads=32, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=16, columns=8192, min_len=131071,
             max_len=131071, top=128, lens_seed=5),
        # a padded batch of long contexts, 64 pages of 32 positions each
        dict(name="sparse_b64", op="sparse", rows=64, pad=3, empty=1, heads=32, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=32, columns=512, min_len=1000,
             max_len=16384, top=64, lens_seed=6),
        # an f32 model, blocks of odd size, three queries a K/V head
        dict(name="sparse_f32_odd", op="sparse", rows=33, pad=1, empty=1, heads=12, kv_heads=4,
             head_dim=32, io="f32", cache="f32", block=5, columns=400, min_len=1, max_len=1900,
             top=37, lens_seed=7),
        # the small model behind a short shared start: latency is all
        dict(name="prefix_b8_short", op="prefix", rows=8, pad=0, alone=0, groups=1, heads=16,
             kv_heads=16, head_dim=64, io="f32", cache="bf16", block=16, columns=32,
             min_prefix=200, max_prefix=200, max_len=40, lens_seed=8),
        # 64 sessions of the 7B shape that start alike, f32 activations
        dict(name="prefix_b64_f32", op="prefix", rows=64, pad=0, alone=0, groups=1, heads=32,
             kv_heads=32, head_dim=128, io="f32", cache="bf16", block=16, columns=190,
             min_prefix=2500, max_prefix=2500, max_len=400, lens_seed=9),
        # 64 requests about one long document, four queries a K/V head
        dict(name="prefix_b64_long", op="prefix", rows=64, pad=0, alone=0, groups=1, heads=32,
             kv_heads=8, head_dim=128, io="bf16", cache="bf16", block=16, columns=2048,
             min_prefix=32768, max_prefix=32768, max_len=512, lens_seed=10),
        # a padded batch: groups of different sizes and prefixes, and requests that share nothing
        dict(name="prefix_groups", op="prefix", rows=250, pad=6, alone=9, groups=5, heads=64,
             kv_heads=8, head_dim=128, io="bf16", cache="bf16", block=32, columns=512,
             min_prefix=300, max_prefix=16000, max_len=300, lens_seed=11),
        # an f32 cache with blocks of odd size
        dict(name="prefix_f32_odd", op="prefix", rows=45, pad=2, alone=1, groups=3, heads=12,
             kv_heads=4, head_dim=64, io="f32", cache="f32", block=24, columns=180,
             min_prefix=100, max_prefix=4000, max_len=90, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "sparse", "prefix", "prefix", "prefix"])
    seed = rng.randrange(1 << 30)
    head_dim = rng.choice([32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16] if kv_heads <= 4 else [1, 2, 4, 8])
    cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
    io = rng.choice(["bf16", "f32"])
    block = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128])
    if op == "bounds":
        requests = _log(rng, 1, 300)
        max_new = rng.choice([1, _log(rng, 1, 4000)])
        return dict(op=op, requests=requests, pad=rng.randint(0, 40), kv_heads=kv_heads,
                    head_dim=head_dim, cache=cache, block=block, max_len=_log(rng, 1, 2000),
                    max_new=max(1, min(max_new, 100000 // requests)), lens_seed=seed)
    if op in ("select", "sparse"):
        rows = _log(rng, 1, 128)
        # pages of the largest row: what the bounds, or the cache, of all rows may take
        cap = max(4, 250_000_000 // (rows * kv_heads * head_dim * (2 if op == "select" else block)))
        max_len = min(_log(rng, 1, 120000), cap * block)
        pages = max_len // block + 1
        first, last = rng.randint(0, 3), rng.randint(1, 4)
        top = max(min(_log(rng, 1, 200), 1 + 8192 // block), first + last)
        c = dict(op=op, rows=rows, pad=rng.randint(0, rows // 6), empty=rng.randint(0, rows // 10),
                 heads=heads, kv_heads=kv_heads, head_dim=head_dim, io=io, cache=cache,
                 block=block, columns=max(1, pages + rng.randint(-pages // 4, 9)),
                 min_len=rng.choice([1, max(1, max_len // 2)]), max_len=max_len, top=top,
                 lens_seed=seed)
        if op == "select":
            c.update(first=first, last=last)
        return c
    rows = _log(rng, 1, 256)
    groups = min(rows, rng.choice([1, 1, 2, 3, 8]))
    # products of queries and keys, and the cache of the largest prefixes
    most = min(8_000_000_000 // (rows * heads * head_dim), 200_000_000 // (groups * kv_heads * head_dim))
    if cache == "f32":
        most //= 4
    max_prefix = min(_log(rng, 1, 50000), max(1, most))
    max_len = min(_log(rng, 1, 1500), max(1, 100_000_000 // (rows * kv_heads * head_dim)))
    return dict(op=op, rows=rows, pad=rng.randint(0, rows // 6), alone=rng.randint(0, rows // 6),
                groups=groups, heads=heads, kv_heads=kv_heads, head_dim=head_dim, io=io,
                cache=cache, block=block,
                columns=max(max_prefix, max_len) // block + 1 + rng.randint(0, 9),
                min_prefix=rng.choice([1, max(1, max_prefix // 2)]), max_prefix=max_prefix,
                max_len=max_len, lens_seed=seed)


# ---------------------------------------------------------------- lengths of a case
def _bounds_tokens(c):
    """Runs of new tokens, one a request: (position of the first, number)."""
    r = random.Random(c["lens_seed"])
    runs = []
    for _ in range(c["requests"]):
        new = r.randint(max(1, c["max_new"] // 8), c["max_new"])
        runs.append((_log(r, 1, c["max_len"]) - 1, new))
    return runs


def _row_positions(c):
    """The query's position of every row: -1 for a request that holds nothing, None for padding."""
    r = random.Random(c["lens_seed"])
    n = c["rows"] - c["pad"] - c["empty"]
    lens = [c["max_len"]] + [_log(r, c["min_len"], c["max_len"]) for _ in range(n - 1)]
    rows = [x - 1 for x in lens[:max(n, 0)]] + [-1] * c["empty"]
    r.shuffle(rows)
    return rows + [None] * c["pad"]


def _live_pages(c, pos):
    """First and last page that the table holds of a row."""
    last = pos // c["block"]
    return max(0, last - c["columns"] + 1), last


def _listed_pages(c):
    """Pages that a sparse case's rows are given, a sorted list for each row and K/V head."""
    r = random.Random(c["lens_seed"] + 1)
    rows = []
    for p in _row_positions(c):
        heads = []
        for _ in range(c["kv_heads"]):
            if p is None or p < 0:
                heads.append([])
                continue
            lo, last = _live_pages(c, p)
            n = min(c["top"], last - lo + 1)
            heads.append(sorted(r.sample(range(lo, last), n - 1)) + [last])
        rows.append(heads)
    return rows


def _prefix_lens(c):
    """(rows of each group, length of each prefix, own position of every row or None): groups
    first, then rows that share nothing, then padding."""
    r = random.Random(c["lens_seed"])
    n = c["rows"] - c["pad"] - c["alone"]
    cuts = sorted(r.randint(0, n) for _ in range(c["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    lens = [c["max_prefix"]] + [_log(r, c["min_prefix"], c["max_prefix"]) for _ in range(c["groups"] - 1)]
    own_pos = [_log(r, 1, c["max_len"]) - 1 for _ in range(c["rows"] - c["pad"])]
    return sizes, lens, own_pos + [None] * c["pad"]


# ---------------------------------------------------------------- inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tables(c, pages, g):
    """A block table whose request b holds pages[b] blocks of a shuffled pool, and the pool's size."""
    N = sum(pages) + 3
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(pages), c["columns"]), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(c["columns"], device="cuda") < _ints(pages)[:, None]] = order[:sum(pages)]
    return table, N


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    hd, Hk, P = c["head_dim"], c["kv_heads"], c["block"]
    kt = DTYPES[c["cache"]]
    s = {"case": c}
    if c["op"] == "bounds":
        runs = _bounds_tokens(c)
        pages = [(first + n - 1) // P + 1 for first, n in runs]
        N = sum(pages) + 3
        order = torch.randperm(N, generator=g, device="cuda")
        pos = [p for first, n in runs for p in range(first, first + n)]
        base = [b for b, (first, n) in enumerate(runs) for _ in range(n)]
        start = [0]
        for n in pages:
            start.append(start[-1] + n)
        at = _ints(pos, torch.int64)
        page = _ints(start, torch.int64)[_ints(base, torch.int64)] + at // P
        slots = torch.cat([order[page] * P + at % P, _ints([-1] * c["pad"], torch.int64)])
        s.update(k=normal(N, P, Hk, hd, dtype=kt), positions=_ints(pos + [-1] * c["pad"]), slots=slots,
                 bounds=normal(N, Hk, 2, hd, dtype=kt))
        # blocks that the step's tokens lie in, as a program that lays out its runs has it
        s["blocks"] = sum((first + n - 1) // P - first // P + 1 for first, n in runs)
        return s
    if c["op"] == "prefix":
        sizes, lens, own_pos = _prefix_lens(c)
        R, G = c["rows"], len(sizes)
        # requests: the rows' own, then the prefixes
        pages = [0 if p is None else p // P + 1 for p in own_pos] + [-(-n // P) for n in lens]
        table, N = _tables(c, pages, g)
        cu = [0]
        for n in sizes:
            cu.append(cu[-1] + n)
        s.update(table=table, cu_rows=_ints(cu), prefix_requests=_ints([R + i for i in range(G)]),
                 prefix_lens=_ints(lens), groups=(cu, lens),
                 requests=_ints([-1 if p is None else r for r, p in enumerate(own_pos)]),
                 positions=_ints([-1 if p is None else p for p in own_pos]))
        s["span"] = max([1] + [p + 1 for p in own_pos if p is not None])
    else:
        rows = _row_positions(c)
        live = [None if p is None or p < 0 else _live_pages(c, p) for p in rows]
        # a table that has wrapped holds its last pages at page % columns, all columns taken
        table, N = _tables(c, [0 if x is None else min(x[1] + 1, c["columns"]) for x in live], g)
        s.update(table=table, requests=_ints([-1 if p is None else r for r, p in enumerate(rows)]),
                 positions=_ints([-1 if p is None else p for p in rows]))
        s["span"] = max([1] + [b - a + 1 for x in live if x is not None for a, b in [x]])
    s["q"] = normal(c["rows"], c["heads"] * hd).to(DTYPES[c["io"]])
    if c["op"] == "select":
        # bounds around means that differ from page to page, as keys of one passage are alike
        mid, half = normal(N, Hk, 1, hd).mul_(0.5), normal(N, Hk, 1, hd).mul_(0.3).abs_().add_(1.3)
        s["bounds"] = torch.cat([mid - half, mid + half], 2).to(kt)
        s["pages"] = torch.full((c["rows"], Hk, c["top"]), -7, dtype=torch.int32, device="cuda")
        return s
    s.update(k=normal(N, P, Hk, hd, dtype=kt), v=normal(N, P, Hk, hd, dtype=kt),
             out=normal(c["rows"], c["heads"] * hd).to(DTYPES[c["io"]]), lse=normal(c["rows"], c["heads"]))
    if c["op"] == "sparse":
        lists = [x + [-1] * (c["top"] - len(x)) for row in _listed_pages(c) for x in row]
        s["pages"] = _ints(lists).view(c["rows"], Hk, c["top"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"bounds": _bounds, "select": _select, "sparse": _sparse, "prefix": _prefix}[c["op"]](c, state)


def _own(c, s):
    from rq_transformer_frame_gb300 import paged

    if c["op"] == "bounds":
        return {"bounds": paged.paged_bounds(s["k"], s["bounds"], s["positions"], s["slots"])}
    if c["op"] == "select":
        return {"pages": paged.paged_select(s["q"], s["bounds"], s["table"], s["positions"],
                                            block_size=c["block"], top=c["top"], first=c["first"],
                                            last=c["last"], requests=s["requests"], pages=s["pages"])}
    if c["op"] == "sparse":
        out, lse = paged.paged_sparse_attention(s["q"], s["k"], s["v"], s["table"], s["positions"],
                                                s["pages"], requests=s["requests"], out=s["out"],
                                                lse=s["lse"])
    else:
        out, lse = paged.paged_prefix_attention(s["q"], s["k"], s["v"], s["table"], s["positions"],
                                                s["cu_rows"], s["prefix_requests"], s["prefix_lens"],
                                                requests=s["requests"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def _bounds(c, s):
    P = c["block"]
    slots = s["slots"]
    live = (s["positions"] >= 0) & (slots >= 0)
    # the last token of each block in the step: its rows so far are the block's live ones
    block = torch.where(live, slots // P, -1)
    last = live & (block != torch.cat([block[1:], torch.full_like(block[:1], -2)]))
    at = torch.sort((~last).int(), stable=True).indices[:s["blocks"]]
    size = max(1, (1 << 26) // (P * c["kv_heads"] * c["head_dim"]))
    for t in range(0, s["blocks"], size):
        b = block[at[t:t + size]]
        keys = s["k"][b].float()
        ok = (torch.arange(P, device=b.device) <= (slots[at[t:t + size]] % P)[:, None])[..., None, None]
        low = torch.where(ok, keys, math.inf).amin(1)
        high = torch.where(ok, keys, -math.inf).amax(1)
        s["bounds"][b] = torch.stack([low, high], 2).to(s["bounds"].dtype)
    return {"bounds": s["bounds"]}


def _select(c, s):
    R, H, Hk, hd, P, W = c["rows"], c["heads"], c["kv_heads"], c["head_dim"], c["block"], c["columns"]
    pos, req = s["positions"].long()[:, None], s["requests"].long()[:, None]
    final = torch.where(pos >= 0, pos // P, -1)
    lo = (final - W + 1).clamp(min=0)
    page = lo + torch.arange(s["span"], device=pos.device)
    block = s["table"][req.clamp(min=0), page % W].long()
    live = (page <= final) & (req >= 0)
    always = live & ((page < lo + c["first"]) | (page > final - c["last"]))
    there = live & ~always & (block >= 0) & (block < s["bounds"].shape[0])
    # scores next to the border of the best ones decide: 64 bits
    q = s["q"].double().view(R, Hk, H // Hk, hd)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    b = s["bounds"][torch.where(there, block, 0)]
    score = torch.stack([(b[r, :, :, 1].double() * up[r] + b[r, :, :, 0].double() * down[r]).sum(-1)
                         for r in range(R)]).transpose(1, 2)
    score = torch.where(there[:, None] & ~score.isnan(), score, -math.inf)
    # the missing behind all others, whatever those score
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(there[:, None].expand_as(score).gather(-1, order).int(), dim=-1,
                                        descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(s["span"], device=pos.device).expand_as(order))
    taken = always[:, None] | (there[:, None] & (rank < c["top"] - c["first"] - c["last"]))
    big = 1 << 40
    chosen = torch.where(taken, page[:, None], big).sort(-1).values[..., :c["top"]]
    chosen = torch.nn.functional.pad(chosen, (0, c["top"] - chosen.shape[-1]), value=big)
    chosen = torch.where(chosen == big, -1, chosen).int()
    s["pages"].copy_(torch.where(req[..., None] >= 0, chosen, s["pages"]))
    return {"pages": s["pages"]}


def _softmax_sums(score, v):
    """(largest score or 0, sum of e^(score - largest), the values' sum by those weights)."""
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0)
    p = (score - top).exp()
    return top, p.sum(-1, keepdim=True), p @ v


def _finish(c, s, top, total, o):
    R, kept = c["rows"], s["requests"].long()[:, None] >= 0
    o = torch.where(total > 0, o / total.clamp(min=1e-30), 0)
    s["out"].copy_(torch.where(kept, o.reshape(R, -1), s["out"].float()))
    s["lse"].copy_(torch.where(kept, (top + total.log()).reshape(R, -1), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _sparse(c, s):
    R, H, Hk, hd, P, W = c["rows"], c["heads"], c["kv_heads"], c["head_dim"], c["block"], c["columns"]
    N = s["k"].shape[0]
    pos, req = s["positions"].long()[:, None, None], s["requests"].long()[:, None, None]
    page = s["pages"].long()
    final = torch.where(pos >= 0, pos // P, -1)
    block = s["table"][req.clamp(min=0).expand_as(page), page.clamp(min=0) % W].long()
    ok = (page >= 0) & (page <= final) & (page > final - W) & (block >= 0) & (block < N) & (req >= 0)
    off = torch.arange(P, device=pos.device)
    live = (ok[..., None] & (page[..., None] * P + off <= pos[..., None])).flatten(2)
    at = (block.clamp(0, N - 1)[..., None] * P + off).flatten(2)
    head = torch.arange(Hk, device=pos.device)[:, None]
    k = s["k"].view(N * P, Hk, hd)[at, head].float()
    v = torch.where(live[..., None], s["v"].view(N * P, Hk, hd)[at, head].float(), 0)
    score = s["q"].float().view(R, Hk, H // Hk, hd) @ k.transpose(2, 3) * (1.0 / math.sqrt(hd))
    return _finish(c, s, *_softmax_sums(torch.where(live[:, :, None], score, -math.inf), v))


def _prefix(c, s):
    R, H, Hk, hd, P, W = c["rows"], c["heads"], c["kv_heads"], c["head_dim"], c["block"], c["columns"]
    scale = 1.0 / math.sqrt(hd)
    pool_k, pool_v = s["k"].view(-1, Hk, hd), s["v"].view(-1, Hk, hd)
    pos, req = s["positions"].long()[:, None], s["requests"].long()[:, None]
    # each row's own request
    j = torch.arange(s["span"], device=pos.device)
    at = s["table"][req.clamp(min=0), j // P].long().clamp(min=0) * P + j % P
    live = (j <= pos)[:, None, None]
    q = s["q"].float().view(R, Hk, H // Hk, hd)
    score = q @ pool_k[at].float().permute(0, 2, 3, 1) * scale
    top, total, o = _softmax_sums(torch.where(live, score, -math.inf),
                                  torch.where(live[:, 0, 0, :, None, None], pool_v[at], 0).float().permute(0, 2, 1, 3))
    # the prefixes, each for all rows of its group
    cu, lens = s["groups"]
    for i, n in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        j = torch.arange(n, device=pos.device)
        at = s["table"][s["prefix_requests"][i].long(), j // P].long() * P + j % P
        k, v = pool_k[at].float().permute(1, 2, 0), pool_v[at].float().transpose(0, 1)
        x = q[a:b].transpose(0, 1).reshape(Hk, -1, hd)
        shared = [y.view(Hk, b - a, H // Hk, -1).transpose(0, 1) for y in _softmax_sums(x @ k * scale, v)]
        most = torch.maximum(top[a:b], shared[0])
        f, g = (top[a:b] - most).exp(), (shared[0] - most).exp()
        # a row that holds nothing of its own weighs nothing
        f = torch.where(total[a:b] > 0, f, 0)
        most = torch.where(total[a:b] > 0, most, shared[0])
        g = torch.where(total[a:b] > 0, g, 1)
        total[a:b] = total[a:b] * f + shared[1] * g
        o[a:b] = o[a:b] * f + shared[2] * g
        top[a:b] = most
    return _finish(c, s, top, total, o)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    hd, Hk, P, kb = c["head_dim"], c["kv_heads"], c["block"], SIZE[c["cache"]]
    if c["op"] == "bounds":
        rows = blocks = tokens = 0
        for first, n in _bounds_tokens(c):
            lo = first // P * P
            rows += first + n - lo
            blocks += (first + n - 1) // P - first // P + 1
            tokens += n
        return {"bytes": (rows + 2 * blocks) * Hk * hd * kb + 12 * tokens, "flops": 2 * rows * Hk * hd}
    H, G = c["heads"], c["heads"] // c["kv_heads"]
    io = SIZE[c["io"]]
    if c["op"] == "prefix":
        sizes, lens, own_pos = _prefix_lens(c)
        mine = sum(p + 1 for p in own_pos if p is not None)
        shared = sum(n for n, m in zip(lens, sizes) if m)
        rows = c["rows"] - c["pad"]
        return {"bytes": (mine + shared) * (Hk * hd * 2 * kb + 4 / P) + rows * (2 * H * hd * io + 4 * H + 8),
                "flops": 4 * H * hd * (mine + sum(n * m for n, m in zip(lens, sizes)))}
    rows = [p for p in _row_positions(c) if p is not None]
    if c["op"] == "select":
        scored = 0
        for p in rows:
            if p >= 0:
                lo, last = _live_pages(c, p)
                n = last - lo + 1
                scored += max(0, n - c["first"] - c["last"]) if n > c["top"] else 0
        return {"bytes": scored * (Hk * 2 * hd * kb + 4) + len(rows) * (H * hd * io + 4 * Hk * c["top"] + 8),
                "flops": scored * Hk * hd * 4 + len(rows) * 2 * H * hd}
    keys = 0
    for p, heads in zip(_row_positions(c), _listed_pages(c)):
        keys += sum(min(P, p + 1 - page * P) for pages in heads for page in pages)
    return {"bytes": keys * hd * 2 * kb + len(rows) * (2 * H * hd * io + 4 * H + 8 + 4 * Hk * c["top"]),
            "flops": 4 * keys * G * hd}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    hd, Hk, P = c["head_dim"], c["kv_heads"], c["block"]
    if c["op"] == "select":
        return None  # whole numbers
    if c["op"] == "bounds":
        out = s["bounds"].double()
        slots = s["slots"].cpu().tolist()
        ends = {}
        for x in slots:
            if x >= 0:
                ends[x // P] = max(ends.get(x // P, 0), x % P)
        for n in set(ends.values()):
            blocks = _ints([b for b, e in ends.items() if e == n], torch.int64)
            rows = s["k"][blocks, :n + 1].double()
            out[blocks] = torch.stack([rows.min(1).values, rows.max(1).values], 2)
        return {"bounds": out}
    out, lse = s["out"].double(), s["lse"].double()
    table, W = s["table"].cpu().long(), c["columns"]
    H = c["heads"]
    G = H // Hk

    def rows_of(request, positions):
        return table[request][(positions // P) % W].cuda(), (positions % P).cuda()

    if c["op"] == "sparse":
        for r, (p, heads) in enumerate(zip(_row_positions(c), _listed_pages(c))):
            if p is None:
                continue
            out[r], lse[r] = 0, -math.inf
            for h, pages in enumerate(heads):
                if not pages:
                    continue
                j = (torch.tensor(pages)[:, None] * P + torch.arange(P)).flatten()
                b, i = rows_of(r, j[j <= p])
                k, v = s["k"][b, i, h].double(), s["v"][b, i, h].double()
                score = s["q"][r].double().view(H, hd)[h * G:(h + 1) * G] @ k.T / math.sqrt(hd)
                lse[r, h * G:(h + 1) * G] = torch.logsumexp(score, -1)
                out[r, h * G * hd:(h + 1) * G * hd] = (torch.softmax(score, -1) @ v).flatten()
        return {"out": out, "lse": lse}
    sizes, lens, own_pos = _prefix_lens(c)
    of = [g for g, m in enumerate(sizes) for _ in range(m)]
    held = {}
    for r, p in enumerate(own_pos):
        if p is None:
            continue
        b, i = rows_of(r, torch.arange(p + 1))
        k, v = s["k"][b, i].double(), s["v"][b, i].double()
        if r < len(of):
            if of[r] not in held:
                held.clear()
                b, i = rows_of(c["rows"] + of[r], torch.arange(lens[of[r]]))
                held[of[r]] = (s["k"][b, i].double(), s["v"][b, i].double())
            k, v = torch.cat([held[of[r]][0], k]), torch.cat([held[of[r]][1], v])
        q = s["q"][r].double().view(Hk, G, hd)
        score = torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(hd)
        lse[r] = torch.logsumexp(score, -1).flatten()
        out[r] = torch.bmm(torch.softmax(score, -1), v.transpose(0, 1)).flatten()
    return {"out": out, "lse": lse}
