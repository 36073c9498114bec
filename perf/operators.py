"""The paged K/V cache's operators, measured one call at a time.

Three operators serve one decode step over a pool of K/V blocks that many requests share:

  plan    lengths -> blocks taken and returned, block table, and request, position and
          cache slot of every new token
  append  the rows of a fused qkv projection: norm of every query and key head, position
          rotation, queries out, keys and values stored at their slots
  attend  one query token per row over the blocks of its request

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
        # one new token for each of 64 live sessions: the step every frame of a server starts with
        dict(name="plan_step_b64", op="plan", batch=64, live=64, tokens=64, block=16, columns=190,
             max_len=2990, prompts=0, ended=0, max_prompt=1, lens_seed=1),
        # a large server's step: most requests add one token, some end, some bring a prompt
        dict(name="plan_mixed_b1000", op="plan", batch=1000, live=940, tokens=65536, block=16,
             columns=512, max_len=7000, prompts=40, ended=50, max_prompt=2500, lens_seed=2),
        # admission of long prompts into few requests
        dict(name="plan_prompts_b8", op="plan", batch=8, live=8, tokens=262144, block=64,
             columns=1024, max_len=500, prompts=8, ended=0, max_prompt=32000, lens_seed=3),
        # one token of one session at the 7B shape: plain rotation, f32 activations, bf16 cache
        dict(name="append_b1", op="append", rows=1, pad=0, heads=32, kv_heads=32, head_dim=128,
             io="f32", out="f32", cache="bf16", norm=False, rope="interleaved", rope_dim=128,
             block=16, max_pos=2999, lens_seed=4),
        # a decode batch padded to its graph's 64 rows, grouped heads, normed queries and keys
        dict(name="append_b64", op="append", rows=64, pad=4, heads=32, kv_heads=8, head_dim=128,
             io="bf16", out="bf16", cache="bf16", norm=True, rope="halves", rope_dim=128,
             block=16, max_pos=40000, lens_seed=5),
        # prompt tokens of many requests in one pass
        dict(name="append_prompts", op="append", rows=16384, pad=0, heads=32, kv_heads=8,
             head_dim=128, io="bf16", out="bf16", cache="bf16", norm=True, rope="halves",
             rope_dim=128, block=64, max_pos=130000, lens_seed=6),
        # an f32 model, odd row count, part of each head rotated, blocks of odd size
        dict(name="append_f32_odd", op="append", rows=777, pad=5, heads=16, kv_heads=4, head_dim=64,
             io="f32", out="f32", cache="f32", norm=True, rope="interleaved", rope_dim=32,
             block=5, max_pos=500, lens_seed=7),
        # the small model's first seconds, one session: latency is all
        dict(name="attend_b1_short", op="attend", rows=1, pad=0, empty=0, heads=16, kv_heads=16,
             head_dim=64, io="f32", cache="bf16", block=16, columns=32, window=512, min_len=200,
             max_len=200, lens_seed=8),
        # one request with a long context: the work is one row's, split over the card
        dict(name="attend_b1_long", op="attend", rows=1, pad=0, empty=0, heads=32, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=64, columns=2048, window=0,
             min_len=131071, max_len=131071, lens_seed=9),
        # 64 sessions of the 7B shape past their window: the block tables have wrapped
        dict(name="attend_b64_window", op="attend", rows=64, pad=0, empty=0, heads=32, kv_heads=32,
             head_dim=128, io="f32", cache="bf16", block=16, columns=190, window=3000,
             min_len=2800, max_len=9000, lens_seed=10),
        # a padded batch of requests from one token to long contexts, eight queries a K/V head
        dict(name="attend_b256_ragged", op="attend", rows=256, pad=6, empty=3, heads=64, kv_heads=8,
             head_dim=128, io="bf16", cache="bf16", block=32, columns=512, window=0, min_len=1,
             max_len=16384, lens_seed=11),
        # an f32 cache with blocks of odd size, three queries a K/V head
        dict(name="attend_f32_odd", op="attend", rows=33, pad=1, empty=1, heads=12, kv_heads=4,
             head_dim=32, io="f32", cache="f32", block=5, columns=400, window=0, min_len=1,
             max_len=1900, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    seed = rng.randrange(1 << 30)
    if op == "plan":
        batch = _log(rng, 1, 1500)
        live = rng.randint(max(1, batch // 2), batch)
        ended = rng.randint(0, live // 8)
        prompts = rng.randint(0, max(1, (live - ended) // 8))
        block = rng.choice([1, 5, 8, 16, 24, 32, 64, 128])
        max_len = _log(rng, 1, 4000)
        max_prompt = max(1, min(_log(rng, 1, 16000), 131072 // max(1, prompts)))
        columns = min(2048, (max_len + max_prompt) // block + 2)
        tokens = live + prompts * max_prompt + rng.randint(0, 64)
        return dict(op=op, batch=batch, live=live, tokens=tokens, block=block, columns=columns,
                    max_len=max_len, prompts=prompts, ended=ended, max_prompt=max_prompt,
                    lens_seed=seed)
    head_dim = rng.choice([32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16] if kv_heads <= 4 else [1, 2, 4, 8])
    cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
    io = rng.choice(["bf16", "f32"])
    block = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128])
    if op == "append":
        rows = _log(rng, 1, max(2, 50_000_000 // ((heads + 2 * kv_heads) * head_dim)) // 4)
        rows = min(rows, 16384)
        return dict(op=op, rows=rows, pad=rng.randint(0, rows // 4), heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, io=io, out=rng.choice([io, "f32"]), cache=cache,
                    norm=rng.random() < 0.7, rope=rng.choice(["interleaved", "halves"]),
                    rope_dim=rng.choice([0, 16, 24, 32, head_dim, head_dim]), block=block,
                    max_pos=_log(rng, 16, 200000), lens_seed=seed)
    rows = _log(rng, 1, 256)
    cap = max(2, 400_000_000 // (rows * kv_heads * head_dim))
    max_len = min(_log(rng, 1, 100000), cap)
    columns = min(max_len // block + 1 + rng.randint(0, 9), 16384)
    window = rng.choice([0, 0, max(1, max_len // 2), _log(rng, 1, 4000)])
    return dict(op=op, rows=rows, pad=rng.randint(0, rows // 6), empty=rng.randint(0, rows // 10),
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, io=io, cache=cache, block=block,
                columns=columns, window=window, min_len=rng.choice([1, max(1, max_len // 2)]),
                max_len=max_len, lens_seed=seed)


# ---------------------------------------------------------------- lengths of a case
def _plan_lens(c):
    """(tokens held, tokens to add; -1: the request has ended) of every request."""
    r = random.Random(c["lens_seed"])
    B, live = c["batch"], c["live"]
    kind = ["end"] * c["ended"] + ["prompt"] * c["prompts"]
    kind += ["step"] * (live - len(kind)) + ["idle"] * (B - live)
    r.shuffle(kind)
    held, new = [], []
    for k in kind:
        held.append(_log(r, 1, c["max_len"]) if k in ("end", "step") else 0)
        new.append({"end": -1, "step": 1, "idle": 0}.get(k, 0))
        if k == "prompt":
            new[-1] = r.randint(max(1, c["max_prompt"] // 4), c["max_prompt"])
    return held, new


def _append_positions(c):
    """Positions of the rows: runs of consecutive ones, as prompts and steps bring them; -1: padding."""
    r = random.Random(c["lens_seed"])
    n, pos = c["rows"] - c["pad"], []
    while len(pos) < n:
        run = min(n - len(pos), _log(r, 1, max(1, n // 4)))
        start = r.randint(0, c["max_pos"])
        pos += range(start, start + run)
    return pos + [-1] * c["pad"]


def _attend_positions(c):
    """The query's position of every row: -1 for a request that holds nothing, None for padding."""
    r = random.Random(c["lens_seed"])
    n = c["rows"] - c["pad"] - c["empty"]
    lens = [c["max_len"]] + [_log(r, c["min_len"], c["max_len"]) for _ in range(n - 1)]
    rows = [x - 1 for x in lens] + [-1] * c["empty"]
    r.shuffle(rows)
    return rows + [None] * c["pad"]


def _first_key(c, pos):
    lo = 0 if not c["window"] else max(0, pos + 1 - c["window"])
    return max(lo, (pos // c["block"] - c["columns"] + 1) * c["block"])


# ---------------------------------------------------------------- inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    s = {"case": c}
    if c["op"] == "plan":
        held, new = _plan_lens(c)
        W, P = c["columns"], c["block"]
        pages = [min(-(-h // P), W) for h in held]
        need = sum(min(-(-(h + n) // P), W) - p for h, n, p in zip(held, new, pages) if n > 0)
        used = sum(pages)
        N = used + need + 17
        order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["batch"], W), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(W, device="cuda") < _ints(pages)[:, None]] = order[:used]
        # the free blocks stand in a ring, from a place of their own
        head = int(torch.randint(0, N, (1,), generator=g, device="cuda"))
        ids = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        ids[(head + torch.arange(N - used, device="cuda")) % N] = order[used:]
        empty = lambda n, dtype=torch.int32: torch.empty(n, dtype=dtype, device="cuda")  # noqa: E731
        s.update(new_lens=_ints(new), lens=_ints(held), table=table, free_ids=ids,
                 pool=_ints([head, N - used, 0, 0]),
                 # the buffers that a serving loop keeps for its step's maps
                 maps=(empty(c["batch"]), empty(4), empty(c["batch"] + 1), empty(c["tokens"]),
                       empty(c["tokens"]), empty(c["tokens"], torch.int64)))
        return s
    hd, Hk, H = c["head_dim"], c["kv_heads"], c["heads"]
    if c["op"] == "append":
        pos = _append_positions(c)
        n = c["rows"] - c["pad"]
        N = n // c["block"] + 4
        slots = torch.full((c["rows"],), -1, dtype=torch.int64, device="cuda")
        slots[:n] = torch.randperm(N * c["block"], generator=g, device="cuda")[:n]
        # one block more than the pool has: plain stores of padding rows land there
        shape = (N + 1, c["block"], Hk, hd)
        s.update(qkv=normal(c["rows"], (H + 2 * Hk) * hd).mul_(2).to(DTYPES[c["io"]]),
                 positions=_ints(pos), slots=slots,
                 k=normal(*shape, dtype=DTYPES[c["cache"]]), v=normal(*shape, dtype=DTYPES[c["cache"]]),
                 q_alpha=1 + 0.1 * normal(hd) if c["norm"] else None,
                 k_alpha=1 + 0.1 * normal(hd) if c["norm"] else None,
                 out=normal(c["rows"], H * hd).to(DTYPES[c["out"]]))
        s.update(pool_k=s["k"][:-1], pool_v=s["v"][:-1])
        return s
    rows = _attend_positions(c)
    P, W = c["block"], c["columns"]
    first = [None if p is None or p < 0 else _first_key(c, p) for p in rows]
    pages = [0 if f is None else min(p // P + 1, W) for p, f in zip(rows, first)]
    N = sum(pages) + 3
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["rows"], W), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(W, device="cuda") < _ints(pages)[:, None]] = order[:sum(pages)]
    requests = [-1 if p is None else r for r, p in enumerate(rows)]
    s.update(q=normal(c["rows"], H * hd).to(DTYPES[c["io"]]),
             k=normal(N, P, Hk, hd, dtype=DTYPES[c["cache"]]), v=normal(N, P, Hk, hd, dtype=DTYPES[c["cache"]]),
             table=table, requests=_ints(requests), positions=_ints([-1 if p is None else p for p in rows]),
             out=normal(c["rows"], H * hd).to(DTYPES[c["io"]]), lse=normal(c["rows"], H))
    # keys of the row that has most, as a program that sizes its buffers has it
    s["span"] = max([p - f + 1 for p, f in zip(rows, first) if f is not None])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"plan": _plan, "append": _append, "attend": _attend}[c["op"]](c, state)


def _own(c, s):
    from rq_transformer_frame_gb300 import paged

    if c["op"] == "plan":
        p = paged.paged_plan(s["new_lens"], s["lens"], s["pool"], s["free_ids"], s["table"],
                             block_size=c["block"], max_tokens=c["tokens"], out=s["maps"])
        return {"table": s["table"], "free_ids": s["free_ids"], "lens": p.lens, "pool": p.pool,
                "cu_tokens": p.cu_tokens, "requests": p.requests, "positions": p.positions,
                "slots": p.slots}
    if c["op"] == "append":
        q = paged.paged_append(s["qkv"], s["pool_k"], s["pool_v"], s["positions"], s["slots"],
                               q_alpha=s["q_alpha"], k_alpha=s["k_alpha"], eps=1e-6,
                               rope=c["rope"], rope_dim=c["rope_dim"], rope_theta=10000.0,
                               out=s["out"])
        return {"q": q, "k": s["pool_k"], "v": s["pool_v"]}
    out, lse = paged.paged_attention(s["q"], s["k"], s["v"], s["table"], s["positions"],
                                     requests=s["requests"], window=c["window"], out=s["out"],
                                     lse=s["lse"])
    return {"out": out, "lse": lse}


def _pages(x, c):
    return ((x + c["block"] - 1) // c["block"]).clamp(max=c["columns"])


def _plan(c, s):
    W, P, M = c["columns"], c["block"], c["tokens"]
    table, ids = s["table"], s["free_ids"]
    N = ids.shape[0]
    new, held = s["new_lens"].long(), s["lens"].long()
    head, count = s["pool"][0].long(), s["pool"][1].long()
    ended, add = new < 0, new.clamp(min=0)
    lens = torch.where(ended, 0, held + add)
    before, after = _pages(held, c), _pages(lens, c)
    need = torch.where(ended, 0, after - before)
    back = torch.where(ended, before, 0)
    taken, given, ends = need.cumsum(0), back.cumsum(0), add.cumsum(0)
    status = ((new < -1) | (held < 0) | (lens > 2**31 - 1)).any() | (head < 0) | (head >= N) \
        | (count < 0) | (count + given[-1] > N)
    status = status.long() + 2 * (ends[-1] > M) + 4 * (taken[-1] > count)
    ok = status == 0
    # returned blocks stand behind the free ones, then new pages take the ring's first blocks
    col = torch.arange(W, device=table.device)
    i = torch.arange(N, device=table.device)
    o = (i - head - count) % N
    b = torch.searchsorted(given, o, right=True).clamp(max=new.shape[0] - 1)
    returned = table[b, (o - (given[b] - back[b])).clamp(0, W - 1)]
    grown = ok & ~ended[:, None] & (col >= before[:, None]) & (col < after[:, None])
    block = ids[(head + (taken - need - before)[:, None] + col) % N]
    table.copy_(torch.where(grown, block, table))
    ids.copy_(torch.where(ok & (o < given[-1]), returned, ids))
    # the tokens
    t = torch.arange(M, device=table.device)
    b = torch.searchsorted(ends, t, right=True)
    live = ok & (b < new.shape[0])
    b = b.clamp(max=new.shape[0] - 1)
    pos = held[b] + t - (ends[b] - add[b])
    page = pos // P
    block = table[b, page % W].long()
    kept = live & (page > (lens[b] - 1) // P - W) & (block >= 0) & (block < N)
    minus = torch.full_like(t, -1)
    pool = torch.stack([(head + taken[-1]) % N, count - taken[-1] + given[-1], status, taken[-1]])
    kept_pool = torch.stack([head, count, status, taken[-1]])
    return {"table": table, "free_ids": ids, "lens": torch.where(ok, lens, held).int(),
            "pool": torch.where(ok, pool, kept_pool).int(),
            "cu_tokens": torch.cat([torch.zeros_like(ends[:1]), torch.where(ok, ends, 0)]).int(),
            "requests": torch.where(live, b, minus).int(),
            "positions": torch.where(live, pos, minus).int(),
            "slots": torch.where(kept, block * P + pos % P, minus)}


def _normed(x, alpha):
    if alpha is None:
        return x
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * alpha


def _rotated(x, positions, c):
    rd = c["rope_dim"]
    if not rd:
        return x
    i = torch.arange(rd // 2, device=x.device, dtype=torch.float64)
    angle = positions.double()[:, None] * 10000.0 ** (-2 * i / rd)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turned, rest = x[..., :rd], x[..., rd:]
    if c["rope"] == "interleaved":
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :rd // 2], turned[..., rd // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _append(c, s):
    T, H, Hk, hd = c["rows"], c["heads"], c["kv_heads"], c["head_dim"]
    x = s["qkv"].float().view(T, H + 2 * Hk, hd)
    q = _rotated(_normed(x[:, :H], s["q_alpha"]), s["positions"], c)
    k = _rotated(_normed(x[:, H:H + Hk], s["k_alpha"]), s["positions"], c)
    live = s["positions"] >= 0
    s["out"].copy_(torch.where(live[:, None], q.reshape(T, -1), s["out"].float()))
    cache_k, cache_v = s["k"], s["v"]
    spare = (cache_k.shape[0] - 1) * c["block"]  # the block past the pool's
    slot = torch.where(live & (s["slots"] >= 0), s["slots"], spare)
    cache_k.view(-1, Hk, hd)[slot] = k.to(cache_k.dtype)
    cache_v.view(-1, Hk, hd)[slot] = x[:, H + Hk:].to(cache_v.dtype)
    return {"q": s["out"], "k": s["pool_k"], "v": s["pool_v"]}


def _attend(c, s):
    R, H, Hk, hd, P, W = c["rows"], c["heads"], c["kv_heads"], c["head_dim"], c["block"], c["columns"]
    pos, req = s["positions"].long()[:, None], s["requests"].long()[:, None]
    lo = torch.maximum((pos + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(pos),
                       (pos.clamp(min=0) // P - W + 1) * P)
    j = lo + torch.arange(s["span"], device=pos.device)
    block = s["table"][req.clamp(min=0), (j // P) % W].long()
    live = (j <= pos) & (block >= 0) & (block < s["k"].shape[0])
    at = block.clamp(0, s["k"].shape[0] - 1) * P + j % P
    k = s["k"].view(-1, Hk, hd)[at].float().permute(0, 2, 3, 1)
    score = s["q"].float().view(R, Hk, H // Hk, hd) @ k * (1.0 / math.sqrt(hd))
    score = torch.where(live[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], s["v"].view(-1, Hk, hd)[at], 0).float().permute(0, 2, 1, 3)
    o = torch.where(total > 0, p @ v / total.clamp(min=1e-30), 0)
    kept = req >= 0
    s["out"].copy_(torch.where(kept, o.reshape(R, -1), s["out"].float()))
    s["lse"].copy_(torch.where(kept, (top + total.log()).reshape(R, H), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "plan":
        held, new = _plan_lens(c)
        P, W = c["block"], c["columns"]
        moved = sum(min(-(-h // P), W) if n < 0 else min(-(-(h + n) // P), W) - min(-(-h // P), W)
                    for h, n in zip(held, new))
        # lengths in and out, prefix sums, blocks moved, request, position and slot of each token
        return {"bytes": 16 * c["batch"] + 8 * moved + 16 * c["tokens"], "flops": 0}
    hd, Hk, H = c["head_dim"], c["kv_heads"], c["heads"]
    if c["op"] == "append":
        n = c["rows"] - c["pad"]
        row = (H + 2 * Hk) * hd * SIZE[c["io"]] + H * hd * SIZE[c["out"]] + 2 * Hk * hd * SIZE[c["cache"]]
        return {"bytes": n * (row + 12), "flops": n * (H + Hk) * hd * 8}
    rows = [p for p in _attend_positions(c) if p is not None]
    keys = sum(p - _first_key(c, p) + 1 for p in rows if p >= 0)
    return {"bytes": keys * Hk * hd * 2 * SIZE[c["cache"]] + 4 * (keys // c["block"])
            + len(rows) * (2 * H * hd * SIZE[c["io"]] + 4 * H + 8),
            "flops": 4 * keys * H * hd}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return None  # whole numbers
    hd, Hk, H, P = c["head_dim"], c["kv_heads"], c["heads"], c["block"]
    if c["op"] == "append":
        n = c["rows"] - c["pad"]
        pos = torch.tensor(_append_positions(c)[:n], dtype=torch.float64, device="cuda")
        x = s["qkv"][:n].double()
        parts = []
        for first, count, alpha in ((0, H, s["q_alpha"]), (H, Hk, s["k_alpha"])):
            y = x[:, first * hd:(first + count) * hd].reshape(n, count, hd)
            if alpha is not None:
                y = y / ((y * y).sum(-1, keepdim=True) / hd + 1e-6).sqrt() * alpha.double()
            z = y.clone()
            for i in range(c["rope_dim"] // 2):
                a, b = (2 * i, 2 * i + 1) if c["rope"] == "interleaved" else (i, i + c["rope_dim"] // 2)
                w = pos * math.exp(-2 * i / c["rope_dim"] * math.log(10000.0))
                z[..., a] = y[..., a] * w.cos()[:, None] - y[..., b] * w.sin()[:, None]
                z[..., b] = y[..., b] * w.cos()[:, None] + y[..., a] * w.sin()[:, None]
            parts.append(z)
        out = s["out"].double()
        out[:n] = parts[0].reshape(n, -1)
        k, v = s["pool_k"].double(), s["pool_v"].double()
        block, at = s["slots"][:n] // P, s["slots"][:n] % P
        k[block, at] = parts[1]
        v[block, at] = x[:, (H + Hk) * hd:].reshape(n, Hk, hd)
        return {"q": out, "k": k, "v": v}
    out, lse = s["out"].double(), s["lse"].double()
    table = s["table"].cpu()
    for r, p in enumerate(_attend_positions(c)):
        if p is None:
            continue
        out[r], lse[r] = 0, -math.inf
        if p < 0:
            continue
        j = torch.arange(_first_key(c, p), p + 1)
        block = table[r][(j // P) % c["columns"]].long().cuda()
        k, v = s["k"][block, (j % P).cuda()].double(), s["v"][block, (j % P).cuda()].double()
        q = s["q"][r].double().reshape(Hk, H // Hk, hd)
        score = torch.einsum("hgd,jhd->hgj", q, k) / math.sqrt(hd)
        lse[r] = torch.logsumexp(score, -1).reshape(-1)
        out[r] = torch.einsum("hgj,jhd->hgd", torch.softmax(score, -1), v).reshape(-1)
    return {"out": out, "lse": lse}
