"""The paged K/V cache on the GPU against the plain implementations of paged_ref.py.

Tolerances, with u = 2^-24 (half an f32 step) and e = half a step of the output's type:
- append: norm and rotation are a handful of f32 operations on each element. The mean of
  squares, the reciprocal square root and two products are within 16 u of y; cos and sin
  within 8 u absolute (the angle in half turns is rounded to f32 once, pi u, the functions
  are within 2 steps); so a rotated value is within 32 u of |(a, b)|, the length of its pair, and
  its store adds e |y|.
- attend: a score's f32 sum over head_dim products strays by about sqrt(hd) steps of its
  terms; with S = scale |q| max|k| four times that is ds = u (8 sqrt(hd) S + 8 |s|max) (the
  tensor cores may cut a sum where f32 rounds it, so a step counts for two). Weights stray
  by 2 ds, their sums over n keys by 4 sqrt(n) + 16 u, and bf16 queries' weights keep 16 bits
  (2^-17): each times sum p |v|. The store adds e |o|."""
import math
import os
import random
import subprocess
import sys
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import paged_ref
from rq_transformer_frame_gb300 import binding, paged

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ---------------------------------------------------------------- plan
def check_plan(new, lens, pool, ids, table, P, M, alias):
    want = paged_ref.plan(new, lens, pool, ids, table, P, M)
    d = dict(lens=ints(lens), pool=ints(pool), ids=ints(ids), table=ints(table))
    B = len(lens)
    e = lambda n, dt=torch.int32: torch.full((n,), 77, dtype=dt, device="cuda")  # noqa: E731
    out = paged.PagedPlan(d["lens"] if alias else e(B), d["pool"] if alias else e(4), e(B + 1), e(M),
                          e(M), e(M, torch.int64))
    got = paged.paged_plan(ints(new), d["lens"], d["pool"], d["ids"], d["table"], P, M, out=out)
    pairs = [("lens", got.lens), ("cu", got.cu_tokens), ("req", got.requests), ("pos", got.positions),
             ("slot", got.slots), ("table", d["table"]), ("free_ids", d["ids"])]
    for name, x in pairs:
        np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=name)
    w = want["pool"]
    g = got.pool.tolist()
    assert g[:3] == w[:3], (g, w)
    if w[2] in (0, 4):
        assert g[3] == w[3]
    if not alias:
        assert d["lens"].tolist() == list(lens) and d["pool"].tolist() == list(pool)
    return want


@pytest.mark.parametrize("B,W,P,N,M,alias", [
    (1, 1, 1, 1, 1, True), (1, 3, 16, 8, 40, False), (5, 2, 4, 40, 64, True), (33, 9, 5, 400, 257, True),
    (300, 12, 16, 2000, 1023, False), (1025, 4, 3, 6000, 2048, True), (2500, 3, 7, 9000, 4099, False),
    (8192, 2, 16, 20000, 30000, True),
])
def test_plan_steps(B, W, P, N, M, alias):
    """Twelve steps in a row of arrivals, growth past the table's width, and ends."""
    r = random.Random(B * 31 + W)
    lens, pool = [0] * B, [0, N, 0, 0]
    table, ids = np.full((B, W), -1, np.int32), np.random.RandomState(B).permutation(N).astype(np.int32)
    for step in range(12):
        new = [r.choice([0, 1, 1, 1, -1 if step else 0, 2]) for _ in range(B)]
        for _ in range(3):
            new[r.randrange(B)] = r.randint(0, max(1, M // 5))
        o = check_plan(new, lens, pool, ids, table, P, M, alias)
        lens, pool, table, ids = o["lens"].tolist(), o["pool"], o["table"], o["free_ids"]


@pytest.mark.parametrize("what,status", [
    ("tokens", 2), ("blocks", 4), ("both", 6), ("new", 1), ("held", 1), ("sum", 1), ("head", 1),
    ("count", 1), ("give", 1)])
def test_plan_refuses_on_the_device(what, status):
    """A step that cannot be done changes nothing and says why."""
    B, W, P, N, M = 7, 6, 4, 30, 20
    new, lens = [1, 0, 3, -1, 1, 1, 2], [4, 0, 8, 9, 1, 0, 23]
    pages = [min(-(-c // P), W) for c in lens]
    order = np.random.RandomState(5).permutation(N)
    table, at = np.full((B, W), -1, np.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    pool, ids = [3, N - at, 0, 0], np.full(N, -1, np.int32)
    for i in range(N - at):
        ids[(3 + i) % N] = order[at + i]
    if what in ("tokens", "both"):
        M = 7  # of 8 tokens
    if what in ("blocks", "both"):
        pool[1] = 2  # of 3 new pages
    if what == "new":
        new[2] = -2
    if what == "held":
        lens[1] = -1
    if what == "sum":
        lens[1], new[1] = 2**31 - 3, 5
    if what == "head":
        pool[0] = N
    if what == "count":
        pool[1] = N + 1
    if what == "give":
        pool[1] = N - 1
    o = check_plan(new, lens, pool, ids, table, P, M, alias=False)
    assert o["pool"][2] & status == status


def test_plan_long_prompts():
    """Prompts longer than the table: only the pages that stay get slots."""
    W, P, N, M = 5, 16, 64, 70000
    o = check_plan([65537, 3, 81, 80], [17, 0, 0, 0], [60, 60, 0, 0],
                   np.r_[np.arange(56), [-1] * 4, np.arange(56, 60)].astype(np.int32),
                   np.array([[61, 62, -1, -1, -1]] + [[-1] * 5] * 3, np.int32), P, M, alias=True)
    assert o["pool"][2] == 0 and (o["slot"] >= 0).sum() > 0


def test_plan_maps_at_any_address():
    """Maps that start at any element: no wide stores there, and nothing around them."""
    B, W, P, N, M = 3, 4, 4, 20, 4103
    lens, new = ints([3, 0, 9]), ints([5, 7, 1])
    table, ids = torch.full((B, W), -1, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32).cuda()
    pool = ints([6, 14, 0, 0])
    table[0, 0], table[2, :3] = 0, ints([1, 2, 3])
    for m in (M, 37):
        req, pos = (torch.full((m + 2,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        slot = torch.full((m + 2,), 77, dtype=torch.int64, device="cuda")
        out = paged.PagedPlan(torch.empty_like(lens), torch.empty_like(pool), torch.empty(B + 1).int().cuda(),
                              req[1:-1], pos[1:-1], slot[1:-1])
        paged.paged_plan(new, lens, pool, ids, table.clone(), P, m, out=out)
        want = paged_ref.plan(new.tolist(), lens.tolist(), pool.tolist(), ids.cpu().numpy(), table.cpu().numpy(), P, m)
        for got, w in ((req, want["req"]), (pos, want["pos"]), (slot, want["slot"])):
            np.testing.assert_array_equal(got[1:-1].cpu().numpy(), w)
            assert got[0] == 77 and got[-1] == 77


def test_plan_far_lengths():
    """Lengths up to 2^31 - 1: tables that have wrapped many times."""
    table = np.array([[3, 1, 2], [4, 0, 5]], np.int32)
    ids = np.array([6, 7, -1, -1, -1, -1, -1, -1], np.int32)
    for P in (1, 5, 16):
        o = check_plan([4, 1], [2**31 - 5, 2**31 - 2], [0, 2, 0, 0], ids, table, P, 8, alias=False)
        assert o["pool"][2] == 0 and o["pos"][3] == 2**31 - 2 and (o["slot"][2:5] >= 0).all()
        assert check_plan([5, 1], [2**31 - 5, 0], [0, 2, 0, 0], ids, table, P, 8, alias=True)["pool"][2] == 1


def test_plan_leaves_bad_blocks_out():
    """A table or ring that holds ids outside the pool gives slots of -1, not addresses."""
    table = np.array([[1000000, 2], [3, -7]], np.int32)
    check_plan([1, 1], [3, 7], [0, 2, 0, 0], np.array([4, 5, 0, 0, 0, 0], np.int32), table, 4, 8, alias=False)
    check_plan([6, 1], [3, 7], [0, 2, 0, 0], np.array([99, -5, 0, 0, 0, 0], np.int32), table, 4, 8, alias=True)


# ---------------------------------------------------------------- append
def run_append(T, heads, hk, hd, io, qdt, cache, style, rd, norm, P, theta=10000.0, pad=0, seed=0,
               positions=None, strided=False, hnd=False):
    g = torch.Generator().manual_seed(seed)
    width = (heads + 2 * hk) * hd
    qkv = (torch.randn(T, width, generator=g) * 2).to(io)
    if T > 2:
        qkv[1] = 0  # a row of zeros: the norm divides by sqrt(eps)
        qkv[2] *= 1e-3
    N = T // P + 3
    slots = torch.randperm(N * P, generator=g)[:T].clone()
    pos = positions or [int(x) for x in torch.randint(0, 5000, (T,), generator=g)]
    pos = [-1 if t >= T - pad else p for t, p in enumerate(pos)]
    if T - pad > 4:
        slots[3] = -1        # a token whose page was taken over
        slots[4] = N * P     # past the pool
    alphas = [1 + 0.3 * torch.randn(hd, generator=g) for _ in range(2)] if norm else [None, None]
    shape = (N, hk, P, hd) if hnd else (N, P, hk, hd)
    k0, v0 = (torch.randn(*shape, generator=g).to(cache) for _ in range(2))
    k, v = k0.cuda(), v0.cuda()
    if hnd:
        k, v, k0, v0 = (x.permute(0, 2, 1, 3) for x in (k, v, k0, v0))
    dev = qkv.cuda()
    if strided:
        dev = torch.full((T, width + 64), float("nan"), dtype=io, device="cuda")[:, :width].copy_(dev)
    out = torch.full((T, heads * hd), 3.0, dtype=qdt, device="cuda")
    paged.paged_append(dev, k, v, ints(pos), slots.cuda(), *(a.cuda() if norm else None for a in alphas),
                       eps=1e-6, rope=style, rope_dim=rd, rope_theta=theta, out=out)
    want_k, want_v = k0.double(), v0.double()
    tol_k = torch.zeros_like(want_k)
    got = out.cpu().double().reshape(T, heads, hd)
    for t in range(T):
        if pos[t] < 0:
            assert (got[t] == 3.0).all()
            continue
        q_, k_, v_ = paged_ref.append_row(qkv[t], pos[t], heads, hk, hd, *alphas, 1e-6, style, rd, theta)

        def tol(y, dtype):
            pair = y.abs().clone()
            for i in range(rd // 2):
                a, b = (2 * i, 2 * i + 1) if style == "interleaved" else (i, i + rd // 2)
                pair[:, a] = pair[:, b] = torch.hypot(y[:, a], y[:, b])
            return 32 * U * pair + half_step(dtype) * (y.abs() + 32 * U * pair) + 1e-30
        assert ((got[t] - q_).abs() <= tol(q_, qdt)).all(), (t, float((got[t] - q_).abs().max()))
        s = int(slots[t])
        if 0 <= s < N * P:
            want_k[s // P, s % P], tol_k[s // P, s % P] = k_, tol(k_, cache)
            want_v[s // P, s % P] = v_.to(cache).double() if io == F32 else v_
    err = (k.cpu().double() - want_k).abs()
    assert (err <= tol_k).all(), float((err - tol_k).max())
    np.testing.assert_array_equal(v.cpu().double().numpy(), want_v.numpy())


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("qdt", [F32, BF16])
@pytest.mark.parametrize("cache", [F32, BF16])
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_append_types(io, qdt, cache, hd):
    run_append(7, 6, 2, hd, io, qdt, cache, "interleaved", hd, True, 4, pad=1, seed=hd)


@pytest.mark.parametrize("hd,rd", [(32, 0), (32, 8), (32, 32), (64, 24), (64, 64), (128, 40), (128, 128)])
@pytest.mark.parametrize("style", ["interleaved", "halves"])
@pytest.mark.parametrize("norm", [False, True])
def test_append_rotations(hd, rd, style, norm):
    run_append(5, 3, 1, hd, F32, F32, F32, style, rd, norm, 5, theta=500000.0, seed=rd)


@pytest.mark.parametrize("T,heads,hk,hd", [(1, 1, 1, 32), (1, 32, 32, 128), (2, 40, 8, 128),
                                           (65, 7, 7, 64), (130, 5, 1, 32), (333, 24, 4, 64),
                                           (1300, 3, 1, 32), (2, 130, 20, 128)])
def test_append_sizes(T, heads, hk, hd):
    run_append(T, heads, hk, hd, BF16, BF16, BF16, "halves", hd, True, 16, pad=T // 4, seed=T)


def test_append_layouts():
    """Rows apart by more than their width, and a cache with a block's positions under each
    head."""
    run_append(9, 4, 2, 64, F32, BF16, BF16, "halves", 64, True, 8, strided=True, seed=1)
    run_append(9, 4, 2, 64, BF16, F32, F32, "interleaved", 32, False, 8, hnd=True, strided=True, seed=2)


def test_append_far_positions():
    """The angle loses nothing at far positions (32 bits of a turn)."""
    far = [0, 1, 131071, 2**24 + 1, 2**30 + 12345, 2**31 - 1]
    for style in ("interleaved", "halves"):
        run_append(6, 2, 1, 128, F32, F32, F32, style, 128, False, 4, positions=far, seed=9)


def test_append_norm_and_rotation_are_optional_each():
    """One alpha without the other, and neither: the rows come through unchanged."""
    T, hd = 3, 64
    qkv = torch.randn(T, 4 * hd, device="cuda")
    k, v = (torch.zeros(4, 2, 1, hd, device="cuda") for _ in range(2))
    a = torch.full((hd,), 2.0, device="cuda")
    pos, slots = ints([5, 6, 7]), ints([0, 3, 5], torch.int64)
    q = paged.paged_append(qkv, k, v, pos, slots, rope_dim=0)
    assert torch.equal(q, qkv[:, :2 * hd])
    assert torch.equal(k.view(8, hd)[slots], qkv[:, 2 * hd:3 * hd])
    assert torch.equal(v.view(8, hd)[slots], qkv[:, 3 * hd:])
    q = paged.paged_append(qkv, k, v, pos, slots, q_alpha=a, rope_dim=0, eps=0.0)
    assert torch.equal(k.view(8, hd)[slots], qkv[:, 2 * hd:3 * hd])
    x = qkv[:, :2 * hd].double().view(T, 2, hd)
    want = 2 * x / x.square().mean(-1, keepdim=True).sqrt()
    assert ((q.double().view_as(want) - want).abs() <= 32 * U * want.abs()).all()


def test_append_and_attend_past_32_bits():
    """A cache whose offsets pass 2^32 elements: its last block is written and read."""
    hd, P, stride = 32, 4, 2**31 + 64
    big = torch.zeros(2 * stride + P * hd, dtype=BF16, device="cuda")
    k = big.as_strided((3, P, 1, hd), (stride, hd, hd, 1))
    big_v = torch.zeros_like(big)
    v = big_v.as_strided((3, P, 1, hd), (stride, hd, hd, 1))
    qkv = torch.randn(2, 3 * hd, device="cuda").to(BF16)
    q = paged.paged_append(qkv, k, v, ints([0, 1]), ints([2 * P, 2 * P + 1], torch.int64), rope_dim=0)
    assert torch.equal(big[2 * stride:2 * stride + 2 * hd], qkv[:, hd:2 * hd].reshape(-1))
    assert int((big != 0).sum()) <= 2 * hd
    out, lse = paged.paged_attention(q[:1], k, v, ints([[2]]), ints([1]), lse=True)
    r = paged_ref.attend_row(qkv[0, :hd].double().cpu().view(1, hd), qkv[:, hd:2 * hd].cpu().view(1, 2, 1, hd),
                             qkv[:, 2 * hd:].cpu().view(1, 2, 1, hd), [0], 1, 0, hd ** -0.5)
    assert ((out[0].double().cpu() - r["out"][0]).abs() <= 2.0 ** -8 * r["mass"][0] * 1.1).all()


# ---------------------------------------------------------------- attention
def make_cache(N, P, hk, hd, dtype, g, layout="nhd"):
    if layout == "hnd":
        k, v = (torch.randn(N, hk, P, hd, generator=g).to(dtype) for _ in range(2))
        return (x.permute(0, 2, 1, 3) for x in (k, v))
    if layout == "joint":  # keys and values of a block side by side
        kv = torch.randn(N, 2, P, hk, hd, generator=g).to(dtype)
        return kv[:, 0], kv[:, 1]
    return (torch.randn(N, P, hk, hd, generator=g).to(dtype) for _ in range(2))


def to_gpu(x):
    """The tensor on the GPU with the strides it has here."""
    base = x._base if x._base is not None else x
    return base.cuda().as_strided(x.shape, x.stride(), x.storage_offset())


def check_rows(out, lse, q, k, v, table, requests, positions, window, scale, was_out, was_lse):
    R, heads, hd = q.shape[0], lse.shape[1], k.shape[3]
    e = half_step(q.dtype)
    for r in range(R):
        b = requests[r] if requests is not None else r
        if not 0 <= b < table.shape[0]:
            assert torch.equal(out[r].view(torch.uint8), was_out[r].view(torch.uint8)), r
            assert torch.equal(lse[r], was_lse[r])
            continue
        w = paged_ref.attend_row(q[r].double().view(heads, hd), k, v, table[b].tolist(), positions[r],
                                 window, scale)
        got, l = out[r].double().view(heads, hd), lse[r].double()
        if w["n"] == 0:
            assert (got == 0).all() and (l == -math.inf).all(), r
            continue
        ds = U * (8 * math.sqrt(hd) * w["norm"] + 8 * w["smax"])
        sums = U * (4 * math.sqrt(w["n"]) + 16)
        part = 2.0 ** -17 if q.dtype == BF16 else 0.0
        tol = (2 * ds + sums + part) * w["mass"] * (1 + e) + e * w["out"].abs() + 1e-30
        err = (got - w["out"]).abs()
        assert (err <= tol).all(), (r, positions[r], float((err / tol).max()), float(err.max()))
        assert ((l - w["lse"]).abs() <= ds + sums + 4 * U * w["lse"].abs()).all(), (r, l, w["lse"])


def run_attend(lens, heads, hk, hd, io, cache, P, W=None, window=0, scale=0.0, seed=0, pad=0, layout="nhd",
               poison=True, requests="rows", extra=None):
    """lens: the requests' lengths (position = length - 1)."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    W = W or max(1, -(-max(lens) // P)) + 1
    pages = [min(-(-n // P), W) for n in lens]
    N = sum(pages) + 2
    k, v = make_cache(N, P, hk, hd, cache, g, layout)
    order = torch.randperm(N, generator=g).tolist()
    table, at = torch.full((R, W), -1, dtype=torch.int32), 0
    used = torch.zeros(N, P, dtype=torch.bool)
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
        for j in paged_ref.live_positions(lens[b] - 1, window, W, P):
            used[int(table[b, (j // P) % W]), j % P] = True
    if poison:  # what no row may see: NaN and infinities
        k[~used] = float("nan")
        v[~used] = float("inf")
        v.view(N, P, hk, hd)[~used, :, ::2] = float("nan")
    q = torch.randn(R + pad, heads * hd, generator=g).to(io)
    req = list(range(R)) + [-1, R, 2**30, -2**31][:pad] if pad else None
    pos = [n - 1 for n in lens] + [5] * pad
    out = torch.full((R + pad, heads * hd), float("nan"), dtype=io, device="cuda")
    lse = torch.full((R + pad, heads), float("nan"), device="cuda")
    was_out = torch.randn(R + pad, heads * hd, generator=g).to(io)
    was_lse = torch.randn(R + pad, heads, generator=g)
    out.copy_(was_out), lse.copy_(was_lse)
    ws = paged.paged_attention_workspace(q, k.cuda(), table, window)
    need = 0 if ws is None else ws.numel()
    guarded = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    paged.paged_attention(q.cuda(), to_gpu(k), to_gpu(v), table.cuda(), ints(pos),
                          requests=None if req is None else ints(req), window=window, scale=scale, out=out,
                          lse=lse, workspace=guarded[:need] if need else None)
    assert (guarded[need:] == 0xff).all()
    check_rows(out.cpu(), lse.cpu(), q, k, v, table, req, pos, window, scale or hd ** -0.5, was_out, was_lse)


# A table of many columns, most of them never used: rows that may be long are cut over the card
# instead of being one thread block's (or cluster's) each.
CUT = 6000


EDGES = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("W", [None, CUT])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("cache", [F32, BF16])
def test_attend_lengths(hd, io, cache, W):
    """Empty, one key, and both sides of every tile's edge, in one ragged batch."""
    run_attend(EDGES, 4, 2, hd, io, cache, 16, W=W, pad=3, seed=hd)


@pytest.mark.parametrize("W", [None, CUT])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("n", [1, 16, 17, 300, 2000])
def test_attend_one_row(io, cache, n, W):
    """A single request, over a cluster or over the card."""
    run_attend([n], 6, 2, 64, io, cache, 16, W=W, seed=n)


@pytest.mark.parametrize("heads,hk", [(1, 1), (5, 5), (2, 1), (6, 2), (8, 2), (5, 1), (14, 2), (8, 1), (9, 1),
                                      (12, 1), (16, 1), (34, 2), (40, 1)])
@pytest.mark.parametrize("W", [None, CUT])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_attend_heads(heads, hk, io, cache, W):
    """Queries a K/V head from one to forty."""
    run_attend([0, 1, 40, 77, 130], heads, hk, 64, io, cache, 8, W=W, seed=heads)


@pytest.mark.parametrize("hd", [32, 128])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("W", [None, CUT])
def test_attend_sixteen_heads(hd, io, cache, W):
    run_attend([0, 1, 40, 77, 130], 32, 2, hd, io, cache, 16, W=W, seed=hd)


@pytest.mark.parametrize("P", [1, 3, 5, 8, 24, 32, 100, 128, 1000])
@pytest.mark.parametrize("cache", [F32, BF16])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("W", [None, 20000])
def test_attend_block_sizes(P, cache, hd, W):
    """Blocks smaller and larger than a tile, of sizes that end inside one; with blocks of one
    position a tile's table entries are as many as are read ahead at a time."""
    run_attend([1, 64, 99, 250, 3, 0, 511], 4, 2, hd, F32, cache, P, W=W, seed=P)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 100, 1000])
@pytest.mark.parametrize("rows", [9, 90])
def test_attend_window(window, rows):
    lens = [0, 1, 16, 33, 65, 130, 400, 999, 1500]
    run_attend([lens[i % 9] + i // 9 for i in range(rows)], 4, 4, 64, F32, BF16, 16, window=window, seed=window)


@pytest.mark.parametrize("W,P", [(1, 1), (1, 16), (3, 5), (5, 16), (2, 64)])
@pytest.mark.parametrize("window", [0, 40])
def test_attend_ring_table(W, P, window):
    """Requests longer than their table: the last W pages are live."""
    run_attend([0, 1, 16, 81, 313, 17, 80, 1000] * 20, 4, 2, 64, BF16, BF16, P, W=W, window=window, seed=W)
    run_attend([0, 1, 15, 16, 17, 80, 81, 100, 313, 1000], 4, 2, 32, BF16, BF16, P, W=W, window=window, seed=W)
    run_attend([0, 1, 16, 81, 313], 4, 2, 32, F32, F32, P, W=W, window=window, seed=W)


@pytest.mark.parametrize("layout", ["hnd", "joint"])
@pytest.mark.parametrize("cache", [F32, BF16])
def test_attend_layouts(layout, cache):
    run_attend([0, 1, 40, 130, 77], 8, 2, 64, F32, cache, 16, layout=layout, poison=layout == "nhd", seed=3)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_attend_short_rows(io, cache, hd):
    """Many rows of a few blocks, empty ones among them, first and last: whole units a warp."""
    r = random.Random(hd)
    lens = [0, 0, 0] + [r.choice([0, 0, 1, 2, 5, 16, 17, 31, 40, 63]) for _ in range(400)] + [0, 0]
    run_attend(lens, 4, 2, hd, io, cache, 8, W=8, pad=2, seed=hd)
    run_attend([0] * 300 + [3], 4, 2, hd, io, cache, 8, W=8, seed=hd)


@pytest.mark.parametrize("heads,hk", [(4, 4), (32, 4), (24, 8), (16, 2), (14, 2), (34, 2), (40, 4), (3, 3), (2, 1)])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("W", [None, CUT])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("hd", [32, 64])
def test_attend_heads_side_by_side(heads, hk, io, W, layout, hd):
    """Heads of 32 and 64 dimensions: two neighbours as one unit, or where they do not lie side by
    side, are odd in number or have many queries, one by one."""
    run_attend([0, 1, 40, 77, 130, 300], heads, hk, hd, io, BF16, 16, W=W, layout=layout, poison=layout == "nhd",
               seed=heads)


@pytest.mark.parametrize("scale", [0.5, 3.0, -0.7])
def test_attend_scale(scale):
    """Sharp and negative scales: large scores of both signs."""
    run_attend([1, 40, 200], 4, 2, 64, F32, BF16, 16, scale=scale, seed=4)
    run_attend([1, 40, 200], 4, 2, 64, F32, F32, 16, scale=scale, seed=4)


@pytest.mark.parametrize("io,cache,hd,lens,heads,hk", [
    (F32, BF16, 128, [9000], 2, 1), (BF16, BF16, 64, [20011, 3], 3, 1), (F32, F32, 32, [7001, 0, 513], 4, 2),
    (BF16, BF16, 128, [4097, 1, 0, 2048, 700], 16, 2), (F32, BF16, 64, [12001, 1, 3000], 4, 4),
    (F32, F32, 128, [9001, 0, 40], 2, 2), (BF16, F32, 64, [9001, 0, 40], 8, 1),
    (BF16, BF16, 32, [1, 30011, 3], 12, 1)])
def test_attend_long(io, cache, hd, lens, heads, hk):
    """Rows long enough to be split over many thread blocks."""
    run_attend(lens, heads, hk, hd, io, cache, 16, seed=7, poison=False)
    run_attend(lens, heads, hk, hd, io, cache, 16, W=20000, seed=7, poison=False)


def test_attend_many_rows():
    """More rows than the grid has blocks, most of them short, some empty."""
    r = random.Random(3)
    run_attend([r.choice([0, 1, 3, 17, 40, 90]) for _ in range(700)], 2, 1, 32, BF16, BF16, 8, seed=8, pad=4)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("P", [1, 5, 16])
@pytest.mark.parametrize("rows", [1, 3, 200])
def test_attend_far_positions(io, cache, P, rows):
    """Positions up to 2^31 - 1 over a ring of blocks: nothing in between overflows."""
    far = [2**31 - 1, 2**31 - 2, 2**31 - 17, 2**30 + 3]
    run_attend([far[i % 4] + (1 if i % 4 else 0) for i in range(rows)], 4, 2, 64, io, cache, P, W=33 if P == 1 else 7,
               seed=P)
    run_attend([2**31 - 1 - i for i in range(rows)], 2, 2, 32, io, cache, P, W=70, window=50, seed=P)


@pytest.mark.parametrize("cache", [F32, BF16])
def test_attend_very_many_rows(cache):
    """More rows than threads look at once: one live key each, so its value."""
    R, hd = 70001, 32
    k, v = (torch.randn(50, 4, 1, hd, device="cuda").to(cache) for _ in range(2))
    table = torch.randint(0, 50, (R, 600), device="cuda", dtype=torch.int32)
    pos = torch.randint(-1, 4, (R,), device="cuda", dtype=torch.int32)
    q = torch.randn(R, 2 * hd, device="cuda")
    out, lse = paged.paged_attention(q, k, v, table, pos, window=1, lse=True)
    want = v[table[:, 0].long(), pos.clamp(min=0).long(), 0].float().repeat(1, 2)
    assert torch.equal(out, torch.where(pos[:, None] >= 0, want, 0.0))
    assert torch.equal(lse == -math.inf, (pos < 0)[:, None].expand(R, 2))


def test_attend_one_key_is_its_value():
    """A single live key: its value, exactly."""
    for io, cache in ((F32, BF16), (BF16, BF16), (F32, F32)):
        k, v = (torch.randn(3, 4, 2, 64, device="cuda").to(cache) for _ in range(2))
        q = torch.randn(2, 256, device="cuda").to(io)
        out, _ = paged.paged_attention(q, k, v, ints([[1], [2]]), ints([0, 3]), window=1)
        want = torch.stack([v[1, 0], v[2, 3]]).repeat_interleave(2, dim=1).reshape(2, 256)
        assert torch.equal(out.float(), want.float())


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("columns", [4, CUT])
def test_attend_bad_blocks(io, cache, columns):
    """Blocks outside the pool are left out; a row with no other has no live position."""
    g = torch.Generator().manual_seed(11)
    N, P, hk, hd, heads = 6, 16, 2, 64, 4
    k, v = make_cache(N, P, hk, hd, cache, g)
    table = torch.tensor([[0, -1, 2, 1], [N, 3, 2**31 - 1, -2**31], [-1, -5, N, N + 1], [5, 4, 3, 2]],
                         dtype=torch.int32)
    table = torch.cat([table, torch.full((4, columns - 4), -1, dtype=torch.int32)], 1)
    pos = [63, 60, 50, 37]
    q = torch.randn(4, heads * hd, generator=g).to(io)
    lse = torch.zeros(4, heads, device="cuda")
    out, _ = paged.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ints(pos), lse=lse)
    check_rows(out.cpu(), lse.cpu(), q, k, v, table, None, pos, 0, hd ** -0.5, None, None)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_attend_rows_of_one_request(io, cache):
    """A prompt's tokens as rows of their request, each over its own prefix, twice the same."""
    g = torch.Generator().manual_seed(12)
    N, P, hk, hd, heads, n = 9, 16, 1, 32, 3, 130
    k, v = make_cache(N, P, hk, hd, cache, g)
    table = torch.arange(N, dtype=torch.int32).flip(0).reshape(1, N)
    q = torch.randn(n, heads * hd, generator=g).to(io)
    args = (q.cuda(), k.cuda(), v.cuda(), table.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    req = torch.zeros(n, dtype=torch.int32, device="cuda")
    out, lse = paged.paged_attention(*args, requests=req, lse=True)
    again, lse2 = paged.paged_attention(*args, requests=req, lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    check_rows(out.cpu(), lse.cpu(), q, k, v, table, [0] * n, list(range(n)), 0, hd ** -0.5, None, None)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_attend_infinite_scores(io, cache):
    """A key that scores -inf has no weight; a row of nothing else is empty."""
    hd = 32
    k = torch.ones(2, 4, 1, hd)
    k[0, 1] = k[1] = -math.inf
    k[0, 2] = -torch.finfo(torch.float32).max / 2 if cache == F32 else -1e38
    v = torch.randn(2, 4, 1, hd)
    q = torch.zeros(2, hd)
    q[:, 0] = 1.0
    k[..., 1:] = 0
    out, lse = paged.paged_attention(q.to(io).cuda(), k.to(cache).cuda(), v.to(cache).cuda(), ints([[0], [1]]),
                                     ints([2, 3]), scale=1.0, lse=True)
    assert torch.equal(out[0].float().cpu(), v.to(cache).to(io)[0, 0, 0].float())
    assert (out[1] == 0).all() and lse.tolist() == [[1.0], [-math.inf]]


def test_streams_and_graphs():
    """On a stream of their own, and captured: a graph replayed on new inputs gives what a
    direct call gives, also while another stream runs its own call."""
    g = torch.Generator().manual_seed(13)
    N, P, hk, hd, heads, R = 200, 16, 4, 64, 8, 6
    k, v = (x.cuda() for x in make_cache(N, P, hk, hd, BF16, g))
    table = torch.randperm(N, generator=g)[:180].view(R, 30).int().cuda()
    q = torch.randn(R, heads * hd, generator=g).cuda()
    pos = ints([479, 3, -1, 100, 250, 0])
    want, want_lse = paged.paged_attention(q, k, v, table, pos, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):  # calls of both streams at once, each with scratch of its own
        outs.append(paged.paged_attention(q, k, v, table, pos, lse=True))
        outs.append(paged.paged_attention(q, k, v, table, pos, lse=True, stream=side))
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    out, lse = torch.empty_like(q), torch.empty(R, heads, device="cuda")
    ws = paged.paged_attention_workspace(q, k, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged.paged_attention(q, k, v, table, pos, out=out, lse=lse, workspace=ws)
    for step in range(3):
        q.copy_(torch.randn(R, heads * hd, generator=g))
        pos.copy_(ints([(7 * step + 53 * r) % 480 - 1 for r in range(R)]))
        graph.replay()
        want, want_lse = paged.paged_attention(q, k, v, table, pos, lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_graphs_share_a_workspace():
    """Graphs of different shapes over one workspace, replayed in turn: each finds what it
    needs whatever the other left there."""
    g = torch.Generator().manual_seed(14)
    N, P, hd = 400, 16, 64
    graphs = []
    ws = None
    for heads, hk, lens in ((8, 4, [900, 3, 2500, 40]), (32, 2, [1, 2700, 0, 600, 1800])):
        k, v = (x.cuda() for x in make_cache(N, P, hk, hd, BF16, g))
        table = torch.stack([torch.randperm(N, generator=g)[:200] for _ in lens]).int().cuda()
        table = torch.cat([table, torch.full((len(lens), CUT), -1, dtype=torch.int32, device="cuda")], 1)
        q = torch.randn(len(lens), heads * hd, generator=g).cuda()
        graphs.append([q, k, v, table, ints([n - 1 for n in lens])])
        need = paged.paged_attention_workspace(q, k, table)
        ws = need if ws is None or need.numel() > ws.numel() else ws
    want = [paged.paged_attention(*a, lse=True) for a in graphs]
    captured = []
    for a in graphs:
        out, lse = torch.empty_like(a[0]), torch.empty(a[0].shape[0], a[0].shape[1] // hd, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            paged.paged_attention(*a, out=out, lse=lse, workspace=ws)
        captured.append((graph, out, lse))
    ws.fill_(0xff)
    for _ in range(3):
        for (graph, out, lse), (o, l) in zip(captured, want):
            out.zero_(), lse.zero_()
            graph.replay()
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_python_refusals():
    """What the binding refuses before the library is called, and what the library refuses."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros(4, 16, 2, 64, device="cuda")
    q, table = torch.zeros(3, 256, device="cuda"), i(3, 4)
    bad = [
        dict(q=q.half()), dict(q=q[:, :100]), dict(q=q.t()), dict(k=k.half(), v=k.half()), dict(v=k.bfloat16()),
        dict(v=k[:2]), dict(k=k[..., :32], v=k[..., :32].contiguous()), dict(k=k.permute(0, 1, 3, 2)),
        dict(block_table=table.long()), dict(block_table=table.t()), dict(positions=i(2)),
        dict(positions=i(3).long()), dict(positions=i(3).cpu()), dict(requests=i(2)), dict(out=q.bfloat16()),
        dict(out=q[:2]), dict(lse=torch.zeros(3, 3, device="cuda")), dict(lse=torch.zeros(3, 4)),
        dict(workspace=torch.zeros(8, dtype=torch.uint8)),
    ]
    ok = dict(q=q, k=k, v=k, block_table=table, positions=i(3))
    for b in bad:
        with pytest.raises(ValueError):
            paged.paged_attention(**{**ok, **b})
    for b in (dict(window=-1), dict(scale=float("inf")), dict(block_table=i(2, 4)), dict(q=torch.zeros(3, 192, device="cuda"))):
        with pytest.raises(binding.RQError):
            paged.paged_attention(**{**ok, **b})
    out, lse = paged.paged_attention(**ok)
    assert lse is None and out.shape == q.shape
    qkv, slots = torch.zeros(3, 6 * 64, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    ok = dict(qkv=qkv, k=k, v=k.clone(), positions=i(3), slots=slots)
    for b in (dict(qkv=qkv.half()), dict(qkv=qkv[:, :256]), dict(qkv=qkv.t()), dict(slots=i(3)), dict(slots=slots[:2]),
              dict(q_alpha=torch.ones(64)), dict(q_alpha=torch.ones(32, device="cuda")), dict(rope="other"),
              dict(out=torch.zeros(3, 128, device="cuda", dtype=torch.half)), dict(out=torch.zeros(3, 64, device="cuda"))):
        with pytest.raises(ValueError):
            paged.paged_append(**{**ok, **b})
    for b in (dict(rope_dim=12), dict(rope_dim=72), dict(rope_theta=1.0), dict(eps=-1.0)):
        with pytest.raises(binding.RQError):
            paged.paged_append(**{**ok, **b})
    with pytest.raises(ValueError):
        paged.paged_plan(i(3), i(2), i(4), i(8), i(2, 4), 16, 8)
    with pytest.raises(ValueError):
        paged.paged_plan(i(2), i(2), i(3), i(8), i(2, 4), 16, 8)
    with pytest.raises(binding.RQError):
        paged.paged_plan(i(2), i(2), i(4), i(8), i(2, 4), 0, 8)


def test_no_rows():
    k = torch.zeros(4, 16, 2, 64, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = paged.paged_append(torch.zeros(0, 6 * 64, device="cuda"), k, k, none, none.long())
    assert q.shape == (0, 128)
    out, lse = paged.paged_attention(q, k, k, torch.zeros(1, 4, dtype=torch.int32, device="cuda"), none, lse=True)
    assert out.shape == (0, 128) and lse.shape == (0, 2)


def test_prompt_rows_over_a_ring():
    """A prompt longer than the ring, in steps of n tokens: with window + n - 1 positions held,
    every token of a step finds its whole window."""
    g = torch.Generator().manual_seed(31)
    P, W, window, n, hd, heads = 4, 7, 18, 8, 32, 2
    assert (W - 1) * P + 1 >= window + n - 1
    c = paged.PagedCache(1, W, P, W, n, 1, hd, dtype=F32)
    keys, values = [], []
    for step in range(9):
        c.plan(ints([n]))
        qkv = torch.randn(n, (heads + 2) * hd, generator=g)
        q = c.append(0, qkv.cuda(), rope_dim=0)
        out, _ = c.attend(0, q, window=window)
        keys += list(qkv[:, heads * hd:(heads + 1) * hd].double())
        values += list(qkv[:, (heads + 1) * hd:].double())
        for i in range(n):
            p = step * n + i
            k, v = (torch.stack(x[max(0, p - window + 1):p + 1]) for x in (keys, values))
            for h in range(heads):
                w = torch.softmax(k @ qkv[i, h * hd:(h + 1) * hd].double() / math.sqrt(hd), 0) @ v
                got = out[i, h * hd:(h + 1) * hd].double().cpu()
                assert (got - w).abs().max() <= 64 * U * 32, (step, i)
    assert c.status() == (0, 0)


# ---------------------------------------------------------------- all of them, as they are used
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("io,cache,heads,hk,hd,P,W,window", [
    (F32, BF16, 4, 4, 32, 4, 6, 21), (BF16, BF16, 8, 2, 64, 16, 4, 0), (F32, F32, 6, 2, 32, 5, 5, 12)])
def test_decode_steps(captured, io, cache, heads, hk, hd, P, W, window):
    """Requests that arrive with a prompt, grow by a token a step past their ring of blocks,
    end and make room: each step's plan, append and attention (two layers) against a plain
    run that keeps every request's keys and values in a list."""
    g = torch.Generator().manual_seed(21)
    r = random.Random(22)
    B, M, layers, theta = 5, 24, 2, 10000.0
    c = paged.PagedCache(B, B * W, P, W, M, hk, hd, layers=layers, dtype=cache)
    width = (heads + 2 * hk) * hd
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(layers, M, width, dtype=io, device="cuda")
    qa, ka = (1 + 0.1 * torch.randn(hd, generator=g).cuda() for _ in range(2))
    qs = torch.zeros(layers, M, heads * hd, dtype=io, device="cuda")
    outs = torch.full((layers, M, heads * hd), 7.0, dtype=io, device="cuda")
    lses = torch.full((layers, M, heads), 7.0, device="cuda")
    ws = paged.paged_attention_workspace(qs[0], c.k[0], c.block_table, window)

    def step():
        c.plan(new)
        for l in range(layers):
            q = c.append(l, qkv[l], q_alpha=qa, k_alpha=ka, eps=1e-6, rope="halves", rope_theta=theta, out=qs[l])
            c.attend(l, q, window=window, out=outs[l], lse=lses[l], workspace=ws)
    if captured:
        step()  # nothing to add: loads the kernels before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    else:
        run = step
    held = [[] for _ in range(B)]  # per request: per position, per layer (k, v) in 64 bits
    for t in range(26):
        want = [r.choice([1, 1, 1, 0]) if held[b] else r.choice([0, 3, 5]) for b in range(B)]
        if t % 7 == 6:
            want[r.randrange(B)] = -1
        new.copy_(ints(want))
        x = torch.randn(layers, M, width, generator=g).to(io)
        qkv.copy_(x)
        outs.fill_(7.0)
        run()
        status, free = c.status()
        assert status == 0
        tok, rows = 0, []
        for b in range(B):
            if want[b] < 0:
                held[b] = []
            for _ in range(max(want[b], 0)):
                p = len(held[b])
                parts = [paged_ref.append_row(x[l, tok], p, heads, hk, hd, qa.cpu(), ka.cpu(), 1e-6, "halves", hd,
                                              theta) for l in range(layers)]
                held[b].append([(k_.to(cache).double(), v_.to(cache).double()) for _, k_, v_ in parts])
                rows.append((b, p, [q_ for q_, _, _ in parts]))
                tok += 1
        assert c.maps.cu_tokens.tolist()[-1] == tok
        assert free == B * W - sum(min(-(-len(h) // P), W) for h in held)
        got, lse = outs.cpu(), lses.cpu()
        assert (got[:, tok:] == 7.0).all()
        for i, (b, p, q_) in enumerate(rows):
            lo = max(0, p - window + 1 if window else 0, (p // P - W + 1) * P)
            # pages that a later token of the same step took over are gone
            lo = max(lo, ((len(held[b]) - 1) // P - W + 1) * P) if window == 0 else lo
            for l in range(layers):
                kk = torch.stack([held[b][j][l][0] for j in range(lo, p + 1)])
                vv = torch.stack([held[b][j][l][1] for j in range(lo, p + 1)])
                for h in range(heads):
                    s = kk[:, h // (heads // hk)] @ q_[l][h] / math.sqrt(hd)
                    o = torch.softmax(s, 0) @ vv[:, h // (heads // hk)]
                    # queries and keys are rounded to their types first: half a step of each
                    # moves a score by at most (e_q + e_k) |q| |k| scale
                    e = half_step(io) + half_step(cache) + 64 * U
                    S = float(q_[l][h].norm() * kk[:, h // (heads // hk)].norm(dim=-1).max()) / math.sqrt(hd)
                    mass = torch.softmax(s, 0) @ vv[:, h // (heads // hk)].abs()
                    tol = (2 * e * S + 2.0 ** -16) * mass + half_step(io) * o.abs() + 1e-6
                    err = (got[l, i, h * hd:(h + 1) * hd].double() - o).abs()
                    assert (err <= tol).all(), (t, b, p, l, h, float((err / tol).max()))
                    assert abs(float(lse[l, i, h]) - float(torch.logsumexp(s, 0))) <= e * S + 1e-5


# ---------------------------------------------------------------- edges of the calls
def test_plan_batches_around_48_kb():
    """Batches whose sums take more shared memory than a block has without asking, in a process
    that has planned no larger one before."""
    code = ("import sys; sys.path[:0] = %r\n"
            "import numpy as np, test_paged_gpu as t\n"
            "for B in (3023, 3024, 3050, 3071, 3080):\n"
            "    t.check_plan([1] * B, [0] * B, [0, B, 0, 0], np.arange(B, dtype=np.int32),\n"
            "                 np.full((B, 1), -1, np.int32), 16, B, True)\n"
            % [os.path.dirname(os.path.dirname(os.path.abspath(paged.__file__))),
               os.path.dirname(os.path.abspath(paged_ref.__file__))])
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("heads,hk", [(2, 1), (16, 1), (4, 2)])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("W", [None, CUT])
def test_attend_infinite_values(heads, hk, io, cache, hd, W):
    """A live value of +-inf gives +-inf in its dimension, both of them or a NaN give NaN, and
    every other element is as without them."""
    g = torch.Generator().manual_seed(hd + heads)
    P, lens = 16, [1, 40, 300]
    pages = [-(-n // P) for n in lens]
    N = sum(pages)
    k, v = make_cache(N, P, hk, hd, cache, g)
    table, at = torch.full((3, W or max(pages)), -1, dtype=torch.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(at, at + n)
        at += n
        for d, j, x in ((0, 0, math.inf), (5, lens[b] - 1, -math.inf), (hd - 1, lens[b] // 2, math.inf),
                        (9, 0, math.inf), (9, lens[b] - 1, -math.inf), (18, lens[b] // 3, math.nan)):
            v[int(table[b, j // P]), j % P, :, d] = x
    q = torch.randn(3, heads * hd, generator=g).to(io)
    out, lse = paged.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ints([n - 1 for n in lens]), lse=True)
    e = half_step(io)
    for r, n in enumerate(lens):
        w = paged_ref.attend_row(q[r].double().view(heads, hd), k, v, table[r].tolist(), n - 1, 0, hd ** -0.5)
        got, want = out[r].double().cpu().view(heads, hd), w["out"]
        odd = ~torch.isfinite(want)
        assert odd.any() and torch.equal(odd, ~torch.isfinite(got)), r
        np.testing.assert_array_equal(got[odd].numpy(), want[odd].numpy())
        ds = U * (8 * math.sqrt(hd) * w["norm"] + 8 * w["smax"])
        sums = U * (4 * math.sqrt(n) + 16)
        tol = (2 * ds + sums + (2.0 ** -17 if io == BF16 else 0.0)) * w["mass"] * (1 + e) + e * want.abs() + 1e-30
        assert ((got - want).abs() <= tol)[~odd].all(), r
        assert ((lse[r].double().cpu() - w["lse"]).abs() <= ds + sums + 4 * U * w["lse"].abs()).all()


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("hk,W", [(1, None), (4, CUT)])
def test_attend_large_values(io, cache, hd, hk, W):
    """Values near the top of f32's range, and one key late in the row whose weight is 2^9.9 times
    the others': what is summed stays in range where the result does."""
    g = torch.Generator().manual_seed(hd)
    P, heads, n, R = 16, 2 * hk, 300, 100
    N = -(-n // P)
    k = torch.zeros(N, P, hk, hd)
    k[-1, (n - 1) % P, :, 0] = 6.875  # 9.92 in base 2; every other key scores 0
    v = 5e35 * (0.7 + 0.3 * torch.rand(N, P, hk, hd, generator=g))
    k, v = k.to(cache), v.to(cache)
    q = torch.zeros(R, heads * hd).to(io)
    q[:, ::hd] = 1
    table = torch.cat([torch.arange(N), torch.full(((W or N) - N,), -1)]).int().view(1, -1)
    out, lse = paged.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ints([n - 1] * R),
                                     requests=ints([0] * R), scale=1.0, lse=True)
    check_rows(out.cpu(), lse.cpu(), q, k, v, table, [0] * R, [n - 1] * R, 0, 1.0, None, None)


@pytest.mark.parametrize("W,hd", [(CUT, 128), (8, 64)])
def test_attend_padding_behind_costs_no_more_than_in_front(W, hd):
    """Rows of padding behind the last request are not walked one after another."""
    P, hk, heads, live, pad = 16, 2, 4, 300, 30000
    k, v = (torch.randn(live * 4, P, hk, hd, device="cuda").to(BF16) for _ in range(2))
    table = torch.full((live, W), -1, dtype=torch.int32, device="cuda")
    table[:, :4] = torch.arange(live * 4, dtype=torch.int32, device="cuda").view(live, 4)
    q = torch.randn(live + pad, heads * hd, device="cuda").to(BF16)
    out = torch.zeros_like(q)
    ws = paged.paged_attention_workspace(q, k, table)
    times = []
    for front in (True, False):
        req = torch.full((live + pad,), -1, dtype=torch.int32, device="cuda")
        rows = slice(pad, pad + live) if front else slice(0, live)
        req[rows] = torch.arange(live, dtype=torch.int32, device="cuda")
        pos = torch.full_like(req, 63)
        call = lambda: paged.paged_attention(q, k, v, table, pos, requests=req, out=out, workspace=ws)  # noqa: E731
        call()
        best = math.inf
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) / 4)
        times.append(best)
    assert times[1] <= 3 * times[0], times


@pytest.mark.parametrize("W,P,longest", [(2000, 16, 300), (8, 8, 64)])
@pytest.mark.parametrize("cache", [F32, BF16])
def test_attend_gaps_between_rows(W, P, longest, cache):
    """Runs that cross empty rows: fewer and more of them than are looked at together."""
    r = random.Random(5)
    lens = [0] * 40
    for _ in range(60):
        lens += [r.randint(longest // 2, longest)] + [0] * r.choice([0, 1, 2, 30, 31, 32, 33, 63, 64, 65, 130])
    run_attend(lens + [0] * 70, 4, 4, 64, BF16, cache, P, W=W, pad=4, seed=W)


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def exact_turn(pos, theta, i, rd):
    """The angle pos * theta^(-2i/rd) as a fraction of a turn, in [0, 1), in 70 digits."""
    with localcontext() as c:
        c.prec = 70
        return float(pos * (Decimal(theta) ** (Decimal(-2 * i) / rd)) / (2 * PI) % 1)


@pytest.mark.parametrize("theta", [1.001, 2.0, 10000.0, 1000000.0])
@pytest.mark.parametrize("style", ["interleaved", "halves"])
@pytest.mark.parametrize("rd", [8, 24, 128])
def test_append_angles(theta, style, rd):
    """cos and sin of every pair, read off the pair (1, 0), against angles in 70 digits. Half a step
    of the f32 half turns is pi 2^-25 = 1.6 u of angle, the functions are within 2 steps of u, and
    2^-31 of a turn is 0.05 u."""
    far = [0, 1, 4097, 131071, 2**24 + 1, 2**30 + 12345, 2**31 - 1]
    hd, T = 128, 7
    qkv = torch.zeros(T, 3 * hd)
    pairs = [(2 * i, 2 * i + 1) if style == "interleaved" else (i, i + rd // 2) for i in range(rd // 2)]
    qkv[:, [a for a, _ in pairs]] = 1
    k, v = (torch.zeros(T, 1, 1, hd, device="cuda") for _ in range(2))
    q = paged.paged_append(qkv.cuda(), k, v, ints(far), torch.arange(T, device="cuda"), rope=style, rope_dim=rd,
                           rope_theta=theta).double().cpu()
    worst = 0.0
    for t, pos in enumerate(far):
        for i, (a, b) in enumerate(pairs):
            w = 2 * math.pi * exact_turn(pos, theta, i, rd)
            worst = max(worst, abs(float(q[t, a]) - math.cos(w)), abs(float(q[t, b]) - math.sin(w)))
    assert worst <= 4 * U, worst / U


def test_binding_refuses_what_does_not_fit():
    """Sizes that modulo 2^32 are others, and scales that f32 takes for 0: a size is never cut."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros(4, 16, 2, 64, device="cuda")
    q, table, big = torch.zeros(3, 256, device="cuda"), i(3, 4), 2**32
    for kw in (dict(window=big), dict(window=big + 5), dict(window=5 - big), dict(scale=1e-60), dict(scale=-1e-39)):
        with pytest.raises(ValueError):
            paged.paged_attention(q, k, k, table, i(3), **kw)
    for scale in (1e300, 3e38, -3e38):
        with pytest.raises(binding.RQError):
            paged.paged_attention(q, k, k, table, i(3), scale=scale)
    with pytest.raises(ValueError):
        paged.paged_attention_workspace(q, k, table, big)
    for rope_dim in (big, big + 64, 64 - big):
        with pytest.raises(ValueError):
            paged.paged_append(torch.zeros(3, 6 * 64, device="cuda"), k, k, i(3), i(3).long(), rope_dim=rope_dim)
    for block_size, max_tokens in ((big + 16, 8), (16 - big, 8), (16, big + 8), (16, 8 - big)):
        with pytest.raises(ValueError):
            paged.paged_plan(i(2), i(2), i(4), i(8), i(2, 4), block_size, max_tokens)
