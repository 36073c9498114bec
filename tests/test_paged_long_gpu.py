"""Block bounds, page selection, attention over listed pages and behind shared prefixes on the GPU
against the plain implementations of paged_long_ref.py.

Tolerances, with u = 2^-24 (half an f32 step) and e = half a step of the output's type:
- bounds and pages: none, values and whole numbers are equal.
- sparse: as attention over a request's positions. A score's f32 sum over head_dim products
  strays by about sqrt(hd) steps of its terms; with S = scale |q| max|k| four times that is
  ds = u (8 sqrt(hd) S + 8 |s|max) (the tensor cores may cut a sum where f32 rounds it, so a step
  counts for two). Weights stray by 2 ds, their sums over n keys by 4 sqrt(n) + 16 u, and bf16
  queries' weights keep 16 bits, cut or rounded (2^-16): each times sum p |v|. The store adds e |o|.
- prefix: the two parts of that apart, then joined by their lse, each of which strays by ds, its
  sums and 4 u of itself: the weights of the parts by twice that."""
import math

import pytest
import torch

import paged_long_ref as ref
from rq_transformer_frame_gb300 import binding, paged

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def to_gpu(x):
    """The tensor on the GPU with the strides it has here."""
    base = x._base if x._base is not None else x
    return base.cuda().as_strided(x.shape, x.stride(), x.storage_offset())


def make_cache(N, P, hk, hd, dtype, g, layout="nhd"):
    if layout == "hnd":
        k, v = (torch.randn(N, hk, P, hd, generator=g).to(dtype) for _ in range(2))
        return k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    if layout == "joint":  # keys and values of a block side by side
        kv = torch.randn(N, 2, P, hk, hd, generator=g).to(dtype)
        return kv[:, 0], kv[:, 1]
    return tuple(torch.randn(N, P, hk, hd, generator=g).to(dtype) for _ in range(2))


def same(a, b):
    """Equal values, NaN where the other has NaN."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def guarded(need):
    """A workspace of exactly `need` bytes, and what stands behind it."""
    ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")
    return (ws[:need] if need else None), ws[need:]


# ---------------------------------------------------------------- bounds
def run_bounds(runs, hk, hd, P, dtype, layout="nhd", pad=0, seed=0, poke=None):
    """runs: (first position, tokens) of each request."""
    g = torch.Generator().manual_seed(seed)
    pages = [(a + n - 1) // P + 1 for a, n in runs]
    N = sum(pages) + 2
    k, _ = make_cache(N, P, hk, hd, dtype, g, layout)
    order = torch.randperm(N, generator=g).tolist()
    pos, slots, at = [], [], 0
    for (a, n), m in zip(runs, pages):
        for p in range(a, a + n):
            pos.append(p)
            slots.append(order[at + p // P] * P + p % P)
        at += m
    pos, slots = pos + [-1] * pad, slots + [0] * pad
    if poke:
        poke(k, pos, slots)
    old = torch.randn(N, hk, 2, hd, generator=g).to(dtype)
    got = old.cuda()
    assert paged.paged_bounds(to_gpu(k), got, ints(pos), ints(slots, torch.int64)) is got
    want = ref.bounds(k, old, pos, slots)
    assert same(got.cpu(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("P", [1, 5, 16, 33])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
def test_bounds_types(dtype, hd, P, layout):
    run_bounds([(0, 1), (3, 1), (P - 1, 1), (0, 3 * P + 1), (P, 2 * P), (7, 40)], 3, hd, P, dtype, layout, pad=2,
               seed=P)


@pytest.mark.parametrize("hk", [1, 2, 16, 40, 130])
def test_bounds_heads(hk):
    run_bounds([(0, 9), (17, 1)], hk, 128, 8, BF16, seed=hk)
    run_bounds([(0, 9), (17, 1)], hk, 32, 8, F32, seed=hk)


def test_bounds_long_step():
    """More tokens than one wave of thread blocks holds."""
    run_bounds([(i % 7, 1 + (i * 37) % 90) for i in range(700)], 2, 32, 16, BF16, pad=9, seed=3)


def test_bounds_special_values():
    """Infinities are values, NaN stays in its own dimension, and rows behind the last token (of a request
    that had the block before) do not count."""
    def poke(k, pos, slots):
        P = k.shape[1]
        k[slots[0] // P, slots[0] % P, 0, 3] = NAN
        k[slots[1] // P, slots[1] % P, 1, 5] = INF
        k[slots[2] // P, slots[2] % P, 1, 6] = -INF
        k[slots[-1] // P, slots[-1] % P + 1:] = NAN
    for dtype in (F32, BF16):
        run_bounds([(0, 12), (0, 3)], 2, 64, 8, dtype, seed=1, poke=poke)


def test_bounds_skips_what_append_does_not_store():
    def poke(k, pos, slots):
        slots[1] = -1
        slots[4] = k.shape[0] * k.shape[1]
        pos[7] = -1
    run_bounds([(2, 1), (9, 1), (5, 1), (6, 1), (3, 1), (1, 1), (2, 1), (4, 1)], 2, 64, 4, F32, seed=2, poke=poke)


def test_bounds_do_not_depend_on_the_steps():
    """A prompt in one step, in two, and token by token."""
    g = torch.Generator().manual_seed(5)
    P, hk, hd, n = 8, 2, 64, 43
    k, _ = make_cache(9, P, hk, hd, BF16, g)
    k, slots = k.cuda(), torch.arange(n, device="cuda") + P
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    results = []
    for cuts in ([0, n], [0, 19, n], list(range(n + 1))):
        b = torch.zeros(9, hk, 2, hd, dtype=BF16, device="cuda")
        for x, y in zip(cuts, cuts[1:]):
            paged.paged_bounds(k, b, pos[x:y], slots[x:y])
        results.append(b)
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
    paged.paged_bounds(k, results[0], pos[:0], slots[:0])  # no token: nothing is done
    assert torch.equal(results[0], results[1])


# ---------------------------------------------------------------- select
def run_select(lens, heads, hk, hd, io, dtype, P, top, first=1, last=1, W=None, pad=0, seed=0, poke=None):
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    W = W or max(1, -(-max(lens) // P)) + 1
    pages = [min(-(-n // P), W) for n in lens]
    N = sum(pages) + 2
    mid, half = torch.randn(N, hk, 1, hd, generator=g), torch.rand(N, hk, 1, hd, generator=g) + 0.5
    b = torch.cat([mid - half, mid + half], 2).to(dtype)
    order = torch.randperm(N, generator=g).tolist()
    table, at = torch.full((R, W), -1, dtype=torch.int32), 0
    for r, n in enumerate(pages):
        table[r, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    q = torch.randn(R + pad, heads * hd, generator=g).to(io)
    if poke:
        poke(q, b, table)
    req = list(range(R)) + [-1, R, 2**30, -2**31][:pad] if pad else None
    pos = [n - 1 for n in lens] + [5] * pad
    dev = dict(q=q.cuda(), b=b.cuda(), table=table.cuda(), pos=ints(pos), req=None if req is None else ints(req))
    ws, behind = guarded(paged.paged_select_workspace(dev["q"], dev["b"], dev["table"], P).numel())
    out = torch.full((R + pad, hk, top), -7, dtype=torch.int32, device="cuda")
    for _ in range(2):  # whatever the scratch holds
        paged.paged_select(dev["q"], dev["b"], dev["table"], dev["pos"], P, top, first, last, requests=dev["req"],
                           pages=out, workspace=ws)
    assert (behind == 0xff).all()
    got = out.cpu()
    for r in range(R):
        want = ref.select(q[r].double().view(heads, hd), b, table[r].tolist(), pos[r], P, top, first, last)
        for h in range(hk):
            assert got[r, h].tolist() == want[h] + [-1] * (top - len(want[h])), (r, h)
    assert (got[R:] == -7).all()
    return got


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_types(hd, io, dtype):
    run_select([0, 1, 5, 80, 81, 160, 333, 1000, 1999], 6, 2, hd, io, dtype, 5, 17, first=2, last=3, pad=3, seed=hd)


@pytest.mark.parametrize("heads,hk", [(1, 1), (5, 5), (2, 1), (16, 1), (34, 2), (12, 12), (40, 10)])
def test_select_heads(heads, hk):
    run_select([700, 64, 1, 333], heads, hk, 64, BF16, BF16, 4, 11, seed=heads)


@pytest.mark.parametrize("top,first,last", [(1, 0, 1), (2, 1, 1), (5, 0, 5), (6, 0, 1), (7, 3, 4), (60, 1, 1),
                                            (61, 1, 1), (62, 2, 2), (63, 0, 1), (64, 1, 1), (100, 5, 9), (300, 0, 1)])
def test_select_counts(top, first, last):
    """From the row's own page alone to more pages than there are."""
    run_select([62 * 8, 61 * 8 + 1, 61 * 8, 3, 1], 4, 2, 32, F32, BF16, 8, top, first, last, seed=top)


@pytest.mark.parametrize("W", [1, 7, 33])
def test_select_ring(W):
    """Tables that have wrapped: the pages they still hold."""
    run_select([1, 20, 4 * W, 4 * W + 1, 1000, 4321], 4, 2, 64, F32, BF16, 4, max(1, min(W - 1, 9)), 0, 1, W=W, seed=W)
    run_select([1, 20, 1000, 4321], 4, 2, 64, F32, F32, 4, 40, 2, 2, W=W, seed=W)


@pytest.mark.parametrize("P,n", [(1, 9000), (16, 40000), (1, 70001)])
def test_select_many_pages(P, n):
    run_select([n, n // 2 + 1], 2, 1, 32, BF16, BF16, P, 100, seed=P)


def test_select_far_positions():
    """Positions up to 2^31 - 1 in a ring."""
    run_select([2**31 - 1, 2**31 - 2, 2**30 + 5], 2, 1, 64, F32, BF16, 1, 4, 1, 1, W=13, seed=2)
    run_select([2**31 - 1, 2**31 - 2, 2**30 + 5], 2, 1, 64, F32, BF16, 5, 4, 1, 1, W=13, seed=2)


def test_select_leaves_missing_blocks_out():
    def poke(q, b, table):
        table[0, 3], table[0, 8], table[0, 20] = -1, b.shape[0], 2**31 - 1
        table[1, 1:30] = -5  # fewer than are wanted remain
    run_select([40 * 4, 40 * 4, 8 * 4], 4, 2, 64, F32, BF16, 4, 12, 1, 2, seed=4, poke=poke)
    run_select([40 * 4, 40 * 4, 8 * 4], 4, 2, 64, F32, BF16, 4, 50, 1, 2, seed=4, poke=poke)


def test_select_equal_scores():
    """Pages that score alike: the lowest are taken."""
    def all_equal(q, b, table):
        b[:] = b[:1]

    def zeros(q, b, table):
        q[:] = 0

    def in_pairs(q, b, table):
        for r in range(table.shape[0]):
            t = table[r][table[r] >= 0].long()
            b[t[1::2]] = b[t[0::2][:t[1::2].numel()]]

    def small_numbers(q, b, table):
        q[:] = (q * 2).round().clamp(-2, 2)
        b[:] = b.float().round().to(b.dtype)
    for poke in (all_equal, zeros, in_pairs, small_numbers):
        for io, dtype in ((F32, F32), (BF16, BF16)):
            run_select([3000, 777, 129], 6, 2, 64, io, dtype, 2, 41, 1, 2, seed=7, poke=poke)


def test_select_scores_that_f32_orders_wrongly():
    """Scores of about 2000 that differ by 2^-20: far below an f32 step, decided in 64 bits."""
    def poke(q, b, table):
        q[:] = 16.0
        b[:] = 1.0
        g = torch.Generator().manual_seed(1)
        # the last dimension's largest key by a multiple of 2^-24, each page another
        b[:, :, 1, -1] += torch.randperm(b.shape[0], generator=g).float()[:, None] * 2.0 ** -23
    got = run_select([900, 450], 2, 1, 64, F32, F32, 1, 50, 1, 1, seed=8, poke=poke)
    assert (got >= 0).all()


@pytest.mark.parametrize("io,dtype", [(F32, F32), (BF16, BF16)])
def test_select_special_values(io, dtype):
    """Infinities order as such, a NaN score is the lowest."""
    def bounds_(q, b, table):
        t = table[0].long()
        b[t[5], 0, 1, 3] = INF
        b[t[9], 0, 0, 3] = -INF
        b[t[11], 1, :, 7] = NAN
        b[t[20], 0, :, 7] = NAN
        b[t[30], :, 0, :] = -INF

    def queries(q, b, table):
        q[0, 5] = INF
        q[1, 70] = -INF
        q[2, 1] = NAN

    def large(q, b, table):
        b[:] = b * 1e38
        q[:] = q * 1e30

    def tiny(q, b, table):
        b[:] = b * 1e-38
    for poke in (bounds_, queries, large, tiny):
        run_select([200, 160, 120], 4, 2, 64, io, dtype, 4, 13, 1, 1, seed=9, poke=poke)


# ---------------------------------------------------------------- attention over lists
def check_row(got, lse, w, io, joined):
    e = torch.finfo(io).eps / 2
    hd = got.shape[1]
    n = w["n"]
    none = n == 0
    assert (got[none] == 0).all() and (lse[none] == -INF).all()
    ds = U * (8 * math.sqrt(hd) * w["norm"] + 8 * w["smax"])
    sums = U * (4 * n.sqrt() + 16)
    part = 2.0 ** -16 if io == BF16 else 0.0
    own = torch.where(none, 0, w["lse"].abs())
    join = 2 * (ds + sums + 4 * U * (own + w["smax"])) if joined else 0 * ds
    tol = (2 * ds + sums + part + join)[:, None] * w["mass"] * (1 + e) + e * w["out"].abs() + 1e-30
    err = (got - w["out"]).abs()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
    l_err = (lse - w["lse"]).abs()[~none]
    assert (l_err <= (ds + sums + join / 2 + 4 * U * own)[~none]).all(), float(l_err.max())


def run_sparse(lens, heads, hk, hd, io, cache, P, top, W=None, scale=0.0, seed=0, pad=0, layout="nhd", lists="some"):
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    W = W or max(1, -(-max(lens) // P)) + 1
    pages = [min(-(-n // P), W) for n in lens]
    N = sum(pages) + 2
    k, v = make_cache(N, P, hk, hd, cache, g, layout)
    order = torch.randperm(N, generator=g).tolist()
    table, at = torch.full((R, W), -1, dtype=torch.int32), 0
    for r, n in enumerate(pages):
        table[r, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    given = torch.full((R + pad, hk, top), -1, dtype=torch.int32)
    seen = torch.zeros(N, P, hk, dtype=torch.bool)
    for r, n in enumerate(lens):
        newest = (n - 1) // P if n else -1
        live = list(range(max(0, newest - W + 1), newest + 1))
        for h in range(hk):
            if lists == "sorted" or not live:
                x = sorted(torch.randperm(len(live), generator=g)[:top].tolist())
                x = [live[i] for i in x]
            else:  # any order, empty entries between, pages that are not there, some twice
                i = torch.randint(0, len(live), (top,), generator=g).tolist()
                x = [live[j] for j in i]
                for j in range(0, top, 5):
                    x[j] = [-1, newest + 1, newest - W, -2**31, 2**31 - 1][(j // 5) % 5]
            given[r, h, :len(x)] = torch.tensor(x, dtype=torch.int32)
            for p in x:
                if 0 <= p <= newest and p > newest - W:
                    seen[int(table[r, p % W]), :min(P, n - p * P), h] = True
    k[~seen], v[~seen] = NAN, INF  # what no row may see
    q = torch.randn(R + pad, heads * hd, generator=g).to(io)
    req = list(range(R)) + [-1, R, 2**30, -2**31][:pad] if pad else None
    pos = [n - 1 for n in lens] + [5] * pad
    was_out, was_lse = torch.randn(R + pad, heads * hd, generator=g).to(io), torch.randn(R + pad, heads, generator=g)
    out, lse = was_out.cuda(), was_lse.cuda()
    kd, vd, qd, gd = to_gpu(k), to_gpu(v), q.cuda(), given.cuda()
    ws = paged.paged_sparse_attention_workspace(qd, kd, gd)
    ws, behind = guarded(0 if ws is None else ws.numel())
    paged.paged_sparse_attention(qd, kd, vd, table.cuda(), ints(pos), gd, requests=None if req is None else ints(req),
                                 scale=scale, out=out, lse=lse, workspace=ws)
    assert (behind == 0xff).all()
    out, lse = out.cpu(), lse.cpu()
    for r in range(R):
        kk, vv = ref.listed_keys(k, v, table[r].tolist(), pos[r], given[r].tolist())
        w = ref.attend_keys(q[r].double().view(heads, hd), kk, vv, scale or hd ** -0.5)
        check_row(out[r].double().view(heads, hd), lse[r].double(), w, io, False)
    assert torch.equal(out[R:], was_out[R:]) and torch.equal(lse[R:], was_lse[R:])


LENS = [0, 1, 2, 15, 16, 17, 33, 64, 100, 129, 300, 1000]


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("cache", [F32, BF16])
@pytest.mark.parametrize("lists", ["sorted", "some"])
def test_sparse_types(hd, io, cache, lists):
    run_sparse(LENS, 4, 2, hd, io, cache, 16, 9, pad=3, seed=hd, lists=lists)


@pytest.mark.parametrize("heads,hk", [(1, 1), (5, 5), (2, 1), (6, 2), (8, 2), (14, 2), (8, 1), (9, 1), (16, 1),
                                      (34, 2), (40, 1)])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_sparse_heads(heads, hk, io, cache):
    run_sparse([0, 1, 40, 77, 130], heads, hk, 64, io, cache, 8, 7, seed=heads)


@pytest.mark.parametrize("P", [1, 3, 5, 8, 24, 32, 100, 128])
@pytest.mark.parametrize("cache", [F32, BF16])
@pytest.mark.parametrize("hd", [32, 128])
def test_sparse_block_sizes(P, cache, hd):
    run_sparse([0, 1, 3 * P + 1, 9 * P, 40 * P + P // 2], 4, 2, hd, F32, cache, P, 13, seed=P)


@pytest.mark.parametrize("top", [1, 2, 31, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("rows", [1, 9, 200])
def test_sparse_list_lengths(top, rows):
    """Lists around the 32 entries that are looked up at a time; few rows, and enough to fill the card."""
    g = torch.Generator().manual_seed(top)
    lens = torch.randint(1, 1500, (rows,), generator=g).tolist()
    run_sparse(lens, 4, 2, 64, BF16, BF16, 4, top, seed=top, lists="sorted")


@pytest.mark.parametrize("rows,heads,hk,P,top", [(1, 8, 2, 16, 500), (40, 32, 8, 16, 40), (150, 4, 4, 32, 20),
                                                 (20, 12, 1, 64, 64)])
@pytest.mark.parametrize("io,cache", [(BF16, BF16), (F32, BF16), (F32, F32)])
def test_sparse_many_positions(rows, heads, hk, P, top, io, cache):
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(1, 12000, (rows,), generator=g).tolist() if rows < 100 else [900] * rows
    run_sparse(lens, heads, hk, 128, io, cache, P, top, seed=rows, lists="sorted")


@pytest.mark.parametrize("layout", ["hnd", "joint"])
def test_sparse_layouts(layout):
    run_sparse(LENS, 6, 3, 64, BF16, BF16, 16, 9, seed=1, layout=layout, pad=2)
    run_sparse(LENS, 6, 3, 64, F32, F32, 16, 9, seed=1, layout=layout, scale=0.3)


def test_sparse_ring_and_far_positions():
    run_sparse([5, 100, 1000, 4321], 4, 2, 64, F32, BF16, 4, 9, W=7, seed=3)
    run_sparse([2**31 - 1, 2**30 + 3], 4, 2, 64, F32, BF16, 4, 9, W=7, seed=3)
    run_sparse([2**31 - 1, 2**30 + 3], 4, 2, 64, BF16, F32, 1, 30, W=21, seed=3)


def test_sparse_missing_blocks():
    """Listed pages whose block is not in the pool are left out; lists of nothing else give 0."""
    k, v = (torch.randn(4, 8, 2, 64, device="cuda") for _ in range(2))
    q = torch.randn(3, 4 * 64, device="cuda")
    table = ints([[0, -1, 4, 1], [9, -1, -3, 2**31 - 1], [2, 3, 0, 1]])
    pages = ints([[[0, 1, 2], [1, 2, 3]], [[0, 1, 2], [0, 1, 3]], [[-1, -1, -1], [0, 3, -1]]])
    pos = ints([31, 31, 26])
    out, lse = paged.paged_sparse_attention(q, k, v, table, pos, pages, lse=True)
    for r in range(3):
        kk, vv = ref.listed_keys(k.cpu(), v.cpu(), table[r].tolist(), int(pos[r]), pages[r].tolist())
        w = ref.attend_keys(q[r].double().cpu().view(4, 64), kk, vv, 0.125)
        check_row(out[r].double().cpu().view(4, 64), lse[r].double().cpu(), w, F32, False)
    assert (out[1] == 0).all() and (out[2, :128] == 0).all()


# ---------------------------------------------------------------- shared prefixes
def run_prefix(sizes, prefix, own, heads, hk, hd, io, cache, P, W=None, scale=0.0, seed=0, pad=0, layout="nhd",
               first=0, poke=None):
    """sizes, prefix: rows and prefix length of each group, after `first` rows of none; own: own length of
    every row."""
    g = torch.Generator().manual_seed(seed)
    R, G = len(own), len(sizes)
    B = R + G
    W = W or max(1, -(-max(own + prefix) // P)) + 1
    pages = [min(-(-n // P), W) for n in own + prefix]
    N = sum(pages) + 2
    k, v = make_cache(N, P, hk, hd, cache, g, layout)
    order = torch.randperm(N, generator=g).tolist()
    table, at = torch.full((B, W), -1, dtype=torch.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cu = [first]
    for n in sizes:
        cu.append(cu[-1] + n)
    preq, plen = [R + i for i in range(G)], list(prefix)
    if poke:
        poke(cu, preq, plen, table)
    group = {}
    for i in range(G):
        for r in range(max(cu[i], 0), min(cu[i + 1], R)):
            group[r] = i
    seen = torch.zeros(N, P, dtype=torch.bool)
    keys = {}
    for r in range(R):
        want = [(r, own[r] - 1)]
        if r in group and 0 <= preq[group[r]] < B and plen[group[r]] > 0:
            want.append((preq[group[r]], plen[group[r]] - 1))
        keys[r] = want
        for b, pos in want:
            for j in range(max(0, (pos // P - W + 1) * P), pos + 1):
                if 0 <= int(table[b, (j // P) % W]) < N:
                    seen[int(table[b, (j // P) % W]), j % P] = True
    k[~seen], v[~seen] = NAN, INF
    q = torch.randn(R + pad, heads * hd, generator=g).to(io)
    req = list(range(R)) + [-1, B, 2**30, -2**31][:pad] if pad else None
    pos = [n - 1 for n in own] + [5] * pad
    was_out, was_lse = torch.randn(R + pad, heads * hd, generator=g).to(io), torch.randn(R + pad, heads, generator=g)
    out, lse = was_out.cuda(), was_lse.cuda()
    kd, vd, qd, td, pl = to_gpu(k), to_gpu(v), q.cuda(), table.cuda(), ints(plen)
    ws, behind = guarded(paged.paged_prefix_attention_workspace(qd, kd, td, pl).numel())
    for _ in range(2):
        paged.paged_prefix_attention(qd, kd, vd, td, ints(pos), ints(cu), ints(preq), pl,
                                     requests=None if req is None else ints(req), scale=scale, out=out, lse=lse,
                                     workspace=ws)
    assert (behind == 0xff).all()
    out, lse = out.cpu(), lse.cpu()
    for r in range(R):
        parts = [ref.request_keys(k, v, table[b].tolist(), p) for b, p in keys[r]]
        kk, vv = (torch.cat(x) for x in zip(*parts))
        w = ref.attend_keys(q[r].double().view(heads, hd), [kk[:, h] for h in range(hk)],
                            [vv[:, h] for h in range(hk)], scale or hd ** -0.5)
        check_row(out[r].double().view(heads, hd), lse[r].double(), w, io, True)
    assert torch.equal(out[R:], was_out[R:]) and torch.equal(lse[R:], was_lse[R:])


OWN = [1, 0, 2, 15, 16, 17, 40, 3, 0, 64, 65, 5, 0, 9]
# A table of many columns, most of them never used: rows that may be long meet their prefix on the tensor cores
# (bf16 caches), short ones each for itself.
CUT = 60000
TABLES = pytest.mark.parametrize("W", [None, CUT])


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("cache", [F32, BF16])
@TABLES
def test_prefix_types(hd, io, cache, W):
    """Groups of several sizes, an empty one, rows before and behind them, and rows that hold nothing."""
    run_prefix([5, 0, 1, 4], [300, 40, 129, 17], OWN, 4, 2, hd, io, cache, 16, W=W, first=2, pad=3, seed=hd)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385, 1000])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@TABLES
def test_prefix_lengths(n, io, cache, W):
    """Both sides of every tile's edge."""
    run_prefix([3], [n], [4, 1, 30], 4, 2, 128, io, cache, 16, W=W, seed=n)


@pytest.mark.parametrize("heads,hk", [(1, 1), (5, 5), (2, 1), (6, 2), (14, 2), (8, 1), (9, 1), (16, 1), (34, 2),
                                      (40, 1)])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@TABLES
def test_prefix_heads(heads, hk, io, cache, W):
    run_prefix([3, 2], [200, 77], [5, 1, 9, 20, 2, 3], heads, hk, 64, io, cache, 8, W=W, seed=heads)


@pytest.mark.parametrize("rows,heads,hk", [(31, 4, 1), (32, 4, 1), (33, 4, 1), (64, 2, 1), (70, 12, 4), (127, 1, 1),
                                           (129, 1, 1), (100, 16, 2), (300, 8, 8)])
@pytest.mark.parametrize("io", [F32, BF16])
@TABLES
def test_prefix_rows(rows, heads, hk, io, W):
    """Groups around the number of queries that read a tile together."""
    own = [1 + (i * 7) % 23 for i in range(rows)]
    run_prefix([rows], [333], own, heads, hk, 64, io, BF16, 16, W=W, seed=rows)
    run_prefix([rows // 3, rows // 3], [130, 500], own, heads, hk, 128, io, BF16, 16, W=W, seed=rows)


@pytest.mark.parametrize("P", [1, 3, 5, 8, 24, 32, 100, 128, 1000])
@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("hd", [32, 64, 128])
@TABLES
def test_prefix_block_sizes(P, io, cache, hd, W):
    run_prefix([3, 2], [2 * P + 1, 700], [P, 1, 9, P + 1, 2], 4, 2, hd, io, cache, P, W=W, seed=P)


@pytest.mark.parametrize("layout", ["hnd", "joint"])
@TABLES
def test_prefix_layouts(layout, W):
    kw = dict(W=W, seed=1, layout=layout)
    run_prefix([5, 4], [300, 40], OWN[:10], 6, 3, 64, BF16, BF16, 16, pad=2, **kw)
    run_prefix([5, 4], [300, 40], OWN[:10], 6, 3, 128, F32, F32, 16, scale=0.3, **kw)
    run_prefix([5, 4], [300, 40], OWN[:10], 6, 3, 32, F32, BF16, 16, scale=-0.2, **kw)
    run_prefix([5, 4], [300, 40], OWN[:10], 6, 3, 128, BF16, BF16, 16, scale=-0.2, **kw)
    run_prefix([5, 4], [300, 40], OWN[:10], 6, 3, 64, BF16, BF16, 5, scale=0.3, **kw)


@pytest.mark.parametrize("scale", [1e-30, 4.0, -4.0, 60.0])
@pytest.mark.parametrize("io", [F32, BF16])
def test_prefix_scales(scale, io):
    """From weights that are all alike to one key's alone: bounds of the scores that rise from tile to tile."""
    run_prefix([9], [2000], [3] * 9, 4, 2, 64, io, BF16, 16, W=CUT, seed=2, scale=scale)
    run_prefix([70], [900], [3] * 70, 8, 2, 128, io, BF16, 16, W=CUT, seed=2, scale=scale)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_prefix_long(io, cache):
    """Prefixes that are cut over the card, of one row and of many."""
    run_prefix([1], [20000], [3], 8, 2, 128, io, cache, 16, seed=1)
    run_prefix([40, 2, 30], [9000, 12000, 700], [1 + i % 9 for i in range(72)], 8, 2, 64, io, cache, 32, seed=2)
    run_prefix([1] * 40, [300 + 7 * i for i in range(40)], [1 + i % 9 for i in range(40)], 4, 2, 64, io, cache, 16, W=CUT,
               seed=3)


def test_prefix_of_a_ring():
    """A prefix longer than its table: the pages that the table still holds."""
    run_prefix([3], [500], [4, 1, 30], 4, 2, 64, BF16, BF16, 16, W=7, seed=3)
    run_prefix([3], [500], [4, 200, 333], 4, 2, 64, F32, F32, 5, W=7, seed=3)
    run_prefix([3], [7000], [4, 200, 333], 8, 8, 128, BF16, BF16, 16, W=300, seed=3)
    run_prefix([3], [7000], [4, 200, 333], 8, 8, 128, F32, BF16, 15, W=330, seed=3)


def test_prefix_words_out_of_range():
    """Groups past the rows, requests that are none, lengths below 1, missing blocks."""
    def poke(cu, preq, plen, table):
        preq[1], plen[2] = -1, 0
        table[preq[0], 2] = -1
        table[preq[0], 5] = 2**31 - 1
        table[0, 0] = -1
    for W in (None, CUT):
        for io, cache in ((F32, BF16), (BF16, BF16), (F32, F32)):
            run_prefix([3, 2, 2, 9], [200, 77, 50, 60], [5, 1, 9, 20, 2, 3, 4, 8, 9], 4, 2, 64, io, cache, 8, W=W, seed=5,
                       poke=poke)
        run_prefix([3], [200], [5, 1, 9], 4, 2, 64, BF16, BF16, 8, W=W, seed=5,
                   poke=lambda cu, preq, plen, table: preq.__setitem__(0, 2**31 - 1))


def test_prefix_shared_by_two_groups_and_own_request():
    """The same request as two groups' prefix, and as a row's own."""
    def poke(cu, preq, plen, table):
        preq[1], plen[1] = preq[0], 90
        preq[2], plen[2] = 4, 12
    for W in (None, CUT):
        run_prefix([2, 2, 2], [200, 200, 77], [5, 1, 9, 20, 30, 3], 4, 2, 64, BF16, BF16, 8, W=W, seed=6, poke=poke)


def test_prefix_no_groups():
    k, v = (torch.randn(6, 8, 2, 64, device="cuda") for _ in range(2))
    q, table, pos = torch.randn(2, 4 * 64, device="cuda"), ints([[0, 1], [2, 3]]), ints([9, 15])
    none = ints([])
    a, al = paged.paged_prefix_attention(q, k, v, table, pos, ints([0]), none, none, lse=True)
    b, bl = paged.paged_attention(q, k, v, table, pos, lse=True)
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-6) and torch.allclose(al, bl, rtol=1e-6)


@pytest.mark.parametrize("io,cache", [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("W", [30, CUT])
def test_prefix_special_values(io, cache, W):
    """An infinite value at a live position reaches its own dimension of the rows that read it; NaN keys
    make those rows NaN and no others."""
    g = torch.Generator().manual_seed(1)
    P, hk, hd, heads = 8, 2, 64, 4
    k, v = make_cache(60, P, hk, hd, cache, g)
    table = torch.full((5, W), -1, dtype=torch.int32)
    table[3, :30], table[4, :20] = torch.arange(30), torch.arange(30, 50)
    for r in range(3):
        table[r, 0] = 50 + r
    v[4, 3, 0, 5], v[33, 1, 1, 7] = INF, -INF
    k[35, 2, 1, 3] = NAN
    q = torch.randn(3, heads * hd, generator=g).to(io)
    out, lse = paged.paged_prefix_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ints([4, 2, 6]), ints([0, 2, 3]),
                                            ints([3, 4]), ints([230, 150]), lse=True)
    out, lse = out.cpu().view(3, heads, hd), lse.cpu()
    bad = torch.zeros(3, heads, hd, dtype=torch.bool)
    bad[:2, :2, 5] = True
    assert (out[:2, :2, 5] == INF).all()
    bad[2, 2:] = True
    assert out[2, 2:].isnan().all() and lse[2, 2:].isnan().all()
    assert out[~bad].isfinite().all()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,io", [(BF16, BF16), (F32, F32)])
def test_steps_of_a_server(dtype, io):
    """Prompts, then tokens one by one: plan, append, bound, select and attend_pages; with every page
    selected the result is attend's."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, P, hk, H, hd, L = 5, 8, 2, 6, 64, 2
    c = paged.PagedCache(B, 400, P, 60, 512, hk, hd, layers=L, dtype=dtype, bounds=True)
    lens = [100, 1, 37, 250, 64]
    for step in range(6):
        new = lens if step == 0 else [1] * B
        c.plan(ints(new))
        T = sum(new)
        for layer in range(L):
            qkv = torch.randn(T, (H + 2 * hk) * hd, generator=g, device="cuda").to(io)
            q = c.append(layer, qkv, rope="halves")
            c.bound(layer, T)
            if step == 0:
                continue
            few = c.select(layer, q, 6, last=2)
            every = c.select(layer, q, 60)
            a, al = c.attend_pages(layer, q, every, lse=True)
            b, bl = c.attend(layer, q, lse=True)
            assert (a.double() - b.double()).abs().max() <= 4 * torch.finfo(io).eps * b.double().abs().max()
            assert torch.allclose(al, bl, rtol=1e-5)
            out, lse = c.attend_pages(layer, q, few, lse=True)
            k, v, table = c.k[layer].cpu(), c.v[layer].cpu(), c.block_table.cpu()
            want_b = ref.bounds(k, c.bounds[layer].cpu(), c.maps.positions[:T].tolist(), c.maps.slots[:T].tolist())
            assert same(c.bounds[layer].cpu(), want_b)
            for r in range(B):
                pos = int(c.maps.positions[r])
                want = ref.select(q[r].double().cpu().view(H, hd), c.bounds[layer].cpu(), table[r].tolist(), pos, P, 6, 1, 2)
                got = few[r].tolist()
                assert got == [x + [-1] * (6 - len(x)) for x in want]
                kk, vv = ref.listed_keys(k, v, table[r].tolist(), pos, got)
                w = ref.attend_keys(q[r].double().cpu().view(H, hd), kk, vv, hd ** -0.5)
                check_row(out[r].double().cpu().view(H, hd), lse[r].double().cpu(), w, io, False)
        assert c.status()[0] == 0


@pytest.mark.parametrize("dtype,io", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_shared_prompt_of_a_server(dtype, io):
    """A prompt appended once, then requests that go on from it at its positions: the same as requests that
    hold all of it themselves."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, P, hk, H, hd, n = 6, 8, 2, 6, 64, 75
    c = paged.PagedCache(B + 1, 600, P, 60, 512, hk, hd, dtype=dtype)
    whole = paged.PagedCache(B, 600, P, 60, 700, hk, hd, dtype=dtype)
    shared = torch.randn(n, (H + 2 * hk) * hd, generator=g, device="cuda").to(io)
    c.plan(ints([0] * B + [n]))
    c.append(0, shared)
    whole.plan(ints([n] * B))
    whole.append(0, shared.repeat(B, 1))
    cu, preq, plen = ints([0, B]), ints([B]), ints([n])
    for step in range(4):
        new = [1] * B if step else [3, 1, 9, 17, 2, 8]
        T = sum(new)
        qkv = torch.randn(T, (H + 2 * hk) * hd, generator=g, device="cuda").to(io)
        c.plan(ints(new + [0]))
        m = c.maps
        # rotated where they stand behind the prefix
        q = paged.paged_append(qkv, c.k[0], c.v[0], m.positions[:T] + n, m.slots[:T])
        rows = torch.tensor([sum(new[:i + 1]) for i in range(B + 0)], dtype=torch.int32, device="cuda")
        out, lse = c.attend_prefix(0, q, torch.stack([rows[0] * 0, rows[-1]]), preq, plen, lse=True)
        whole.plan(ints(new))
        q2 = whole.append(0, qkv)
        assert torch.equal(q, q2)
        b, bl = whole.attend(0, q2, lse=True)
        assert (out.double() - b.double()).abs().max() <= 4 * torch.finfo(io).eps * b.double().abs().max() + 1e-5 * (io == F32)
        assert torch.allclose(lse, bl, rtol=1e-5)


def _calls(seed, io=BF16, scratch=None):
    """The four calls on one set of inputs, as closures on tensors that stay."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, H, hk, hd, P, W = 9, 8, 2, 128, 8, 500
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(io)  # noqa: E731
    N = (R + 1) * W
    k, v = rnd(N, P, hk, hd), rnd(N, P, hk, hd)
    table = torch.randperm(N, generator=g, device="cuda").to(torch.int32).view(R + 1, W)
    q, pos = rnd(R, H * hd), torch.randint(100, W * P, (R,), generator=g, device="cuda").to(torch.int32)
    slots = torch.arange(N * P, device="cuda")
    every = (torch.arange(N * P, device="cuda") % P).to(torch.int32)
    bounds = torch.zeros(N, hk, 2, hd, dtype=io, device="cuda")
    pages = torch.zeros(R, hk, 7, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(2, R, H * hd, dtype=io, device="cuda"), torch.zeros(2, R, H, device="cuda")
    cu, preq, plen = ints([0, 5, 9]), ints([R, 3]), ints([W * P - 3, 50])
    ws = [paged.paged_select_workspace(q, bounds, table, P), paged.paged_sparse_attention_workspace(q, k, pages),
          paged.paged_prefix_attention_workspace(q, k, table, plen)]
    if scratch is not None:
        ws = scratch + ws[len(scratch):]

    def run(stream=None):
        paged.paged_bounds(k, bounds, every, slots, stream=stream)
        paged.paged_select(q, bounds, table, pos, P, 7, pages=pages, workspace=ws[0], stream=stream)
        paged.paged_sparse_attention(q, k, v, table, pos, pages, out=out[0], lse=lse[0], workspace=ws[1], stream=stream)
        paged.paged_prefix_attention(q, k, v, table, pos, cu, preq, plen, out=out[1], lse=lse[1], workspace=ws[2],
                                     stream=stream)
    run.scratch = ws
    return run, [bounds, pages, out, lse], [k, v, q, pos]


def test_calls_in_a_graph_and_twice():
    """Captured and replayed on other inputs; the same bits each time."""
    run, outs, ins = _calls(1)
    run()
    first = [x.clone() for x in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for x in outs:
        x.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    _, _, other = _calls(2)
    for a, b in zip(ins, other):
        a.copy_(b)
    graph.replay()
    replayed = [x.clone() for x in outs]
    run()
    assert all(torch.equal(a, b) for a, b in zip(replayed, outs))
    assert not torch.equal(first[2], outs[2])


def test_two_graphs_one_after_the_other():
    """Two captured graphs that share scratch, replayed in turn on one stream."""
    run1, outs1, _ = _calls(3)
    run2, outs2, _ = _calls(4, scratch=run1.scratch)
    run1(), run2()
    first = [[x.clone() for x in o] for o in (outs1, outs2)]
    graphs = []
    for r in (run1, run2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            r()
    for _ in range(20):
        for gr in graphs:
            gr.replay()
    for o, f in zip((outs1, outs2), first):
        assert all(torch.equal(a, b) for a, b in zip(o, f))


def test_calls_on_another_stream():
    run, outs, _ = _calls(5)
    run()
    first = [x.clone() for x in outs]
    for x in outs:
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_two_streams_at_once():
    calls = [_calls(6), _calls(7)]
    for run, _, _ in calls:
        run()
    first = [[x.clone() for x in outs] for _, outs, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for s, (run, _, _) in zip(streams, calls):
            run(stream=s)
    torch.cuda.synchronize()
    for (_, outs, _), f in zip(calls, first):
        assert all(torch.equal(a, b) for a, b in zip(outs, f))


def test_past_32_bits():
    """Cache offsets past 2^32 elements, in every call that reads them."""
    hd, P, stride = 32, 4, 2**31 + 64
    big_k, big_v = (torch.zeros(2 * stride + P * hd, dtype=BF16, device="cuda") for _ in range(2))
    k, v = (x.as_strided((3, P, 1, hd), (stride, hd, hd, 1)) for x in (big_k, big_v))
    k[2], v[2] = torch.randn(P, 1, hd, device="cuda").to(BF16), torch.randn(P, 1, hd, device="cuda").to(BF16)
    bounds = torch.zeros(3, 1, 2, hd, dtype=BF16, device="cuda")
    paged.paged_bounds(k, bounds, ints([0, 1, 2, 3]), ints([8, 9, 10, 11], torch.int64))
    assert torch.equal(bounds[2, 0, 0], k[2, :, 0].amin(0)) and torch.equal(bounds[2, 0, 1], k[2, :, 0].amax(0))
    q = torch.randn(1, 2 * hd, device="cuda").to(BF16)
    want, lse = paged.paged_attention(q, k, v, ints([[2]]), ints([3]), lse=True)
    a, al = paged.paged_sparse_attention(q, k, v, ints([[2]]), ints([3]), ints([[[0]]]), lse=True)
    b, bl = paged.paged_prefix_attention(q, k, v, ints([[1], [2]]), ints([-1]), ints([0, 1]), ints([1]), ints([4]), lse=True)
    for x, xl in ((a, al), (b, bl)):
        assert (x.double() - want.double()).abs().max() <= 4 * 2.0 ** -8 * want.double().abs().max()
        assert torch.allclose(xl, lse, rtol=1e-5)


def test_binding_refusals():
    """Tensors of the wrong type, shape, order or size, before anything runs."""
    k, v = (torch.zeros(6, 8, 2, 64, device="cuda") for _ in range(2))
    q, table, pos = torch.zeros(3, 4 * 64, device="cuda"), ints([[0, 1]] * 4), ints([9, 3, 15])
    bounds, pages = torch.zeros(6, 2, 2, 64, device="cuda"), torch.zeros(3, 2, 5, dtype=torch.int32, device="cuda")
    slots, cu, one = ints([0, 1, 2], torch.int64), ints([0, 3]), ints([3])
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(6, 2, 2, 128, device="cuda")
    for call in (
            lambda: paged.paged_bounds(k, bounds.to(BF16), pos, slots),
            lambda: paged.paged_bounds(k, wide[..., ::2], pos, slots),
            lambda: paged.paged_bounds(k, bounds[:5], pos, slots),
            lambda: paged.paged_bounds(k, bounds, pos, slots[:2]),
            lambda: paged.paged_bounds(k, bounds, pos, pos),
            lambda: paged.paged_select(q, wide[..., ::2], table, pos, 8, 5),
            lambda: paged.paged_select(q, bounds[:, :, 0], table, pos, 8, 5),
            lambda: paged.paged_select(q[:, :100], bounds, table, pos, 8, 5),
            lambda: paged.paged_select(q, bounds, table.long(), pos, 8, 5),
            lambda: paged.paged_select(q, bounds, table, pos[:2], 8, 5),
            lambda: paged.paged_select(q, bounds, table, pos, 8, 5, pages=pages[:, :, :4]),
            lambda: paged.paged_select(q, bounds, table, pos, 8, -1),
            lambda: paged.paged_select(q, bounds, table, pos, 2**32 + 8, 5),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages[:2]),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages[:, :1]),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages.long()),
            lambda: paged.paged_sparse_attention(q, k, v.to(BF16), table, pos, pages),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages, out=q.to(BF16)),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages, scale=1e-40),
            lambda: paged.paged_prefix_attention(q, k, v, table, pos, one, one, one),
            lambda: paged.paged_prefix_attention(q, k, v, table, pos, cu, cu[:0], one),
            lambda: paged.paged_prefix_attention(q, k, v, table, pos, cu, one, one.float()),
            lambda: paged.paged_prefix_attention(q, k, v, table, pos, cu, one, one, requests=pos.long()),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: paged.paged_select(q, bounds, table, pos, 8, 0),
            lambda: paged.paged_select(q, bounds, table, pos, 8, 5, first=4, last=2),
            lambda: paged.paged_select(q, bounds, table, pos, 8, 5, workspace=small),
            lambda: paged.paged_sparse_attention(q, k, v, table, pos, pages[:, :, :0].contiguous()),
            lambda: paged.paged_sparse_attention(q, k, v, table[:2], pos, pages),
            lambda: paged.paged_prefix_attention(q, k, v, table, pos, cu, one, one, workspace=small),
            lambda: paged.paged_prefix_attention(q, k, v, table[:2], pos, cu, one, one),
    ):
        with pytest.raises(binding.RQError):
            call()
