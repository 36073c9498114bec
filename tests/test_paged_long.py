"""Block bounds, page selection, attention over listed pages and behind shared prefixes without a GPU:
what the calls refuse, on the host, before anything is enqueued, and the plain implementations that
the GPU tests compare with, against one another."""
import random

import pytest
import torch

import __graft_entry__
import paged_long_ref as ref
import paged_ref
from rq_transformer_frame_gb300 import binding, paged

A, B_, C_ = 1 << 12, 1 << 13, 1 << 14  # addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load()


def _kv(**kw):
    d = dict(k=A, v=B_, bs=16 * 512, rs=512, hs=128, dtype=binding.RQ_BF16, heads=4, hd=128, p=16, n=8)
    d.update(kw)
    return paged._KV.pack(d["k"], d["v"], d["bs"], d["rs"], d["hs"], d["dtype"], d["heads"], d["hd"],
                          d["p"], d["n"])


def _bounds(lib, kv=None, **kw):
    d = dict(bounds=C_, tokens=3, pos=A, slots=A)
    d.update(kw)
    return lib.rq_paged_bounds(kv or _kv(), d["bounds"], d["tokens"], d["pos"], d["slots"], None)


def _select(lib, kv=None, **kw):
    d = dict(bounds=C_, rows=3, heads=8, batch=3, W=40, table=A, req=None, pos=A, top=9, first=1, last=2, qdt=1,
             q=A, pages=B_, ws=C_, wsb=1 << 30)
    d.update(kw)
    return lib.rq_paged_select(kv or _kv(), d["bounds"], d["rows"], d["heads"], d["batch"], d["W"], d["table"],
                               d["req"], d["pos"], d["top"], d["first"], d["last"], d["qdt"], d["q"], d["pages"],
                               d["ws"], d["wsb"], None)


def _sparse(lib, kv=None, **kw):
    d = dict(rows=3, heads=8, batch=3, W=40, table=A, req=None, pos=A, list=9, pages=A, scale=0.0, qdt=1, q=A,
             out=B_, lse=None, ws=C_, wsb=1 << 30)
    d.update(kw)
    return lib.rq_paged_sparse_attention(kv or _kv(), d["rows"], d["heads"], d["batch"], d["W"], d["table"], d["req"],
                                         d["pos"], d["list"], d["pages"], d["scale"], d["qdt"], d["q"], d["out"],
                                         d["lse"], d["ws"], d["wsb"], None)


def _prefix(lib, kv=None, **kw):
    d = dict(rows=3, heads=8, batch=3, W=40, table=A, req=None, pos=A, groups=2, cu=A, preq=A, plen=A, scale=0.0,
             qdt=1, q=A, out=B_, lse=None, ws=C_, wsb=1 << 40)
    d.update(kw)
    return lib.rq_paged_prefix_attention(kv or _kv(), d["rows"], d["heads"], d["batch"], d["W"], d["table"], d["req"],
                                         d["pos"], d["groups"], d["cu"], d["preq"], d["plen"], d["scale"], d["qdt"],
                                         d["q"], d["out"], d["lse"], d["ws"], d["wsb"], None)


BAD_KV = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=A + 8), 1), (dict(v=B_ + 2), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(heads=0), 1), (dict(p=0), 1), (dict(n=0), 1),
    (dict(hd=48), 6), (dict(hd=256), 6), (dict(bs=4), 1), (dict(rs=-512), 1), (dict(hs=100), 1),
    (dict(dtype=0, hs=2), 1),
]


@pytest.mark.parametrize("kw,status", BAD_KV)
def test_cache_refusals(lib, kw, status):
    for call in (_bounds, _select, _sparse, _prefix):
        assert call(lib, _kv(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(bounds=None), 1), (dict(bounds=C_ + 8), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(tokens=2**30 + 1), 6)])
def test_bounds_refusals(lib, kw, status):
    assert _bounds(lib, **kw) == status


ROWS = [(dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=6), 1), (dict(batch=0), 1), (dict(W=0), 1),
        (dict(qdt=2), 1), (dict(table=None), 1), (dict(pos=None), 1), (dict(q=None), 1), (dict(q=A + 8), 1),
        (dict(ws=C_ + 8), 1), (dict(rows=4), 1), (dict(rows=2**30, batch=2**30), 6), (dict(rows=1, heads=2**24), 6),
        (dict(rows=3, heads=2**26, req=A), 6)]


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(bounds=None), 1), (dict(bounds=C_ + 8), 1), (dict(pages=None), 1), (dict(ws=None), 1), (dict(top=0), 1),
    (dict(first=-1), 1), (dict(last=0), 1), (dict(last=9), 1), (dict(first=2**31 - 1, last=2**31 - 1), 1),
    (dict(W=2**30 + 1), 6), (dict(rows=2**20, req=A, W=2**30), 6), (dict(top=2**30 + 1), 6),
    (dict(kv=_kv(dtype=0, heads=2**22, bs=2**33), rows=1, heads=2**22), 6)])
def test_select_refusals(lib, kw, status):
    assert _select(lib, **kw) == status


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(list=0), 1), (dict(list=-3), 1), (dict(pages=None), 1), (dict(out=None), 1), (dict(out=B_ + 4), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(list=2**27), 6),
    (dict(list=2**31 // 16 - 4), 6)])
def test_sparse_refusals(lib, kw, status):
    assert _sparse(lib, **kw) == status


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(groups=-1), 1), (dict(groups=2**16 + 1), 6), (dict(cu=None), 1), (dict(preq=None), 1), (dict(plen=None), 1),
    (dict(out=None), 1), (dict(out=B_ + 4), 1), (dict(ws=None), 1), (dict(scale=float("nan")), 1),
    (dict(scale=-3e38), 1)])
def test_prefix_refusals(lib, kw, status):
    assert _prefix(lib, **kw) == status


def test_the_calls_want_their_whole_workspace(lib):
    need = lib.rq_paged_select_workspace_size(_kv(), 3, 40)
    assert need > 0 and _select(lib, wsb=need - 1) == binding.RQ_ERR_ARG
    need = lib.rq_paged_prefix_attention_workspace_size(_kv(), 3, 8, 40, 2)
    assert need > 0 and _prefix(lib, wsb=need - 1) == binding.RQ_ERR_ARG
    need = lib.rq_paged_sparse_attention_workspace_size(_kv(), 300, 8, 400)
    many = dict(rows=300, batch=300, list=400)
    assert need > 0 and _sparse(lib, **many, wsb=need - 1) == binding.RQ_ERR_ARG
    assert _sparse(lib, **many, ws=None) == binding.RQ_ERR_ARG
    for bad in (dict(hd=48), dict(n=0)):
        assert lib.rq_paged_select_workspace_size(_kv(**bad), 3, 40) == 0
        assert lib.rq_paged_sparse_attention_workspace_size(_kv(**bad), 300, 8, 400) == 0
        assert lib.rq_paged_prefix_attention_workspace_size(_kv(**bad), 3, 8, 40, 2) == 0
    assert lib.rq_paged_sparse_attention_workspace_size(_kv(), 300, 6, 400) == 0
    assert lib.rq_paged_prefix_attention_workspace_size(_kv(), 3, 8, 40, -1) == 0


def test_no_rows_is_not_an_error(lib):
    """Zero rows or tokens: nothing is enqueued, and no pointer of theirs is needed."""
    assert _bounds(lib, tokens=0, bounds=None, pos=None, slots=None) == binding.RQ_OK
    none = dict(rows=0, q=None, pos=None, table=None, ws=None)
    assert _select(lib, **none, pages=None, bounds=None) == binding.RQ_OK
    assert _sparse(lib, **none, pages=None, out=None) == binding.RQ_OK
    assert _prefix(lib, **none, out=None, cu=None, preq=None, plen=None) == binding.RQ_OK


def test_binding_refuses_host_tensors(lib):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k, q = torch.zeros(4, 16, 2, 64), torch.zeros(3, 256)
    with pytest.raises(ValueError):
        paged.paged_bounds(k, torch.zeros(4, 2, 2, 64), i(3), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        paged.paged_select(q, torch.zeros(4, 2, 2, 64), i(3, 4), i(3), 16, 2)
    with pytest.raises(ValueError):
        paged.paged_sparse_attention(q, k, k, i(3, 4), i(3), i(3, 2, 2))
    with pytest.raises(ValueError):
        paged.paged_prefix_attention(q, k, k, i(4, 4), i(3), i(2), i(1), i(1))



BIG = 2**32 + 5


@pytest.mark.parametrize("rows,p,W,n", [(BIG, 16, 4, 2), (3, BIG, 4, 2), (3, 16, BIG, 2), (3, 16, 4, BIG)])
def test_workspaces_of_sizes_past_32_bits(lib, rows, p, W, n):
    """A size that ctypes would take modulo 2^32 is refused (tensors that are shapes alone)."""
    e = lambda *s, dtype=torch.int32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    q, k, table = e(rows, 256, dtype=torch.bfloat16), e(4, p, 2, 64, dtype=torch.bfloat16), e(3, W)
    calls = [lambda: paged.paged_prefix_attention_workspace(q, k, table, e(n))]
    if W < BIG:
        calls.append(lambda: paged.paged_sparse_attention_workspace(q, k, e(rows, 2, n)))
    calls.append(lambda: paged.paged_attention_workspace(q, k, table, window=n))
    for call in calls:
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()


def test_a_cache_without_bounds_says_so():
    c = paged.PagedCache.__new__(paged.PagedCache)  # the host's side of one: its buffers are on a GPU
    c.bounds, c.k, c.block_size = None, torch.zeros(1, 4, 16, 2, 64), 16
    c.block_table = torch.zeros(3, 4, dtype=torch.int32)
    c.maps = paged.PagedPlan(*[torch.zeros(3, dtype=torch.int32)] * 6)
    for call in (lambda: c.bound(0, 3), lambda: c.select(0, torch.zeros(3, 256), 2)):
        with pytest.raises(ValueError, match="bounds=True"):
            call()

@pytest.mark.parametrize("seed", range(4))
def test_plain_attention_over_all_pages_is_attention(seed):
    """Every live page listed, or the positions cut into a prefix and the rest: paged_ref's attention."""
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    P, hk, heads, hd, W, N = r.choice([1, 3, 8]), 2, 4, 32, 9, 12
    k, v = torch.randn(N, P, hk, hd, generator=g), torch.randn(N, P, hk, hd, generator=g)
    table = torch.randperm(N, generator=g)[:W].tolist()
    pos = r.randint(0, 3 * W * P)
    q = torch.randn(heads, hd, generator=g).double()
    want = paged_ref.attend_row(q, k, v, table, pos, 0, 0.2)
    live = list(range(max(0, pos // P - W + 1), pos // P + 1))
    kk, vv = ref.listed_keys(k, v, table, pos, [live, live[::-1] + [-1, pos // P + 1]])
    got = ref.attend_keys(q, kk, vv, 0.2)
    a, b = ref.request_keys(k, v, table, pos)
    again = ref.attend_keys(q, [a[:, h] for h in range(hk)], [b[:, h] for h in range(hk)], 0.2)
    for x in (got, again):
        assert torch.allclose(x["out"], want["out"], rtol=1e-12) and torch.allclose(x["lse"], want["lse"], rtol=1e-12)


@pytest.mark.parametrize("seed", range(4))
def test_plain_scores_bound_every_key(seed):
    """No sum of the queries' products with a key of a page is above the page's score, so with room for
    all but one page the one left out is a lowest score."""
    g = torch.Generator().manual_seed(seed)
    P, hk, heads, hd, n = 4, 2, 6, 16, 9
    k = torch.randn(n, P, hk, hd, generator=g)
    b = ref.bounds(k, torch.zeros(n, hk, 2, hd), [p for _ in range(n) for p in range(P)], list(range(n * P)))
    assert torch.equal(b[:, :, 0], k.amin(1)) and torch.equal(b[:, :, 1], k.amax(1))
    q = torch.randn(heads, hd, generator=g).double()
    score = torch.zeros(n, hk, dtype=torch.float64)
    for h in range(hk):
        x = q[h * 3:(h + 1) * 3]
        score[:, h] = b[:, h, 1].double() @ x.clamp(min=0).sum(0) + b[:, h, 0].double() @ x.clamp(max=0).sum(0)
        sums = (k[:, :, h].double() @ x.T).sum(-1)
        assert (sums <= score[:, h, None] + 1e-12).all()
    lists = ref.select(q, b, list(range(n)), n * P - 1, P, n - 1, 0, 1)
    for h in range(hk):
        left = set(range(n)) - set(lists[h])
        assert left == {int(score[:n - 1, h].argmin())}
