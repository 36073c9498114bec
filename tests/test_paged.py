"""The paged K/V cache without a GPU: what its calls refuse, on the host, before anything
is enqueued, and the plain plan that the GPU tests compare with, against its invariants."""
import ctypes as C
import os
import random
import re

import numpy as np
import pytest
import torch

import __graft_entry__
import paged_ref
from rq_transformer_frame_gb300 import binding, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def test_struct_matches_header():
    src = open(os.path.join(ROOT, "include", "rq.h")).read()
    body = src[src.index("typedef struct {\n  void *k, *v;"):src.index("} rq_paged_kv;")]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"([a-z_]+)(?=[,;])", body)
    assert names == ["k", "v", "block_stride", "row_stride", "head_stride", "dtype", "heads",
                     "head_dim", "block_size", "n_blocks"]

    class Kv(C.Structure):
        _fields_ = [(n, C.c_void_p) for n in names[:2]] + [(n, C.c_int64) for n in names[2:5]] + \
            [(n, C.c_int32) for n in names[5:]]
    assert C.sizeof(Kv) == paged._KV.size
    x = Kv.from_buffer_copy(_kv())
    assert (x.k, x.v, x.block_stride, x.row_stride, x.head_stride) == (A, B_, 16 * 512, 512, 128)
    assert (x.dtype, x.heads, x.head_dim, x.block_size, x.n_blocks) == (1, 4, 128, 16, 8)


BAD_KV = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=A + 8), 1), (dict(v=B_ + 2), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(heads=0), 1), (dict(p=0), 1), (dict(n=0), 1),
    (dict(hd=48), 6), (dict(hd=256), 6), (dict(bs=4), 1), (dict(rs=-512), 1), (dict(hs=100), 1),
    (dict(dtype=0, hs=2), 1),
]


def _append(lib, kv=None, **kw):
    d = dict(tokens=3, heads=8, dt=1, qkv=A, stride=16 * 128, qa=None, ka=None, eps=1e-6, style=0,
             rd=128, theta=1e4, pos=A, slots=A, qdt=1, out=C_)
    d.update(kw)
    return lib.rq_paged_append(kv or _kv(), d["tokens"], d["heads"], d["dt"], d["qkv"], d["stride"],
                               d["qa"], d["ka"], d["eps"], d["style"], d["rd"], d["theta"], d["pos"],
                               d["slots"], d["qdt"], d["out"], None)


def _attend(lib, kv=None, **kw):
    d = dict(rows=3, heads=8, batch=3, W=4, table=A, req=None, pos=A, window=0, scale=0.0, qdt=1,
             q=A, out=B_, lse=None, ws=C_, wsb=1 << 30)
    d.update(kw)
    return lib.rq_paged_attention(kv or _kv(), d["rows"], d["heads"], d["batch"], d["W"], d["table"],
                                  d["req"], d["pos"], d["window"], d["scale"], d["qdt"], d["q"],
                                  d["out"], d["lse"], d["ws"], d["wsb"], None)


@pytest.mark.parametrize("kw,status", BAD_KV)
def test_cache_refusals(lib, kw, status):
    assert _append(lib, _kv(**kw)) == status
    assert _attend(lib, _kv(**kw)) == status


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(heads=0), dict(heads=2**31 - 5), dict(dt=2), dict(qdt=3), dict(qkv=None), dict(qkv=A + 8),
    dict(stride=16 * 128 - 8), dict(stride=16 * 128 + 4), dict(qa=A + 4), dict(ka=A + 8),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(style=2), dict(style=-1),
    dict(rd=-8), dict(rd=136), dict(rd=12), dict(theta=1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(pos=None), dict(slots=None), dict(out=None), dict(out=C_ + 8),
])
def test_append_refusals(lib, kw):
    assert _append(lib, **kw) == binding.RQ_ERR_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=6), 1), (dict(batch=0), 1), (dict(W=0), 1),
    (dict(window=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(qdt=2), 1), (dict(table=None), 1), (dict(pos=None), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=A + 8), 1), (dict(out=B_ + 4), 1),
    (dict(ws=C_ + 8), 1), (dict(rows=4), 1),
    (dict(rows=2**30, batch=2**30), 6),
])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


def test_attention_wants_its_whole_workspace(lib):
    """Rows that may be long are cut over the card and need scratch for their pieces."""
    many = dict(rows=300, batch=300, W=400)
    need = lib.rq_paged_attention_workspace_size(_kv(), 300, 8, 400, 0)
    assert need > 0
    assert _attend(lib, **many, wsb=need - 1) == binding.RQ_ERR_ARG
    assert _attend(lib, **many, ws=None) == binding.RQ_ERR_ARG
    size = lambda **kw: lib.rq_paged_attention_workspace_size(  # noqa: E731
        kw.get("kv", _kv()), kw.get("rows", 300), kw.get("heads", 8), kw.get("W", 400), kw.get("window", 0))
    assert size() == need
    assert [size(**kw) for kw in (dict(kv=_kv(hd=48)), dict(rows=0), dict(heads=6), dict(W=0),
                                  dict(window=-1))] == [0] * 5


def test_no_rows_is_not_an_error(lib):
    """Zero rows: nothing is enqueued, and no pointer of theirs is needed."""
    assert _append(lib, tokens=0, qkv=None, pos=None, slots=None, out=None) == binding.RQ_OK
    assert _attend(lib, rows=0, q=None, out=None, pos=None, table=None, ws=None) == binding.RQ_OK


def _plan(lib, **kw):
    d = dict(B=4, W=8, P=16, N=100, M=64, ptrs=[A] * 11)
    d.update(kw)
    return lib.rq_paged_plan(d["B"], d["W"], d["P"], d["N"], d["M"], *d["ptrs"], None)


@pytest.mark.parametrize("kw,status", [(dict(B=0), 1), (dict(W=0), 1), (dict(P=0), 1), (dict(N=0), 1),
                                       (dict(M=0), 1), (dict(B=8193), 6), (dict(M=2**30 + 1), 6)] +
                         [(dict(ptrs=[A] * i + [None] + [A] * (10 - i)), 1) for i in range(11)])
def test_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status


def test_pool_init_refusals(lib):
    assert lib.rq_paged_pool_init(0, A, B_, None) == binding.RQ_ERR_ARG
    assert lib.rq_paged_pool_init(8, None, B_, None) == binding.RQ_ERR_ARG
    assert lib.rq_paged_pool_init(8, A, None, None) == binding.RQ_ERR_ARG


def test_binding_refuses_host_tensors(lib):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        paged.paged_plan(i(2), i(2), i(4), i(8), i(2, 4), 16, 8)
    k = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError):
        paged.paged_append(torch.zeros(3, 6 * 64), k, k, i(3), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        paged.paged_attention(torch.zeros(3, 128), k, k, i(3, 4), i(3))


@pytest.mark.parametrize("seed", range(6))
def test_plain_plan_keeps_the_ledger(seed):
    """Over many steps of arrivals, growth and ends: every block is either free once or held
    by one request once, and every token's slot is its own."""
    r = random.Random(seed)
    B, W, P, N = 6, r.choice([2, 5]), r.choice([1, 4, 5]), 23
    lens, pool = [0] * B, [0, N, 0, 0]
    table, ids = np.full((B, W), -1, np.int32), np.arange(N, dtype=np.int32)
    for _ in range(60):
        new = [r.choice([0, 1, 1, 1, 3, 9, -1]) for _ in range(B)]
        was = (list(lens), list(pool), table.copy(), ids.copy())
        o = paged_ref.plan(new, lens, pool, ids, table, P, 40)
        lens, pool, table, ids = list(o["lens"]), o["pool"], o["table"], o["free_ids"]
        if pool[2]:
            assert lens == was[0] and pool[:2] == was[1][:2]
            assert (table == was[2]).all() and (ids == was[3]).all() and (o["req"] == -1).all()
        held = [int(table[b, i]) for b in range(B) for i in range(min(-(-lens[b] // P), W))]
        free = [int(ids[(pool[0] + i) % N]) for i in range(pool[1])]
        assert sorted(held + free) == list(range(N))
        slots = o["slot"][o["slot"] >= 0]
        assert len(set(slots.tolist())) == len(slots)


@pytest.mark.parametrize("n", [2**30 + 1, 2**31 - 300, 2**31 - 1])
def test_pools_past_32_bit_counting_are_refused(lib, n):
    """A thread's next ring entry, up to 1024 past the last, has to stay below 2^31."""
    assert lib.rq_paged_pool_init(n, A, B_, None) == binding.RQ_ERR_UNSUPPORTED
    assert _plan(lib, N=n) == binding.RQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scales_past_f32_are_refused(lib, scale):
    """Finite themselves, but not times log2(e), as the kernels take them: 0 times that is NaN."""
    assert _attend(lib, scale=scale) == binding.RQ_ERR_ARG


def test_rows_past_32_bit_counting_are_refused(lib):
    """A row's elements are counted in 32 bits: 2^24 heads of 128 dimensions are 2^31."""
    assert _attend(lib, rows=1, heads=2**24) == binding.RQ_ERR_UNSUPPORTED
    assert _attend(lib, rows=3, heads=2**26, req=A) == binding.RQ_ERR_UNSUPPORTED


def test_a_threads_next_row_and_element_stay_in_32_bits(lib):
    """A warp steps over all rows by up to 1216, a block over a row's elements by 256."""
    one = _kv(heads=1)
    assert _attend(lib, one, rows=2**31 - 1, heads=1, batch=2**31 - 1) == binding.RQ_ERR_UNSUPPORTED
    assert _attend(lib, one, rows=2**30 + 1, heads=1, batch=2**31 - 1) == binding.RQ_ERR_UNSUPPORTED
    assert _attend(lib, one, rows=1, heads=2**24 - 1) == binding.RQ_ERR_UNSUPPORTED
    assert _attend(lib, rows=1, heads=2**23 + 4) == binding.RQ_ERR_UNSUPPORTED
