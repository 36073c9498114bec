"""The paged K/V cache: a pool of blocks that many requests share (include/rq.h, the
rq_paged_* calls; argument marshalling only, like `binding`).

  paged_plan       block tables and token maps of a step, from the requests' lengths
  paged_append     per-head norm, position rotation, and K/V stored by slot
  paged_attention  one query token per row over its request's blocks
  paged_attention_workspace  scratch for it, where a call's addresses must stay
  PagedCache       the buffers of one cache, with the three as methods

A layer's cache is a pair of tensors k, v [n_blocks][block_size][kv_heads][head_dim] (f32
or bf16, of any strides that keep head_dim contiguous and every row 16-byte aligned).
Nothing here synchronizes except PagedCache.status(), so a step can be captured into a CUDA
graph; a captured step keeps its tensors' addresses, so pass `out`, `lse` and `workspace` (paged_attention_workspace).
Every call runs on `stream` (a torch.cuda.Stream; default: the current one of the
tensors' device); tensors it allocates belong to that stream. As with any work on a side
stream, a tensor of another one has to be ready there and to live until the call has run
(wait_stream, record_stream).
"""
from __future__ import annotations

import struct
from collections import namedtuple
from contextlib import contextmanager
from functools import lru_cache

import torch

from .binding import (RQ_BF16, RQ_F32, RQ_OK, RQ_PAGED_BAD_INPUT, RQ_PAGED_NO_BLOCKS,
                      RQ_PAGED_NO_TOKENS, RQ_ROPE_HALVES, RQ_ROPE_INTERLEAVED, RQError, load)

_F32, _I32, _I64 = torch.float32, torch.int32, torch.int64
# the device and stream that a call finds current, without building the Python objects for them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_KV = struct.Struct("@PPqqqiiiii4x")  # rq_paged_kv
_TYPE = {torch.float32: RQ_F32, torch.bfloat16: RQ_BF16}
_ROPE = {"interleaved": RQ_ROPE_INTERLEAVED, "halves": RQ_ROPE_HALVES}

# What rq_paged_plan writes: lengths and pool words afterwards, and the step's maps.
PagedPlan = namedtuple("PagedPlan", "lens pool cu_tokens requests positions slots")


# ctypes takes an int32 argument modulo 2^32, and the smallest scales as the 0 that means the default
_TINY = torch.finfo(torch.float32).tiny


def _fail(what, rc):
    raise RQError(rc, "%s failed" % what)


@contextmanager
def _on(device, stream):
    """The tensors' device, and the stream the call runs on, made current."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if stream.device != device:
                raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
            with torch.cuda.stream(stream):
                yield


# The checks stand in line in the calls below (a Python call costs as much as the check); these
# two say what was wrong.
def _bad_ints(name, n, dev, dtype=_I32):
    raise ValueError("%s: a contiguous %s tensor of %d elements on cuda:%d is wanted" % (name, dtype, n, dev))


def _bad_rows(name, shape, dtype, dev):
    raise ValueError("%s: a contiguous %s tensor of shape %s on cuda:%d is wanted" %
                     (name, dtype, tuple(shape), dev))


def _past_int32(*sizes):
    """What the calls ask where an `or` of their sizes is negative or past 31 bits: a negative size
    alone is the library's to refuse."""
    for x in sizes:
        if x >> 31 not in (0, -1):
            raise ValueError("a size of %d does not fit 32 bits" % x)


def _cache(k, v):
    """(rq_paged_kv packed, heads, head_dim, device index) of a layer's cache."""
    dev, dtype = k.get_device(), k.dtype
    if dev < 0 or dtype not in _TYPE or k.dim() != 4:
        raise ValueError("k, v: f32 or bf16 CUDA tensors [n_blocks][block_size][heads][head_dim]")
    n, p, h, hd = shape = k.shape
    strides = k.stride()
    if v.shape != shape or v.dtype is not dtype or v.get_device() != dev or v.stride() != strides:
        raise ValueError("k and v differ in shape, strides, type or device")
    if strides[3] != 1:
        raise ValueError("k, v: the elements of a head must be contiguous")
    return _KV.pack(k.data_ptr(), v.data_ptr(), strides[0], strides[1], strides[2], _TYPE[dtype],
                    h, hd, p, n), h, hd, dev


@lru_cache(maxsize=1024)
def _workspace_size(dev, dtype, rows, heads, kv_heads, head_dim, head_stride, block_size, max_blocks,
                    window):
    # the size goes by these alone: any pointer and other strides stand for a cache
    kv = _KV.pack(16, 16, 0, 0, head_stride, dtype, kv_heads, head_dim, block_size, 1)
    return load().rq_paged_attention_workspace_size(kv, rows, heads, max_blocks, window)


def paged_attention_workspace(q, k, block_table, window=0):
    """Scratch for paged_attention with these shapes, for calls whose addresses must stay (a
    captured graph), or None where the call needs none."""
    n, p, hk, hd = k.shape
    if (window | block_table.shape[1]) >> 31:
        _past_int32(window, block_table.shape[1])
    with _on(k.device, None):
        size = _workspace_size(k.get_device(), _TYPE[k.dtype], q.shape[0], q.shape[1] // hd, hk, hd,
                               k.stride(2), p, block_table.shape[1], window)
    return torch.empty(size, dtype=torch.uint8, device=k.device) if size else None


# Each call below runs on the current stream of the tensors' device; a call on another
# stream, or while another device is current, first makes those current.

def paged_plan(new_lens, lens, pool, free_ids, block_table, block_size, max_tokens, out=None,
               stream=None) -> PagedPlan:
    """rq_paged_plan: new_lens, lens [B] int32, pool [4] int32, free_ids [n_blocks] int32 and
    block_table [B][max_blocks] int32 (the last two updated in place).

    out: a PagedPlan (or the same tuple) of tensors to write, lens [B], pool [4], cu_tokens
    [B + 1], requests and positions [max_tokens] int32 and slots [max_tokens] int64; its lens
    and pool may be the inputs themselves.  pool[2] says whether the call did anything
    (RQ_PAGED_*)."""
    dev = lens.get_device()
    if dev < 0 or block_table.dim() != 2:
        raise ValueError("lens, block_table: CUDA tensors [B] and [B][max_blocks] are wanted")
    if stream is not None or _current_device() != dev:
        with _on(lens.device, stream):
            return paged_plan(new_lens, lens, pool, free_ids, block_table, block_size, max_tokens, out)
    B, W = block_table.shape
    M = int(max_tokens)
    N = free_ids.numel()
    if (block_size | M | B | W | N) >> 31:
        _past_int32(block_size, M, B, W, N)
    if out is None:
        e = lambda n, dt=_I32: torch.empty(n, dtype=dt, device=lens.device)  # noqa: E731
        out = PagedPlan(e(B), e(4), e(B + 1), e(M), e(M), e(M, _I64))
    elif type(out) is not PagedPlan:
        out = PagedPlan(*out)
    if lens.numel() != B or new_lens.numel() != B:
        raise ValueError("new_lens, lens and block_table differ in their requests")
    o_lens, o_pool, cu, req, pos, slots = out
    for name, t, n in (("new_lens", new_lens, B), ("lens", lens, B), ("pool", pool, 4), ("free_ids", free_ids, 1),
                       ("block_table", block_table, B * W), ("out.lens", o_lens, B), ("out.pool", o_pool, 4),
                       ("out.cu_tokens", cu, B + 1), ("out.requests", req, M), ("out.positions", pos, M)):
        if t.dtype is not _I32 or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
            _bad_ints(name, n, dev)
    if slots.dtype is not _I64 or slots.get_device() != dev or slots.numel() < M or not slots.is_contiguous():
        _bad_ints("out.slots", M, dev, _I64)
    rc = load().rq_paged_plan(
        B, W, block_size, N, M, new_lens.data_ptr(), lens.data_ptr(), pool.data_ptr(),
        free_ids.data_ptr(), block_table.data_ptr(), o_lens.data_ptr(), o_pool.data_ptr(), cu.data_ptr(),
        req.data_ptr(), pos.data_ptr(), slots.data_ptr(), _current_stream(dev))
    if rc != RQ_OK:
        _fail("rq_paged_plan", rc)
    return out


def paged_append(qkv, k, v, positions, slots, q_alpha=None, k_alpha=None, eps=1e-8,
                 rope="interleaved", rope_dim=None, rope_theta=10000.0, q_dtype=None, out=None,
                 stream=None):
    """rq_paged_append: rows qkv [T][(heads + 2 kv_heads) * head_dim] f32 or bf16 (rows may be
    strided) -> queries [T][heads * head_dim] in q_dtype (default: qkv's, or out's), keys and
    values stored in k, v at `slots` (int64 [T]).  rope: "interleaved" or "halves" over the
    first rope_dim (default: all) dimensions; alphas: f32 [head_dim] or None for no norm."""
    kv, hk, hd, dev = _cache(k, v)
    if stream is not None or _current_device() != dev:
        with _on(k.device, stream):
            return paged_append(qkv, k, v, positions, slots, q_alpha, k_alpha, eps, rope, rope_dim,
                                rope_theta, q_dtype, out)
    dtype = qkv.dtype
    if qkv.dim() != 2 or dtype not in _TYPE or qkv.get_device() != dev or qkv.stride(1) != 1:
        raise ValueError("qkv: an f32 or bf16 tensor [T][width], rows contiguous, on cuda:%d" % dev)
    T, width = qkv.shape
    heads = width // hd - 2 * hk
    if heads < 1 or width % hd:
        raise ValueError("qkv: %d columns are not queries, %d keys and %d values of %d" %
                         (width, hk, hk, hd))
    if rope not in _ROPE:
        raise ValueError("rope: 'interleaved' or 'halves'")
    if out is None:
        out = torch.empty((T, heads * hd), dtype=q_dtype or dtype, device=k.device)
    o_dtype = out.dtype
    if o_dtype not in _TYPE or (q_dtype is not None and o_dtype is not q_dtype):
        raise ValueError("out: f32 or bf16, as q_dtype says")
    if out.shape != (T, heads * hd) or out.get_device() != dev or not out.is_contiguous():
        _bad_rows("out", (T, heads * hd), o_dtype, dev)
    for alpha in (q_alpha, k_alpha):
        if alpha is not None and (alpha.dtype is not _F32 or alpha.get_device() != dev or alpha.shape != (hd,) or
                                  not alpha.is_contiguous()):
            _bad_rows("q_alpha, k_alpha", (hd,), _F32, dev)
    if positions.dtype is not _I32 or positions.get_device() != dev or positions.numel() < T or \
            not positions.is_contiguous():
        _bad_ints("positions", T, dev)
    if slots.dtype is not _I64 or slots.get_device() != dev or slots.numel() < T or not slots.is_contiguous():
        _bad_ints("slots", T, dev, _I64)
    rope_dim = hd if rope_dim is None else rope_dim
    if rope_dim >> 31:
        _past_int32(rope_dim)
    rc = load().rq_paged_append(
        kv, T, heads, _TYPE[dtype], qkv.data_ptr(), qkv.stride(0) if T > 1 else width,
        None if q_alpha is None else q_alpha.data_ptr(), None if k_alpha is None else k_alpha.data_ptr(), eps,
        _ROPE[rope], rope_dim, rope_theta, positions.data_ptr(), slots.data_ptr(),
        _TYPE[o_dtype], out.data_ptr(), _current_stream(dev))
    if rc != RQ_OK:
        _fail("rq_paged_append", rc)
    return out


def paged_attention(q, k, v, block_table, positions, requests=None, window=0, scale=0.0, out=None,
                    lse=None, workspace=None, stream=None):
    """rq_paged_attention: q [R][heads * head_dim] f32 or bf16, block_table [B][max_blocks],
    positions [R] (-1: an empty request), requests [R] (-1: padding, its output left as it
    was; None: row r is request r), all int32 -> (out [R][heads * head_dim], lse [R][heads]
    f32, None unless a tensor or True is passed for it).  workspace: what
    paged_attention_workspace gives for these shapes (allocated here if None)."""
    kv, hk, hd, dev = _cache(k, v)
    if stream is not None or _current_device() != dev:
        with _on(k.device, stream):
            return paged_attention(q, k, v, block_table, positions, requests, window, scale, out, lse,
                                   workspace)
    dtype = q.dtype
    if q.dim() != 2 or dtype not in _TYPE or q.shape[1] % hd or block_table.dim() != 2:
        raise ValueError("q: an f32 or bf16 tensor [R][heads * head_dim]; block_table [B][max_blocks]")
    shape = q.shape
    R, heads = shape[0], shape[1] // hd
    B, W = block_table.shape
    if (window | B | W) >> 31:
        _past_int32(window, B, W)
    if scale and -_TINY < scale < _TINY:
        raise ValueError("scale: 0 for 1 / sqrt(head_dim), or at least %g" % _TINY)
    if out is None:
        out = torch.empty_like(q)
    if lse is True:
        lse = torch.empty((R, heads), dtype=_F32, device=k.device)
    if q.get_device() != dev or not q.is_contiguous():
        _bad_rows("q", shape, dtype, dev)
    if out.dtype is not dtype or out.get_device() != dev or out.shape != shape or not out.is_contiguous():
        _bad_rows("out", shape, dtype, dev)
    if lse is not None and (lse.dtype is not _F32 or lse.get_device() != dev or lse.shape != (R, heads) or
                            not lse.is_contiguous()):
        _bad_rows("lse", (R, heads), _F32, dev)
    if block_table.dtype is not _I32 or block_table.get_device() != dev or not block_table.is_contiguous():
        _bad_ints("block_table", B * W, dev)
    if positions.dtype is not _I32 or positions.get_device() != dev or positions.numel() < R or \
            not positions.is_contiguous():
        _bad_ints("positions", R, dev)
    if requests is not None and (requests.dtype is not _I32 or requests.get_device() != dev or
                                 requests.numel() < R or not requests.is_contiguous()):
        _bad_ints("requests", R, dev)
    if workspace is None:
        nbytes = _workspace_size(dev, _TYPE[k.dtype], R, heads, hk, hd, k.stride(2), k.shape[1], W, window)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=k.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on cuda:%d" % dev)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    rc = load().rq_paged_attention(
        kv, R, heads, B, W, block_table.data_ptr(), None if requests is None else requests.data_ptr(),
        positions.data_ptr(), window, scale, _TYPE[dtype], q.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), nbytes,
        _current_stream(dev))
    if rc != RQ_OK:
        _fail("rq_paged_attention", rc)
    return out, lse


class PagedCache:
    """The buffers of one paged cache and its step's maps, at fixed addresses.

    batch request rows, n_blocks blocks of block_size positions per layer, at most
    max_blocks blocks a request (past that its table is a ring) and max_tokens new tokens a
    step.  All layers share the block table; layer l's cache is k[l], v[l]."""

    def __init__(self, batch, n_blocks, block_size, max_blocks, max_tokens, kv_heads, head_dim,
                 layers=1, dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        shape = (layers, n_blocks, block_size, kv_heads, head_dim)
        e = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device=dev)  # noqa: E731
        self.block_size, self.max_tokens = int(block_size), int(max_tokens)
        self.k = torch.zeros(shape, dtype=dtype, device=dev)
        self.v = torch.zeros(shape, dtype=dtype, device=dev)
        self.block_table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device=dev)
        self.free_ids = e(n_blocks)
        self.maps = PagedPlan(e(batch), e(4), e(batch + 1), e(max_tokens), e(max_tokens),
                              e(max_tokens, torch.int64))
        with _on(self.k.device, None):
            rc = load().rq_paged_pool_init(n_blocks, self.maps.pool.data_ptr(), self.free_ids.data_ptr(),
                                           _current_stream(self.k.get_device()))
        if rc != RQ_OK:
            _fail("rq_paged_pool_init", rc)

    def plan(self, new_lens, stream=None) -> PagedPlan:
        """Add new_lens [batch] tokens (-1: the request has ended), in place."""
        m = self.maps
        return paged_plan(new_lens, m.lens, m.pool, self.free_ids, self.block_table,
                          self.block_size, self.max_tokens, out=m, stream=stream)

    def append(self, layer, qkv, **kw):
        """The step's rows qkv [T][...], T <= max_tokens, into layer `layer` -> queries."""
        T = qkv.shape[0]
        return paged_append(qkv, self.k[layer], self.v[layer], self.maps.positions[:T],
                            self.maps.slots[:T], **kw)

    def attend(self, layer, q, **kw):
        """Each of the step's tokens over its own request, q [T][heads * head_dim].  With n new
        tokens of a request in the step and a table that is a ring, the window has to leave
        them room: (max_blocks - 1) * block_size + 1 >= window + n - 1."""
        T = q.shape[0]
        return paged_attention(q, self.k[layer], self.v[layer], self.block_table,
                               self.maps.positions[:T], requests=self.maps.requests[:T], **kw)

    def status(self):
        """(why the last plan did nothing: RQ_PAGED_* bits, 0 if it did; free blocks).
        Synchronizes."""
        head, count, status, taken = self.maps.pool.tolist()
        return status, count
