"""The long-context calls where their kernels have long work, against sums in 64 bits on the GPU. A CTA of the
tensor cores' prefix kernel has a share of all tiles (128 keys for bf16 queries, 64 for f32 ones) of all units (128
queries of a group and K/V head): what a case gives each is worked out and asserted."""
import math

import pytest
import torch

from rq_transformer_frame_gb300 import binding, paged

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


class Prefixes:
    """A bf16 cache with a request for each row, of own[r] positions, and one for each group's prefix, in blocks of
    any order; what lies behind their ends is NaN and infinite. sizes: rows of each group."""

    def __init__(self, sizes, prefix, own, heads, hk, hd, io, P=16, seed=0, q_scale=1.0, keys=None, values=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.prefix, self.own, self.heads, self.hk, self.hd, self.P = sizes, prefix, own, heads, hk, hd, P
        R, lens = len(own), own + prefix
        pages = [-(-n // P) for n in lens]
        # wide enough for the tensor cores' kernel: more than 32 MB that the rows might read
        W = max(max(pages) + 1, 32_000_000 // (4 * R * hk * hd * P) + 2)
        self.first = [0]
        for n in pages:
            self.first.append(self.first[-1] + n)
        N = self.first[-1] + 1
        self.order = torch.randperm(N, generator=g, device="cuda")
        table = torch.full((len(lens), W), -1, dtype=torch.int32)
        order = self.order.cpu()
        for b, n in enumerate(pages):
            table[b, :n] = order[self.first[b]:self.first[b] + n]
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.k, self.v = rnd(N, P, hk, hd).to(BF16), rnd(N, P, hk, hd).to(BF16)
        if keys is not None or values is not None:  # f(position of a request as [n, 1, 1], [n][hk][hd]) of its own
            for b in range(len(lens)):
                at, pos = self._at(b)
                if keys is not None:
                    self.k[at] = keys(pos, self.k[at])
                if values is not None:
                    self.v[at] = values(pos, self.v[at])
        live = torch.zeros(N, P, dtype=torch.bool, device="cuda")
        for b in range(len(lens)):
            live[self._at(b)[0]] = True
        self.k[~live], self.v[~live] = NAN, INF
        self.q = (rnd(R, heads * hd) * q_scale).to(io)
        cu = [0]
        for n in sizes:
            cu.append(cu[-1] + n)
        self.group = [i for i, n in enumerate(sizes) for _ in range(n)] + [-1] * (R - cu[-1])
        self.table = table.cuda()
        self.words = (ints([n - 1 for n in own]), ints(cu), ints([R + i for i in range(len(sizes))]), ints(prefix))
        self.R = R

    def _at(self, b):
        """(block, row) of request b's positions, and these."""
        pos = torch.arange((self.own + self.prefix)[b], device="cuda")
        return (self.order[self.first[b] + pos // self.P], pos % self.P), pos.view(-1, 1, 1)

    def run(self, q=None, **kw):
        pos, cu, preq, plen = self.words
        return paged.paged_prefix_attention(self.q if q is None else q, self.k, self.v, self.table, pos, cu, preq, plen,
                                            lse=True, **kw)

    def of_a_cta(self):
        """(tiles, units) that a CTA of 152 meets, about."""
        units = [-(-n * (self.heads // self.hk) // 128) * self.hk for n in self.sizes]
        tiles = [-(-n // (128 if self.q.dtype is BF16 else 64)) for n in self.prefix]
        return sum(a * b for a, b in zip(units, tiles)) / 152, sum(units) / 152

    def exact(self, rows):
        """For each of the rows: out, mass = sum p |v| [heads][hd], lse, norm [heads] in 64 bits."""
        G, scale = self.heads // self.hk, self.hd ** -0.5
        by_group = {}
        for r in rows:
            by_group.setdefault(self.group[r], []).append(r)
        out = {}
        for g, some in by_group.items():
            at = self._at(self.R + g)[0] if g >= 0 else None
            for h in range(self.hk):
                pk = self.k[at][:, h].double() if g >= 0 else self.k.new_zeros(0, self.hd, dtype=F64)
                pv = self.v[at][:, h].double() if g >= 0 else pk
                for i in range(0, len(some), 64):
                    part = some[i:i + 64]
                    q = self.q[part].view(len(part), self.hk, G, self.hd)[:, h].double()
                    s = (q.reshape(-1, self.hd) @ pk.T * scale).view(len(part), G, -1)
                    top = s.amax(-1) if s.shape[-1] else s.new_full(s.shape[:2], -INF)
                    e = torch.exp(s - top[..., None])
                    l, o, m = e.sum(-1), e @ pv, e @ pv.abs()  # noqa: E741
                    for j, r in enumerate(part):
                        own = self._at(r)[0]
                        ok, ov = self.k[own][:, h].double(), self.v[own][:, h].double()
                        t = q[j] @ ok.T * scale
                        most = torch.maximum(top[j], t.amax(-1)) if t.shape[-1] else top[j]
                        f, x = torch.exp(top[j] - most), torch.exp(t - most[:, None])
                        f = torch.where(top[j] == -INF, 0.0, f)
                        total = l[j] * f + x.sum(-1)
                        norm = q[j].norm(dim=-1) * torch.cat([pk, ok]).norm(dim=-1).max() * scale
                        out.setdefault(r, []).append((
                            (o[j] * f[:, None] + x @ ov) / total[:, None], (m[j] * f[:, None] + x @ ov.abs()) / total[:, None],
                            most + torch.log(total), norm))
        return {r: [torch.cat(x) for x in zip(*heads)] for r, heads in out.items()}


# ---------------------------------------------------------------- sums over long pieces
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("sign", ["one sign", "any"])
def test_long_sums_are_those_of_f32(hd, sign):
    """256 rows behind 50000 positions: pieces of hundreds of tiles. bf16 outputs are the exact ones rounded, but
    for those that lie so near the middle of two bf16 values that the f32 sums decide: a share of err / step, the
    step at least 2^-8 of the value. err, on average: 24 products a tile cut by half a step of half the tile's sum,
    24 / 4 * 2^-23; 165 to 330 tiles added to the sums, and to l, each rounded: twice 2^-24 sqrt(330) / 3; weights of
    24 bits from scores off by some 2^-21: 2^-19 in all, so values of one sign have a share of 2^-11. Values
    of any sign leave outputs around 0, where the step is finer than err's own scale: with outputs of normal
    distribution and size 1, E min(1, err / |o|) is about 2 phi(0) err (1 + ln(1 / err)) = 11 err, 2^3.5 times as
    much. (With weights of 16 bits and one sum cut along all tiles the shares were 2^-5.7 and 2^-6.3.) f32 outputs
    are within 2^-19 of the values on average."""
    f = 1 + torch.rand(8, hd, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    values = (lambda pos, v: (1 + v.abs().float().clamp(max=2) / 2).mul(f).to(BF16)) if sign == "one sign" else None
    for io in (BF16, F32):
        c = Prefixes([256], [50000], [0] * 256, 32, 8, hd, io, seed=3, q_scale=1.5, values=values)
        assert c.of_a_cta()[0] > 150
        out, lse = c.run()
        want = c.exact(range(256))
        o = torch.stack([want[r][0] for r in range(256)]).view(256, -1)
        if io is BF16:
            share = (out != o.to(BF16)).double().mean().item()
            print("share", share, math.log2(share) if share else None)
            assert share <= 2.0 ** (-11 if sign == "one sign" else -7.5)
            assert ((out.double() - o).abs() <= o.abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-6).all()
        else:
            err = ((out.double() - o).abs().mean() / o.abs().mean()).item()
            print("error", err, math.log2(err))
            assert err <= 2.0 ** -19
        exact_lse = torch.stack([want[r][2] for r in range(256)])
        assert ((lse.double() - exact_lse).abs() <= 2.0 ** -19 + 2 * U * exact_lse.abs()).all()


# ---------------------------------------------------------------- many tiles, many units
def check(c, out, lse, rows):
    """Against the exact rows, with the tolerances of test_paged_long_gpu.py (scores at most norm)."""
    e, part = torch.finfo(out.dtype).eps / 2, 2.0 ** -16 if out.dtype is BF16 else 0.0
    out, lse = out.double().view(c.R, c.heads, c.hd), lse.double()
    for r, (o, mass, exact_lse, norm) in c.exact(rows).items():
        n = c.own[r] + (c.prefix[c.group[r]] if c.group[r] >= 0 else 0)
        ds = U * (8 * math.sqrt(c.hd) + 8) * norm
        sums = U * (4 * math.sqrt(n) + 16)
        join = 2 * (ds + sums + 4 * U * (exact_lse.abs() + norm))
        tol = (2 * ds + sums + part + join)[:, None] * mass * (1 + e) + e * o.abs() + 1e-30
        err = (out[r] - o).abs()
        assert (err <= tol).all(), (r, float((err / tol).max()))
        assert ((lse[r] - exact_lse).abs() <= ds + sums + join / 2 + 4 * U * exact_lse.abs()).all(), r


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("P", [5, 16, 128])
def test_many_tiles(hd, io, P):
    """More tiles a CTA than its ring and its masks hold, in pieces that are cut: blocks by TMA and by copies."""
    c = Prefixes([64], [27000], [1 + r % 40 for r in range(64)], 32, 8, hd, io, P=P, seed=hd + P)
    assert c.of_a_cta()[0] > 20
    check(c, *c.run(), range(64))


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("P", [5, 16])
def test_many_units(hd, io, P):
    """More than twenty units a CTA: 420 groups of one row behind one to four tiles (more groups than a CTA has
    threads), two of 30 rows behind a hundred, and rows behind none."""
    sizes = [1] * 200 + [30] + [1] * 220 + [30]
    prefix = [1 + i * 53 % 250 for i in range(200)] + [9000] + [1 + i * 91 % 250 for i in range(220)] + [7777]
    own = [i * 7 % 23 for i in range(sum(sizes) + 3)]
    c = Prefixes(sizes, prefix, own, 16, 8, hd, io, P=P, seed=hd + P)
    assert c.of_a_cta()[1] > 20 and len(sizes) > 384
    rows = [0, 1, 199] + list(range(200, 230, 7)) + list(range(230, 450, 13)) + [449, 450, 479, 480, 481, 482]
    check(c, *c.run(), [r for r in rows if own[r] or c.group[r] >= 0])


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise(io, rising):
    """Scores that grow along the prefix, so that the bound moves and sums are scaled again and again, or that
    shrink, so that the first tiles' stays."""
    n = 27000
    grow = lambda pos: 0.1 + 3 * (pos if rising else n - pos) / n  # noqa: E731
    c = Prefixes([40, 24], [n, n], [3] * 64, 32, 8, 64, io, seed=5, keys=lambda pos, k: (k.float() * grow(pos)).to(BF16))
    assert c.of_a_cta()[0] > 20
    check(c, *c.run(), range(0, 64, 3))


@pytest.mark.parametrize("P", [5, 8])
@pytest.mark.parametrize("io", [F32, BF16])
def test_prefix_past_32_bits(P, io):
    """Blocks past 2^32 elements in the tensor cores' kernel: whole boxes and the rows of one that is torn by the
    prefix's end (blocks of 8), and copies (blocks of 5)."""
    hd, W, stride = 32, 40000, 2**31 + 64
    big_k, big_v = (torch.zeros(2 * stride + P * hd, dtype=BF16, device="cuda") for _ in range(2))
    k, v = (x.as_strided((3, P, 1, hd), (stride, hd, hd, 1)) for x in (big_k, big_v))
    for x in (k, v):
        x[1:] = torch.randn(2, P, 1, hd, device="cuda").to(BF16)
    n = 2 * P - 3
    k[2, P - 3:], v[2, P - 3:] = NAN, INF
    table = torch.full((3, W), -1, dtype=torch.int32, device="cuda")
    table[2, :2] = ints([1, 2])
    assert 4 * 2 * hd * W * P > 32e6
    q = torch.randn(2, 4 * hd, device="cuda").to(io)
    got, got_lse = paged.paged_prefix_attention(q, k, v, table, ints([-1, -1]), ints([0, 2]), ints([2]), ints([n]), lse=True)
    kk, vv = (torch.cat([x[1, :, 0], x[2, :P - 3, 0]]).double() for x in (k, v))
    s = q.double().view(2, 4, hd) @ kk.T * hd ** -0.5
    want = (torch.softmax(s, -1) @ vv).view(2, -1)
    mass, e = (torch.softmax(s, -1) @ vv.abs()).view(2, -1), torch.finfo(io).eps / 2
    # scores at most norm: their f32 sums, weights and their sum, the store, as in check
    norm = q.double().view(2, 4, hd).norm(dim=-1).max() * kk.norm(dim=-1).max() * hd ** -0.5
    tol = U * (4 * (8 * math.sqrt(hd) + 8) * norm + 100)
    assert ((got.double() - want).abs() <= tol * mass * (1 + e) + e * want.abs()).all()
    assert ((got_lse.double() - torch.logsumexp(s, -1)).abs() <= tol).all()


def test_select_of_many_rows():
    """More rows than one launch has in y: three pages, of which the last is taken and one of the others."""
    R, hd, P = 66000, 32, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    mid = torch.randn(50, 1, 1, hd, generator=g, device="cuda")
    bounds = torch.cat([mid - 1, mid + 1], 2)
    table = torch.randint(0, 50, (R, 3), generator=g, device="cuda").to(torch.int32)
    q = torch.randn(R, hd, generator=g, device="cuda")
    pages = paged.paged_select(q, bounds, table, ints([3 * P - 1]).repeat(R), P, 2, first=0, last=1)
    b, x = bounds.double()[:, 0], q.double()
    score = ((x.clamp(min=0)[:, None] * b[table[:, :2].long(), 1]).sum(-1) +
             (x.clamp(max=0)[:, None] * b[table[:, :2].long(), 0]).sum(-1))
    best = (score[:, 1] > score[:, 0]).to(torch.int32)
    assert torch.equal(pages[:, 0], torch.stack([best, torch.full_like(best, 2)], 1))


# ---------------------------------------------------------------- a wait that runs out
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("P", [5, 16])
def test_a_wait_that_runs_out_is_reported(io, P):
    """One thread block never gets its prefix: after 20 ms its waits run out, the call says so, the rows that hang on
    it are NaN and no others; the calls before and behind it are as ever."""
    c = Prefixes([64], [9000], [1 + r % 9 for r in range(64)], 16, 8, 64, io, P=P, seed=P)
    L = binding.load()
    ws = paged.paged_prefix_attention_workspace(c.q, c.k, c.table, c.words[3])
    ws.fill_(0xff)
    out, lse = c.run(workspace=ws)
    assert paged.paged_prefix_attention_status(ws) == 0 and out.isfinite().all()
    try:
        assert L.rq_paged_set_wait_limit(20_000_000, -2) == binding.RQ_ERR_ARG
        assert L.rq_paged_set_wait_limit(20_000_000, 0) == binding.RQ_OK
        bad, bad_lse = c.run(workspace=ws)
        assert paged.paged_prefix_attention_status(ws) == binding.RQ_PAGED_TIMEOUT
    finally:
        L.rq_paged_set_wait_limit(0, -1)
    # the first thread block has tiles of the first K/V head's queries alone: two heads of all rows
    gone = torch.zeros(64, 16, dtype=torch.bool, device="cuda")
    gone[:, :2] = True
    assert torch.equal(bad_lse.isnan(), gone) and torch.equal(bad_lse[~gone], lse[~gone])
    bad, out = bad.view(64, 16, 64), out.view(64, 16, 64)
    assert bad[gone].isnan().all() and torch.equal(bad[~gone], out[~gone])
    again, again_lse = c.run(workspace=ws)
    assert paged.paged_prefix_attention_status(ws) == 0
    assert torch.equal(again.view(64, 16, 64), out) and torch.equal(again_lse, lse)


def test_status_of_the_other_forms():
    """Rows each for itself, and no groups at all: nothing there waits, and the status says so."""
    k, v = (torch.randn(6, 8, 2, 64, device="cuda") for _ in range(2))
    q, table, pos, one = torch.randn(2, 4 * 64, device="cuda"), ints([[0, 1], [2, 3], [4, 5]]), ints([9, 15]), ints([2])
    for cu, group, n in ((ints([0, 2]), one, ints([11])), (ints([0]), ints([]), ints([]))):
        ws = paged.paged_prefix_attention_workspace(q, k, table, n)
        ws.fill_(0xff)
        out, _ = paged.paged_prefix_attention(q, k, v, table, pos, cu, group, n, workspace=ws)
        assert paged.paged_prefix_attention_status(ws) == 0
        captured = torch.zeros_like(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            paged.paged_prefix_attention(q, k, v, table, pos, cu, group, n, out=captured, workspace=ws)
        ws.fill_(0xff)
        graph.replay()
        assert paged.paged_prefix_attention_status(ws) == 0 and torch.equal(captured, out)
    none = paged.paged_prefix_attention_workspace(q[:0], k, table, one)
    paged.paged_prefix_attention(q[:0], k, v, table, pos, ints([0, 0]), one, one, workspace=none)
    assert paged.paged_prefix_attention_status(none) == 0


# ---------------------------------------------------------------- behind a shared prompt
@pytest.mark.parametrize("rope", ["interleaved", "halves"])
@pytest.mark.parametrize("io", [F32, BF16])
def test_rotations_behind_a_shared_prompt(rope, io):
    """Two prompts appended once, then steps of requests behind them, through PagedCache alone: the queries, keys and
    results of requests that hold all of it themselves."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, P, hk, H, hd = 5, 8, 2, 4, 64
    plen = [37, 90]
    of = [0, 0, 0, 1, 1]  # each request's prompt
    c = paged.PagedCache(B + 2, 400, P, 60, 512, hk, hd, layers=2, dtype=io)
    whole = paged.PagedCache(B, 400, P, 60, 512, hk, hd, layers=2, dtype=io)
    prompts = [torch.randn(n, (H + 2 * hk) * hd, generator=g, device="cuda").to(io) for n in plen]
    c.plan(ints([0] * B + plen))
    whole.plan(ints([plen[i] for i in of]))
    for layer in range(2):
        c.append(layer, torch.cat(prompts), rope=rope)
        whole.append(layer, torch.cat([prompts[i] for i in of]), rope=rope)
    behind = ints([plen[i] for i in of] + [0, 0])
    for new in ([3, 1, 9, 2, 5], [1] * B, [1, 2, 1, 1, 4]):
        T, n = sum(new), sum(new[:3])
        qkv = torch.randn(T, (H + 2 * hk) * hd, generator=g, device="cuda").to(io)
        c.plan(ints(new + [0, 0]))
        whole.plan(ints(new))
        at = c.maps.positions[:T] + behind[c.maps.requests[:T]]
        for layer in range(2):
            q = c.append(layer, qkv, positions=at, rope=rope)
            q2 = whole.append(layer, qkv, rope=rope)
            assert torch.equal(q, q2)
            out, lse = c.attend_prefix(layer, q, ints([0, n, T]), ints([B, B + 1]), ints(plen), lse=True)
            want, want_lse = whole.attend(layer, q2, lse=True)
            assert (out.double() - want.double()).abs().max() <= 4 * torch.finfo(io).eps * want.double().abs().max() + \
                1e-5 * (io is F32)
            assert torch.allclose(lse, want_lse, rtol=1e-5)
