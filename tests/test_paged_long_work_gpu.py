"""The long-context calls where their kernels have long work, against sums in 64 bits on the GPU. A CTA of the
tensor cores' prefix kernel has a share of all tiles (128 keys for bf16 queries, 64 for f32 ones) of all units (128
queries of a group and K/V head): what a case gives each is worked out and asserted."""
import math

import pytest
import torch

from rq_transformer_frame_gb300 import paged

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
