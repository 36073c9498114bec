"""Plain implementations of the calls for long paged contexts, in 64 bits, one row, one page and one
key after another."""
import numpy as np
import torch


def bounds(k, old, positions, slots):
    """rq_paged_bounds on CPU tensors: k [N][P][hk][hd], old [N][hk][2][hd] (copied)."""
    N, P = k.shape[:2]
    out = old.clone()
    ends = {}
    for p, s in zip(positions, slots):
        if p >= 0 and 0 <= s < N * P:
            ends[s // P] = s % P  # the last token of the block stands last
    for b, o in ends.items():
        rows = k[b, :o + 1]
        nan = rows.isnan().any(0)
        lo, hi = rows.double().amin(0), rows.double().amax(0)
        for i, x in enumerate((lo, hi)):
            out[b, :, i] = torch.where(nan, float("nan"), x).to(k.dtype)
    return out


def select(q, bounds_, table_row, pos, P, top, first, last):
    """The pages of one row: q [heads][hd] f64 -> a list of lists, one for each K/V head."""
    N, hk, _, hd = bounds_.shape
    W, G = len(table_row), q.shape[0] // hk
    if pos < 0:
        return [[] for _ in range(hk)]
    newest = pos // P
    live = list(range(max(0, newest - W + 1), newest + 1))
    fixed = sorted(set(live[:first]) | set(live[len(live) - min(last, len(live)):]))
    others = [p for p in live if p not in fixed and 0 <= table_row[p % W] < N]
    want = top - first - last if len(live) > top else len(others)
    lists = []
    for h in range(hk):
        up = q[h * G:(h + 1) * G].clamp(min=0).sum(0)
        down = q[h * G:(h + 1) * G].clamp(max=0).sum(0)
        scored = []
        for p in others:
            b = bounds_[table_row[p % W], h].double()
            s = float((up * b[1] + down * b[0]).sum())
            scored.append((-np.inf if s != s else s, p))
        scored.sort(key=lambda x: (-x[0], x[1]))
        lists.append(sorted(fixed + [p for _, p in scored[:want]]))
    return lists


def attend_keys(q, kk, vv, scale):
    """q [heads][hd] f64, kk, vv: for each K/V head its keys and values [n][hd] -> dict(out, lse,
    mass = sum p |v|, smax, norm, n [heads]): what the tolerances are made of."""
    heads, hd = q.shape
    G = heads // len(kk)
    out, mass = torch.zeros(heads, hd, dtype=torch.float64), torch.zeros(heads, hd, dtype=torch.float64)
    lse = torch.full((heads,), -float("inf"), dtype=torch.float64)
    smax, norm, n = (torch.zeros(heads, dtype=torch.float64) for _ in range(3))
    for h in range(heads):
        k, v = kk[h // G].double(), vv[h // G].double()
        n[h] = k.shape[0]
        if k.shape[0] == 0:
            continue
        s = k @ q[h] * scale
        top = s.max()
        p = torch.exp(s - top)
        total = p.sum()
        out[h], mass[h] = (p / total) @ v, (p / total) @ v.abs()
        lse[h] = top + torch.log(total)
        smax[h] = s.abs().max()
        norm[h] = q[h].norm() * k.norm(dim=-1).max() * abs(scale)
    return dict(out=out, lse=lse, mass=mass, smax=smax, norm=norm, n=n)


def listed_keys(k, v, table_row, pos, pages):
    """Keys and values of one row's lists: pages [hk][list] -> two lists of [n][hd]."""
    N, P, hk, hd = k.shape
    W = len(table_row)
    kk, vv = [], []
    for h in range(hk):
        at = []
        for p in pages[h]:
            if pos < 0 or p < 0 or p > pos // P or p <= pos // P - W:
                continue
            b = int(table_row[p % W])
            if 0 <= b < N:
                at += [(b, j) for j in range(P) if p * P + j <= pos]
        b, j = (torch.tensor(x, dtype=torch.int64) for x in (zip(*at) if at else ((), ())))
        kk.append(k[b, j, h])
        vv.append(v[b, j, h])
    return kk, vv


def request_keys(k, v, table_row, pos):
    """The live keys and values of a request up to position pos, [n][hk][hd] each."""
    N, P = k.shape[:2]
    W = len(table_row)
    at = []
    if pos >= 0:
        for j in range(max(0, (pos // P - W + 1) * P), pos + 1):
            b = int(table_row[(j // P) % W])
            if 0 <= b < N:
                at.append((b, j % P))
    b, j = (torch.tensor(x, dtype=torch.int64) for x in (zip(*at) if at else ((), ())))
    return k[b, j], v[b, j]
