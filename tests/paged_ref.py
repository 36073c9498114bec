"""Plain implementations of the paged K/V cache's calls: the plan in Python integers, the
append and the attention in 64 bits, one row and one key after another."""
import numpy as np
import torch


def plan(new, lens, pool, free_ids, table, P, M):
    """Python restatement of rq_paged_plan on lists and numpy arrays (copied, not changed)."""
    B, W = table.shape
    N = len(free_ids)
    head, count = int(pool[0]), int(pool[1])
    table, free_ids = table.copy(), free_ids.copy()
    pages = lambda c: min(-(-c // P), W)  # noqa: E731
    bad = not (0 <= head < N and 0 <= count <= N)
    need = give = tokens = 0
    for n, c in zip(new, lens):
        if n < -1 or c < 0 or c + max(n, 0) > 2**31 - 1:
            bad = True
        elif n < 0:
            give += pages(c)
        else:
            need += pages(c + n) - pages(c)
            tokens += n
    status = (1 if bad or count + give > N else 0) | (2 if tokens > M else 0) | (4 if need > count else 0)
    req, pos, slot = np.full(M, -1, np.int32), np.full(M, -1, np.int32), np.full(M, -1, np.int64)
    cu = np.zeros(B + 1, np.int32)
    if status:
        return dict(lens=np.array(lens, np.int32), pool=[head, count, status, need], cu=cu, req=req,
                    pos=pos, slot=slot, table=table, free_ids=free_ids)
    t = took = gave = 0
    out = []
    for b, (n, c) in enumerate(zip(new, lens)):
        cu[b] = t
        if n < 0:
            for i in range(pages(c)):
                free_ids[(head + count + gave) % N] = table[b, i]
                gave += 1
            out.append(0)
            continue
        for col in range(pages(c), pages(c + n)):
            table[b, col] = free_ids[(head + took) % N]
            took += 1
        for j in range(n):
            p = c + j
            req[t], pos[t] = b, p
            block = table[b, (p // P) % W]
            overwritten = p // P + W <= (c + n - 1) // P
            if not overwritten and 0 <= block < N:
                slot[t] = int(block) * P + p % P
            t += 1
        out.append(c + n)
    cu[B] = t
    return dict(lens=np.array(out, np.int32), pool=[(head + took) % N, count - took + gave, 0, took],
                cu=cu, req=req, pos=pos, slot=slot, table=table, free_ids=free_ids)


def rotate(x, pos, rope_dim, style, theta):
    """x [heads][hd] f64 rotated at position pos."""
    y = x.clone()
    for i in range(rope_dim // 2):
        a, b = (2 * i, 2 * i + 1) if style == "interleaved" else (i, i + rope_dim // 2)
        w = pos * float(theta) ** (-2.0 * i / rope_dim)
        c, s = np.cos(w), np.sin(w)
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, a] * s + x[:, b] * c
    return y


def append_row(row, pos, heads, hk, hd, q_alpha, k_alpha, eps, style, rope_dim, theta):
    """One qkv row (f64, on the CPU) -> (q [heads][hd], k [hk][hd], v [hk][hd])."""
    x = row.double().reshape(heads + 2 * hk, hd)
    parts = []
    for y, alpha in ((x[:heads], q_alpha), (x[heads:heads + hk], k_alpha)):
        if alpha is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * alpha.double()
        parts.append(rotate(y, pos, rope_dim, style, theta))
    return parts[0], parts[1], x[heads + hk:]


def live_positions(pos, window, W, P):
    if pos < 0:
        return range(0)
    first = max(0, (pos // P - W + 1) * P)
    if window:
        first = max(first, pos - window + 1)
    return range(first, pos + 1)


def attend_row(q, k, v, table_row, pos, window, scale):
    """q [heads][hd] f64, k, v [N][P][hk][hd] on the CPU -> dict(out, lse, mass = sum p |v|,
    smax, qk): what the tolerances are made of."""
    N, P, hk, hd = k.shape
    W, heads = len(table_row), q.shape[0]
    keys = [(int(table_row[(j // P) % W]), j % P) for j in live_positions(pos, window, W, P)]
    keys = [(b, i) for b, i in keys if 0 <= b < N]
    out = torch.zeros(heads, hd, dtype=torch.float64)
    lse = torch.full((heads,), -float("inf"), dtype=torch.float64)
    mass = torch.zeros(heads, hd, dtype=torch.float64)
    if not keys:
        return dict(out=out, lse=lse, mass=mass, smax=0.0, norm=0.0, n=0)
    b, i = (torch.tensor(x) for x in zip(*keys))
    kk, vv = k[b, i].double(), v[b, i].double()  # [n][hk][hd]
    g = heads // hk
    smax = norm = 0.0
    for h in range(heads):
        s = kk[:, h // g] @ q[h] * scale
        top = s.max()
        p = torch.exp(s - top)
        total = p.sum()
        out[h] = (p / total) @ vv[:, h // g]
        mass[h] = (p / total) @ vv[:, h // g].abs()
        lse[h] = top + torch.log(total)
        smax = max(smax, float(s.abs().max()))
        norm = max(norm, float(q[h].norm() * kk[:, h // g].norm(dim=-1).max()) * abs(scale))
    return dict(out=out, lse=lse, mass=mass, smax=smax, norm=norm, n=len(keys))
