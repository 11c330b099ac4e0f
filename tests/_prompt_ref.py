"""Plain references of the attention layers' prompt path and of the cache's upkeep (chunk attention, norms and rotation,
forks, releases, copies, kept paths): 64 bits, or plain loops over whole numbers.  CPU only."""
import math

import numpy as np
import torch


# ------------------------------------------------------------------ chunk attention
def chunk_attention(q, k_cache, v_cache, table, ctx, cu, scale):
    """(out, bound, mass) in fp64, [T, Hq, D]: the definition; an elementwise bound of the error that fp32 arithmetic
    may leave (without the dtype's own roundings); sum of weights * |v|.  Tokens whose page is not there are left out."""
    q, kc, vc = (x.detach().cpu().double() for x in (q, k_cache, v_cache))
    T, H, D = q.shape
    P, ps, Hk, _ = kc.shape
    out, bound, mass = (torch.zeros(T, H, D, dtype=torch.float64) for _ in range(3))
    for b in range(len(ctx)):
        n, first, m = int(ctx[b]), int(cu[b]), int(cu[b + 1]) - int(cu[b])
        if m == 0:
            continue
        t = torch.arange(n + m)
        page = table[b].long()[t // ps]
        there = (page >= 0) & (page < P)
        page = torch.where(there, page, 0)
        sees = (t[None] <= n + torch.arange(m)[:, None]) & there          # [m, n + m]
        gone = ~sees.any(0)
        for h in range(H):
            k, v = kc[page, t % ps, h * Hk // H], vc[page, t % ps, h * Hk // H]
            k, v = (torch.where(gone[:, None], 0.0, x) for x in (k, v))
            x = q[first:first + m, h]
            s = (x @ k.T) * scale
            ds = (D + 4) * 2.0 ** -24 * abs(scale) * torch.where(sees, x.abs() @ k.abs().T, 0.0).amax(1) + 2.0 ** -23 * torch.where(sees, s.abs(), 0.0).amax(1)
            w = torch.softmax(s.masked_fill(~sees, -math.inf), 1)
            w = torch.where(sees.any(1, keepdim=True), w, 0.0)
            rows = slice(first, first + m)
            out[rows, h] = w @ v
            mass[rows, h] = w @ v.abs()
            bound[rows, h] = (2 * ds + 2.0 ** -19 + sees.sum(1) * 2.0 ** -23)[:, None] * mass[rows, h]
    return out, bound, mass


def paged(lens, Hk, D, dtype, ps, seed=0, poison=True, spare=3):
    """(cache [P, 2, ps, Hk, D], table): rows of that many tokens; what no row owns is NaN (poison)."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // ps) for n in lens]
    P, cols = sum(pages) + spare, max(pages) + 1
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(lens), cols), 0x7fffffff, dtype=torch.int32)
    kv = torch.full((P, 2, ps, Hk, D), float("nan") if poison else 0.0)
    at = 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        if n:
            t = torch.arange(n)
            kv[table[b].long()[t // ps], :, t % ps] = torch.randn(n, 2, Hk, D, generator=g)
    return kv.to(dtype), table


# ------------------------------------------------------------------ norms and rotation
def norm_rotate(x, positions, freq, weight, eps, norm=True, interleaved=False):
    """(y, bound) in fp64: the definition, and the error that fp32 arithmetic may leave.  A norm's factor: a sum of D
    squares, a mean, a root, a quotient; two products with it and the weight: (D + 8) half-ulps at most.  A rotation: the sine and the
    cosine within 2^-22 (a few ulp of the functions at 1, and the angle to 2^-31 of a turn), two products and a sum."""
    y = x.detach().cpu().double()
    D, R = y.shape[-1], 2 * freq.numel()
    rel = 0.0
    if norm:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double()
        rel = (D + 8) * 2.0 ** -24
    bound = rel * y.abs()
    if R:
        angle = positions.double()[:, None, None] * freq.double()
        c, s = angle.cos(), angle.sin()
        a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        p, q = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = p * c - q * s, p * s + q * c
        turn = (p.abs() + q.abs()) * (rel + 2.0 ** -22 + 3 * 2.0 ** -24)
        bound[..., a], bound[..., b] = turn, turn
    return y, bound


# ------------------------------------------------------------------ pages
def page_fork(parents, children, lens, held, table, shares, free, ps):
    """(held, table, shares, copies, taken, bad) from loops over the forks."""
    held, table, shares = list(held), np.array(table), list(shares)
    R, cols = table.shape
    before, old = list(held), table.copy()
    copies, used, short, bad = [], 0, False, False
    kids = [c for c in children if 0 <= c < R]
    for p, c, n in zip(parents, children, lens):
        ok = 0 <= p < R and 0 <= c < R and n >= 0 and p not in kids and kids.count(c) == 1
        ok = ok and before[c] == 0 and 0 <= before[p] <= cols and before[p] * ps >= n
        copies.append((-1, -1, 0))
        if not ok:
            bad = True
            continue
        full, rest = divmod(n, ps)
        if rest:
            if short or used >= len(free):
                short = True
                continue
            table[c, full] = free[used]
            s, d = int(old[p, full]), int(free[used])
            used += 1
            if 0 <= s < len(shares) and 0 <= d < len(shares):
                copies[-1] = (s, d, rest)
            else:
                bad = True
        for j in range(full):
            table[c, j] = old[p, j]
            if 0 <= old[p, j] < len(shares):
                shares[old[p, j]] += 1
            else:
                bad = True
        held[c] = full + (rest > 0)
    return held, table, shares, copies, used, bad


def page_release(keep, held, table, shares, ps):
    """(held, shares, freed, bad) from loops over the rows."""
    start, now, out, bad = list(shares), list(shares), [], False
    cols, P = table.shape[1], len(shares)
    for r, (k, h) in enumerate(zip(keep, held)):
        out.append(h)
        if k < 0 or h < 0 or h > cols:
            bad = True
            continue
        pages = -(-k // ps)
        if pages > h:
            continue
        if k % ps:
            last = int(table[r][pages - 1])
            if not 0 <= last < P or start[last] > 0:
                bad = True
                continue
        out[-1] = pages
        for j in range(pages, h):
            p = int(table[r][j])
            if 0 <= p < P:
                now[p] -= 1
            else:
                bad = True
    freed = [p for p in range(P) if now[p] < 0]
    bad |= any(s < -1 for s in now)
    return out, [max(s, 0) for s in now], freed, bad


def cache_copy(copies, cache, ps):
    """cache [L, P, 2, ps, H, D] (a copy, changed)."""
    c = cache.clone()
    for s, d, n in copies:
        c[:, d, :, :n] = cache[:, s, :, :n]
    return c


def keep_path(slots, path, n, cache):
    """cache [L, P, 2, ps, H, D] (a copy, changed)."""
    c, ps = cache.clone(), cache.shape[3]
    for b in range(len(n)):
        for e in range(int(n[b])):
            s, d = int(slots[b][int(path[b][e])]), int(slots[b][e])
            c[:, d // ps, :, d % ps] = cache[:, s // ps, :, s % ps]
    return c
