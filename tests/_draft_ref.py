"""Plain 64-bit references of the draft-step operators (page tables, tree attention, KDA on a
draft tree, draft verification) and the trees the tests run them on.  CPU only."""
import numpy as np
import torch

import oracle

PAD = -2


def trees(kind, batch, nodes, seed=0):
    """parents [batch, nodes] int32: 'chain', 'star' (all on the context), 'binary', 'random'
    or 'ragged' (random, with sequence b ending early; absent nodes in the middle too)."""
    r = np.random.default_rng(seed)
    i = np.arange(nodes)
    if kind == "chain":
        p = i - 1
    elif kind == "star":
        p = np.full(nodes, -1)
    elif kind == "binary":
        p = (i + 1) // 2 - 1
    else:
        p = np.stack([[int(r.integers(-1, j)) if j else -1 for j in range(nodes)] for _ in range(batch)])
    p = np.broadcast_to(p, (batch, nodes)).astype(np.int32).copy()
    if kind == "ragged":
        for b in range(batch):
            p[b, max(1, nodes - b - 1):] = PAD
            if nodes > 4:
                gone = 1 + b % (nodes - 2)
                p[b, gone] = PAD
                p[b][p[b] == gone] = -1
    return p


def path_to(parents, i):
    up = []
    while i >= 0:
        up.append(i)
        i = int(parents[i])
    return up[::-1]


# ------------------------------------------------------------------ attention
def attention(q, k_cache, v_cache, table, ctx, parents, scale):
    """(out, bound) in fp64, [B, K, Hq, D]: the definition, and an elementwise bound of the error that fp32
    arithmetic with the stated roundings may leave (without the dtype's own roundings), as weights * |v|."""
    q, kc, vc = (x.detach().cpu().double() for x in (q, k_cache, v_cache))
    B, K, H, D = q.shape
    P, ps, Hk, _ = kc.shape
    G = H // Hk
    out, bound = torch.zeros(B, K, H, D, dtype=torch.float64), torch.zeros(B, K, H, D, dtype=torch.float64)
    mass = torch.zeros_like(out)
    for b in range(B):
        n = int(ctx[b])
        for i in range(K):
            if parents[b][i] == PAD:
                continue
            pos = list(range(n)) + [n + j for j in path_to(parents[b], i)]
            pos = [t for t in pos if 0 <= int(table[b][t // ps]) < P]
            if not pos:
                continue
            t = torch.tensor(pos)
            pages = torch.as_tensor(table[b]).long()[t // ps]
            for h in range(H):
                k, v = kc[pages, t % ps, h // G], vc[pages, t % ps, h // G]
                s = (k @ q[b, i, h]) * scale
                w = torch.softmax(s, 0)
                ds = (D + 4) * 2.0 ** -24 * abs(scale) * (k.abs() @ q[b, i, h].abs()).max() + 2.0 ** -23 * s.abs().max()
                out[b, i, h] = w @ v
                mass[b, i, h] = w @ v.abs()
                bound[b, i, h] = (2 * ds + 2.0 ** -19 + len(pos) * 2.0 ** -23) * mass[b, i, h]
    return out, bound, mass


# ------------------------------------------------------------------ KDA on a tree
def kda_tree(x, state0, parents):
    """(out, writes, states) in fp64 from the recurrence along every node's own path: out, writes
    [B, K, H, dv]; states [B][node] = [H, dk, dv].  x: q, k, v, g, beta [B, K, H, .] (CPU)."""
    B, K, H, D = x["k"].shape
    paths = [(b, path_to(parents[b], i)) for b in range(B) for i in range(K) if parents[b][i] != PAD]
    pick = lambda t: torch.cat([t[b, p] for b, p in paths]).contiguous()
    cu = np.concatenate([[0], np.cumsum([len(p) for _, p in paths])]).astype(np.int32)
    s0 = torch.stack([state0[b] for b, _ in paths])
    o, s = oracle.recurrent(pick(x["q"]), pick(x["k"]), pick(x["v"]), pick(x["g"]), pick(x["beta"]), cu, s0)
    out, writes = np.zeros((B, K, H, D)), np.zeros((B, K, H, D))
    states = [dict() for _ in range(B)]
    f64 = lambda t: t.double().numpy()
    for n, (b, p) in enumerate(paths):
        states[b][p[-1]] = s[n]
        out[b, p[-1]] = o[cu[n + 1] - 1]
    for b, p in paths:
        i = p[-1]
        before = f64(state0[b]) if len(p) == 1 else states[b][p[-2]]
        decayed = np.exp(f64(x["g"][b, i]))[:, :, None] * before
        writes[b, i] = f64(x["beta"][b, i])[:, None] * (f64(x["v"][b, i]) - np.einsum("hcd,hc->hd", decayed, f64(x["k"][b, i])))
    return out, writes, states


# ------------------------------------------------------------------ verification
def verify(target, draft, tokens, parents, u, noise):
    """(path, n_accept, next_token): the rule, one IEEE fp32 operation at a time (numpy)."""
    B, K = tokens.shape
    path, count, nxt = np.full((B, K), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    f = np.float32
    for b in range(B):
        cur, mass, down = -1, f(1), []
        for c in range(K):
            if parents[b, c] != cur:
                continue
            x, p = tokens[b, c], target[b, cur + 1, tokens[b, c]]
            if draft is None:
                if x in [tokens[b, d] for d in down]:
                    continue
                keep = u[b, c] * mass < p
            else:
                keep = u[b, c] * draft[b, c, x] < p
            if keep:
                path[b, count[b]] = c
                count[b] += 1
                cur, mass, down = c, f(1), []
            else:
                down.append(c)
                mass = f(mass - p)
        p = target[b, cur + 1]
        rest = p.copy()
        if draft is None:
            rest[[tokens[b, d] for d in down]] = 0
        elif down:
            rest = np.maximum(p - draft[b, down[0]], f(0))
        if not (rest > 0).any():
            rest = p
        nxt[b] = int(np.argmax(rest / noise[b]))
    return path, count, nxt


# ------------------------------------------------------------------ page tables
def page_tables(ctx, new, held, table, free, ps, max_tokens):
    """(slots, cu, held_out, taken, table): one request after the other."""
    table, slots, cu, out, used, open_ = table.copy(), [], [0], [], 0, True
    cols = table.shape[1]
    for b in range(len(ctx)):
        need = max(0, -(-(int(ctx[b]) + int(new[b])) // ps) - int(held[b]))
        fits = int(ctx[b]) + int(new[b]) <= cols * ps
        if fits and need > 0:
            if open_ and used + need <= len(free):
                table[b, held[b]:held[b] + need] = free[used:used + need]
                used += need
            else:
                open_, fits = False, False
        out.append(int(held[b]) + (need if fits else 0))
        for t in range(int(ctx[b]), int(ctx[b]) + int(new[b])):
            slots.append(int(table[b, t // ps]) * ps + t % ps if fits else -1)
        cu.append(len(slots))
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return np.array(slots, np.int64), np.array(cu, np.int32), np.array(out, np.int32), used, table
