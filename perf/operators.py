"""The operators of a speculative decoding step, as they are measured: cases, inputs, plain forms and exact values.

Four operators work on one draft tree per sequence (``parents`` [B, K]: -1 hangs a node on the context, i < j hangs node
j on node i, -2 marks an absent node):

* ``tables``   pages and slots for the tokens that a step appends to a paged cache;
* ``attn``     softmax attention of the tree's tokens over that cache (the context and each node's own ancestors);
* ``tree``     Kimi Delta Attention of the tree's tokens over the recurrent state (the step, and the commit of a path);
* ``verify``   which drafted tokens the target's probabilities keep, and the token after them.
"""
import math
import random

import numpy as np
import torch

own = False  # True: the framework's kernels; False: the plain forms below

DEV = "cuda"
PAD = -2


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the tables of one draft step of a mid-size batch: a few hundred numbers, so only latency
        {"name": "tables_draft_b48", "op": "tables", "batch": 48, "lo": 1, "hi": 8192, "new_lo": 16, "new_hi": 16, "page": 64},
        # the varlen prompt batch (32 prompts of 512 to 16384 tokens), paged from nothing
        {"name": "tables_prompts_b32", "op": "tables", "batch": 32, "lo": 0, "hi": 0, "new_lo": 512, "new_hi": 16384, "page": 16},
        # one user, a chain of four drafted tokens and a small odd vocabulary: only latency
        {"name": "verify_chain_b1", "op": "verify", "batch": 1, "nodes": 4, "vocab": 32003, "chain": True},
        # a batch of 32-node trees, drafts chosen by rank (no draft distribution)
        {"name": "verify_tree_b64", "op": "verify", "batch": 64, "nodes": 32, "vocab": 131072, "chain": False},
        # the decode workload's 256 sequences, chains of four drawn from a draft model, an odd vocabulary
        {"name": "verify_chain_b256", "op": "verify", "batch": 256, "nodes": 4, "vocab": 100003, "chain": True},
        # plain single-token decode over the cache: four users, short contexts, small pages
        {"name": "attn_one_b4", "op": "attn", "batch": 4, "nodes": 1, "heads": 32, "kv_heads": 8, "dim": 128, "lo": 500, "hi": 1500, "page": 16, "bf16": True},
        # 16-node trees of a ragged batch, twelve query heads to a cache head (the 96 heads of the other layers)
        {"name": "attn_tree_b32", "op": "attn", "batch": 32, "nodes": 16, "heads": 96, "kv_heads": 8, "dim": 128, "lo": 512, "hi": 16384, "page": 64, "bf16": True},
        # 64-node trees over the long workload's 131072 tokens
        {"name": "attn_long_b2", "op": "attn", "batch": 2, "nodes": 64, "heads": 32, "kv_heads": 8, "dim": 128, "lo": 131072, "hi": 131072, "page": 128, "bf16": True},
        # the fp32 path: narrow heads, three query heads to a cache head, odd lengths (0 among them), pages no power of two
        {"name": "attn_f32_b7", "op": "attn", "batch": 7, "nodes": 5, "heads": 6, "kv_heads": 2, "dim": 64, "lo": 0, "hi": 3001, "page": 24, "bf16": False},
        # one user's 6-node tree through a 96-head layer
        {"name": "tree_step_b1", "op": "tree", "batch": 1, "nodes": 6, "heads": 96, "dim": 128, "bf16": True, "commit": False},
        # 64 users' 16-node trees through a 96-head layer
        {"name": "tree_step_b64", "op": "tree", "batch": 64, "nodes": 16, "heads": 96, "dim": 128, "bf16": True, "commit": False},
        # the decode workload's 256 x 96 states moved to the end of each accepted path
        {"name": "tree_commit_b256", "op": "tree", "batch": 256, "nodes": 8, "heads": 96, "dim": 128, "bf16": True, "commit": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "verify", "attn", "attn", "tree", "tree"])
    if op == "tables":
        prompts = rng.random() < 0.5
        batch = _log(rng, 1, 64) if prompts else _log(rng, 1, 3000)
        c = {"op": op, "batch": batch, "page": rng.choice([1, 8, 16, 24, 64, 128, 256])}
        if prompts:
            return {**c, "lo": 0, "hi": rng.choice([0, 4000]), "new_lo": 1, "new_hi": _log(rng, 2, 16384)}
        k = rng.randint(1, 64)
        return {**c, "lo": 0, "hi": _log(rng, 10, 8192), "new_lo": rng.choice([0, k]), "new_hi": k}
    if op == "verify":
        chain = rng.random() < 0.5
        nodes = rng.randint(1, 8) if chain else rng.randint(1, 64)
        vocab = _log(rng, 1000, 160000)
        most = min(256, int(2.5e8 / (vocab * (nodes + 1) * (2 if chain else 1))))
        return {"op": op, "batch": _log(rng, 1, max(1, most)), "nodes": nodes, "vocab": vocab, "chain": chain}
    if op == "attn":
        bf16 = rng.random() < 0.75
        kv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "nodes": _log(rng, 1, 64), "heads": kv * rng.choice([1, 2, 3, 4, 6, 8, 12]), "kv_heads": kv,
             "dim": rng.choice([64, 128]), "page": rng.choice([8, 16, 24, 64, 128, 256]), "bf16": bf16}
        length = _log(rng, 30, 131072 if bf16 else 20000)
        most = min(64, int(5e8 / (c["nodes"] * c["heads"] * length)), int(2.5e5 * 8 / (kv * length)) if bf16 else int(1e10 / (c["nodes"] * c["heads"] * length * c["dim"])))
        return {**c, "batch": _log(rng, 1, max(1, most)), "lo": rng.choice([0, length // 2, length]), "hi": length}
    commit = rng.random() < 0.4
    c = {"op": op, "nodes": _log(rng, 1, 64), "heads": rng.choice([2, 7, 16, 32, 38, 96]), "dim": rng.choice([64, 128, 128]),
         "bf16": rng.random() < 0.75, "commit": commit}
    most = 20000 if commit else min(6000, int(1.5e8 / (c["nodes"] ** 2 * c["dim"])))
    return {**c, "batch": _log(rng, 1, max(1, min(256, most // c["heads"])))}


def _lengths(case, salt, lo, hi, n):
    """n whole numbers of [lo, hi], fixed by the case alone (so that work() knows them); the first is lo, the last hi."""
    r = random.Random("%s %s" % (salt, sorted((k, v) for k, v in case.items() if k != "name")))
    got = [r.randint(lo, hi) for _ in range(n)]
    got[0], got[-1] = lo, hi
    return got


# ------------------------------------------------------------------ inputs
def _trees(batch, nodes, seed, chain=False):
    """parents [batch, nodes]: chains, or trees whose nodes hang on one of the nodes just before them; some end early."""
    r = np.random.RandomState(seed % (1 << 31))
    at = np.tile(np.arange(nodes, dtype=np.int64), (batch, 1))
    back = np.ones((batch, nodes), np.int64) if chain else r.geometric(0.35, (batch, nodes))
    p = np.maximum(at - back, -1)
    used = np.where(r.rand(batch) < 0.75, nodes, r.randint(1, nodes + 1, batch))
    return np.where(at < used[:, None], p, PAD).astype(np.int32)


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _prepare_tables(case, seed, gen):
    B, ps = case["batch"], case["page"]
    ctx = np.array(_lengths(case, "ctx", case["lo"], case["hi"], B))
    new = np.array(_lengths(case, "new", case["new_lo"], case["new_hi"], B))
    r = np.random.RandomState(seed % (1 << 31))
    held = -(-ctx // ps)
    want = -(-(ctx + new) // ps)
    M = int(want.max()) + 2
    ids = r.permutation(int(np.maximum(held, want).sum()) + 5).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    owned = np.arange(M)[None] < held[:, None]
    table[owned] = ids[: int(held.sum())]
    return {"ctx": _gpu(ctx.astype(np.int32)), "new": _gpu(new.astype(np.int32)), "held": _gpu(held.astype(np.int32)),
            "table": _gpu(table), "free": _gpu(ids[int(held.sum()):]), "page": ps, "tokens": int(new.sum()) + 3}


def _prepare_verify(case, seed, gen):
    B, K, V = case["batch"], case["nodes"], case["vocab"]
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)
    noise = lambda *s: torch.empty(s, device=DEV).exponential_(generator=gen).clamp_min_(1e-30)
    parents = _gpu(_trees(B, K, seed, case["chain"]))
    s = {"parents": parents, "u": torch.rand((B, K), generator=gen, device=DEV), "noise": noise(B, V), "draft": None}
    z = rnd(B, K + 1, V) * 4
    s["target"] = torch.softmax(z, -1)
    if case["chain"]:  # the draft model is near the target; its tokens are drawn from it
        s["draft"] = torch.softmax(z[:, :K] + rnd(B, K, V) * 0.7, -1)
        del z
        s["tokens"] = (s["draft"] / noise(B, K, V)).argmax(-1).to(torch.int32)
    else:              # the j-th child of a node is the j-th likeliest token there, as a good draft model has it
        del z
        same = (parents[:, :, None] == parents[:, None, :]) & torch.ones(K, K, dtype=torch.bool, device=DEV).tril(-1)
        rank = same.sum(-1).clamp_max(min(8, V) - 1)
        top = s["target"].topk(min(8, V), -1).indices
        row = (parents.clamp_min(-1) + 1).long()
        s["tokens"] = top[torch.arange(B, device=DEV)[:, None], row, rank].to(torch.int32)
    return s


def _prepare_attn(case, seed, gen):
    B, K, H, Hk, D, ps = (case[k] for k in ("batch", "nodes", "heads", "kv_heads", "dim", "page"))
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    ctx = np.array(_lengths(case, "ctx", case["lo"], case["hi"], B))
    r = np.random.RandomState(seed % (1 << 31))
    pages = -(-(ctx + K) // ps)
    M, P = int(pages.max()), int(pages.sum()) + 1
    table = np.full((B, M), -1, np.int32)
    table[np.arange(M)[None] < pages[:, None]] = r.permutation(P)[: P - 1].astype(np.int32)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=dt)
    kv = rnd(P, 2, ps, Hk, D)  # keys and values of a page side by side
    return {"q": rnd(B, K, H, D), "k": kv[:, 0], "v": kv[:, 1], "table": _gpu(table), "ctx": _gpu(ctx.astype(np.int32)),
            "parents": _gpu(_trees(B, K, seed)), "scale": 1.0 / math.sqrt(D)}


def _prepare_tree(case, seed, gen):
    B, K, H, D = (case[k] for k in ("batch", "nodes", "heads", "dim"))
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)
    parents = _trees(B, K, seed)
    s = {"k": unit(rnd(B, K, H, D)), "g": -5 * torch.sigmoid(rnd(B, K, H, D)), "state": rnd(B, H, D, D) * 0.02}
    if case["commit"]:
        r = np.random.RandomState(seed % (1 << 31))
        path = np.full((B, K), -1, np.int32)
        n = np.zeros(B, np.int32)
        for b in range(B):  # from a random node up to the context, or nothing accepted
            i = int(r.randint(-1, K))
            while i >= 0 and parents[b, i] == PAD:
                i -= 1
            up = []
            while i >= 0:
                up.append(i)
                i = int(parents[b, i])
            n[b] = len(up)
            path[b, : len(up)] = up[::-1]
        return {**s, "path": _gpu(path), "n": _gpu(n), "writes": rnd(B, K, H, D) * 0.5}
    return {**s, "q": unit(rnd(B, K, H, D)), "v": rnd(B, K, H, D).to(dt), "beta": torch.sigmoid(rnd(B, K, H)), "parents": _gpu(parents)}


_PREPARE = {"tables": _prepare_tables, "verify": _prepare_verify, "attn": _prepare_attn, "tree": _prepare_tree}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"case": case, **_PREPARE[case["op"]](case, seed, gen)}


# ------------------------------------------------------------------ the plain forms
def _plain_tables(s):
    ps, F, T = s["page"], s["free"].numel(), s["tokens"]
    ctx, new, held = s["ctx"].long(), s["new"].long(), s["held"].long()
    B, M = s["table"].shape
    total = ctx + new
    fits = total <= M * ps
    need = torch.where(fits, ((total + ps - 1) // ps - held).clamp_min(0), 0)
    upto = need.cumsum(0)
    fits &= (need == 0) | (upto <= F)
    taken = torch.where(fits & (need > 0), upto, 0).amax().reshape(1)
    col = torch.arange(M, device=DEV)
    fresh = fits[:, None] & (col >= held[:, None]) & (col < (held + need)[:, None])
    at = (upto - need)[:, None] + col - held[:, None]
    s["table"].copy_(torch.where(fresh, s["free"][at.clamp(0, max(F - 1, 0))] if F else s["table"], s["table"]))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(B - 1)
    pos = ctx[b] + t - cu[b]
    page = s["table"][b, (pos // ps).clamp(0, M - 1)].long()
    slot = torch.where((t < cu[-1]) & fits[b], page * ps + pos % ps, -1)
    return {"slots": slot, "cu": cu.int(), "held": torch.where(fits, held + need, held).int(), "taken": taken.int(), "table": s["table"]}


def _plain_verify(s):
    P, Q, tok, par = s["target"], s["draft"], s["tokens"].long(), s["parents"].long()
    B, K = tok.shape
    rows = torch.arange(B, device=DEV)
    cur, mass = tok.new_full((B,), -1), P.new_ones(B)
    turned = torch.zeros((B, K), dtype=torch.bool, device=DEV)  # children of `cur` turned down so far
    kept = torch.zeros((B, K), dtype=torch.bool, device=DEV)
    for c in range(K):  # children come after their parents, so one pass in index order is the walk
        here = par[:, c] == cur
        p = P[rows, cur + 1, tok[:, c]]
        if Q is None:
            again = (turned & (tok == tok[:, c:c + 1])).any(-1)
            ok = here & ~again & (s["u"][:, c] * mass < p)
            mass = torch.where(ok, 1.0, torch.where(here & ~again, mass - p, mass))
        else:
            ok = here & (s["u"][:, c] * Q[rows, c, tok[:, c]] < p)
        turned[:, c] = here
        turned &= ~ok[:, None]
        kept[:, c] = ok
        cur = torch.where(ok, c, cur)
    p = P[rows, cur + 1]
    if Q is None:
        rest = torch.where(torch.zeros_like(p).scatter_add_(1, tok, turned.float()) > 0, 0.0, p)
    else:
        first = turned.int().argmax(-1)
        rest = torch.where(turned.any(-1, keepdim=True), (p - Q[rows, first]).clamp_min(0), p)
    rest = torch.where((rest > 0).any(-1, keepdim=True), rest, p)
    nxt = (rest / s["noise"]).argmax(-1)
    n = kept.sum(-1)
    order = torch.where(kept, torch.arange(K, device=DEV), K).sort(-1).values
    return {"path": torch.where(order < K, order, -1).int(), "accepted": n.int(), "next": nxt.int()}


def _ancestors(parents):
    """[B, K, K] truth values: node j is node i or above it (none for absent nodes)."""
    B, K = parents.shape
    par = parents.long()
    eye = torch.eye(K, dtype=torch.bool, device=parents.device)
    up = (par[:, :, None] == torch.arange(K, device=parents.device)).float()  # one step up
    anc = eye.float().expand(B, K, K)
    step = up
    for _ in range(max(1, (K - 1).bit_length())):  # 1, 2, 4, ... steps
        anc = ((anc + step @ anc) > 0).float()
        step = step @ step
    return (anc > 0) & (par != PAD)[:, :, None]


def _plain_attn(s):
    q, ctx = s["q"], s["ctx"].long()
    B, K, H, D = q.shape
    ps, Hk = s["k"].shape[1:3]
    L = s["table"].shape[1] * ps
    t = torch.arange(L, device=DEV)
    page = s["table"].long().clamp_min(0)
    inside = t < (ctx + K)[:, None]
    pick = lambda c: torch.where(inside[..., None, None], c[page].reshape(B, L, Hk, D), 0).float()
    node = t - ctx[:, None]
    anc = _ancestors(s["parents"])
    on = torch.gather(anc, 2, node.clamp(0, K - 1)[:, None, :].expand(B, K, L)) & (node >= 0)[:, None] & (node < K)[:, None]
    on = on | ((node < 0)[:, None] & (s["parents"] != PAD)[:, :, None])
    qf = q.float().reshape(B, K, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    sc = (qf @ pick(s["k"]).permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, Hk, H // Hk, K, L)
    sc.masked_fill_(~on[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    sc.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    den = sc.sum(-1, keepdim=True)
    o = (sc.view(B, Hk, -1, L) @ pick(s["v"]).permute(0, 2, 1, 3)).view(B, Hk, H // Hk, K, D)
    o = torch.where(den > 0, o / den, 0.0)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, K, H, D).to(q.dtype)}


def _plain_tree_step(s):
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))  # [B, H, K, D]
    g, beta, S = s["g"].transpose(1, 2), s["beta"].transpose(1, 2), s["state"]
    K = q.shape[2]
    anc = _ancestors(s["parents"])[:, None]
    there = (s["parents"] != PAD)[:, None, :, None]
    G = anc.float() @ g                                                       # decay along each node's path
    decay = torch.where(anc[..., None], G[:, :, :, None] - G[:, :, None], float("-inf")).exp_()
    A = torch.where(torch.eye(K, dtype=torch.bool, device=DEV), 0.0, (decay * k[:, :, :, None] * k[:, :, None]).sum(-1))
    Pm = (decay * q[:, :, :, None] * k[:, :, None]).sum(-1)
    del decay
    eG = G.exp()
    rest = v - (eG * k) @ S
    w = torch.zeros_like(v)
    for i in range(K):  # a node's write needs those above it
        w[:, :, i] = beta[:, :, i, None] * (rest[:, :, i] - (A[:, :, i, :, None] * w).sum(2))
    w = torch.where(there, w, 0.0)
    o = torch.where(there, (eG * q) @ S + Pm @ w, 0.0)
    return {"out": o.transpose(1, 2).contiguous(), "writes": w.transpose(1, 2).contiguous()}


def _plain_tree_commit(s):
    B, K = s["path"].shape
    on = torch.arange(K, device=DEV) < s["n"][:, None]
    at = s["path"].long().clamp_min(0)
    pick = lambda x: torch.where(on[:, :, None, None], x[torch.arange(B, device=DEV)[:, None], at].float(), 0.0).transpose(1, 2)
    k, g, w = pick(s["k"]), pick(s["g"]), pick(s["writes"])                  # [B, H, K, D] along the path
    after = g.flip(2).cumsum(2).flip(2) - g                                  # decay after each token's write
    S = s["state"]
    S.copy_(g.sum(2).exp()[..., None] * S + (after.exp() * k).transpose(2, 3) @ w)
    return {"state": S}


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "tree":
            return _plain_tree_commit(s) if s["case"]["commit"] else _plain_tree_step(s)
        return {"tables": _plain_tables, "verify": _plain_verify, "attn": _plain_attn}[op](s)
    import linear_attention_serving_chunkwise_gb300 as kda
    if op == "tables":
        slots, cu, held, taken = kda.page_tables(s["ctx"], s["new"], s["held"], s["table"], s["free"], page_size=s["page"], max_tokens=s["tokens"])
        return {"slots": slots, "cu": cu, "held": held, "taken": taken, "table": s["table"]}
    if op == "verify":
        path, n, nxt = kda.verify_drafts(s["target"], s["tokens"], s["parents"], s["u"], s["noise"], draft_probs=s["draft"])
        return {"path": path, "accepted": n, "next": nxt}
    if op == "attn":
        return {"out": kda.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["parents"], scale=s["scale"])}
    if s["case"]["commit"]:
        return {"state": kda.tree_commit(s["k"], s["g"], s["writes"], s["path"], s["n"], s["state"])}
    out, writes = kda.tree_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parents"], s["state"])
    return {"out": out, "writes": writes}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B, op = case["batch"], case["op"]
    if op == "tables":
        tokens = sum(_lengths(case, "new", case["new_lo"], case["new_hi"], B))
        pages = sum(-(-n // case["page"]) for n in _lengths(case, "ctx", case["lo"], case["hi"], B))
        return {"bytes": 8.0 * tokens + 20 * B + 8.0 * tokens / case["page"] + 4 * min(pages, B), "flops": 0}
    if op == "verify":  # the last row of the target and the noise; the draft's row where a token was turned down is not counted
        return {"bytes": B * (8.0 * case["vocab"] + 24 * case["nodes"]), "flops": B * case["vocab"]}
    K, H, D = case["nodes"], case["heads"], case["dim"]
    e = 2 if case["bf16"] else 4
    if op == "attn":
        tokens = sum(n + K for n in _lengths(case, "ctx", case["lo"], case["hi"], B))
        return {"bytes": 2.0 * tokens * case["kv_heads"] * D * e + 2.0 * B * K * H * D * e + 4.0 * tokens / case["page"], "flops": 4.0 * K * H * D * tokens}
    state, row = 4.0 * B * H * D * D, 1.0 * B * K * H * D
    if case["commit"]:  # paths are half as long as the trees at most; the rows of what was turned down are not needed
        return {"bytes": 2 * state, "flops": 3.0 * B * H * D * D}
    return {"bytes": state + row * (3 * e + 4 + 8), "flops": 4.0 * K * B * H * D * D}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] in ("tables", "verify"):  # whole numbers only
        return None
    s = prepare(case, seed)
    return (_exact_attn if case["op"] == "attn" else _exact_commit if case["commit"] else _exact_step)(s)


def _path_to(parents, i):
    up = []
    while i >= 0:
        up.append(i)
        i = parents[i]
    return up[::-1]


def _exact_attn(s):
    q = s["q"]
    B, K, H, D = q.shape
    ps, Hk = s["k"].shape[1:3]
    out = torch.zeros((B, K, H, D), dtype=torch.float64, device=DEV)
    parents, table, ctx = s["parents"].tolist(), s["table"].long(), s["ctx"].tolist()
    for b in range(B):
        n = ctx[b]
        t = torch.arange(n + K, device=DEV)
        page = table[b][t // ps]
        for h in range(Hk):
            kk, vv = (s[c][page, t % ps, h].double() for c in ("k", "v"))
            G = H // Hk
            qq = q[b, :, h * G:(h + 1) * G].double()                          # [K, G, D]
            near = torch.full((K, K), -math.inf, dtype=torch.float64, device=DEV)
            rows = [i for i in range(K) if parents[b][i] != PAD]
            for i in rows:
                near[i, _path_to(parents[b], i)] = 0.0
            logits = torch.einsum("igd,td->igt", qq, kk) * s["scale"]
            logits[:, :, n:] += near[:, None]
            for i in rows:
                out[b, i, h * G:(h + 1) * G] = torch.softmax(logits[i], -1) @ vv
    return {"out": out}


def _exact_step(s):
    B, K, H, D = s["q"].shape
    out, writes = (torch.zeros((B, K, H, D), dtype=torch.float64, device=DEV) for _ in range(2))
    parents = s["parents"].tolist()
    for b in range(B):
        states = {-1: s["state"][b].double()}
        for i in range(K):
            if parents[b][i] == PAD:
                continue
            q, k, v, g = (s[n][b, i].double() for n in ("q", "k", "v", "g"))  # [H, D]
            S = g.exp()[:, :, None] * states[parents[b][i]]
            w = s["beta"][b, i].double()[:, None] * (v - torch.einsum("hcd,hc->hd", S, k))
            states[i] = S + k[:, :, None] * w[:, None]
            writes[b, i] = w
            out[b, i] = torch.einsum("hcd,hc->hd", states[i], q)
    return {"out": out, "writes": writes}


def _exact_commit(s):
    path, n = s["path"].tolist(), s["n"].tolist()
    S = s["state"].double()
    for b in range(len(n)):
        for i in path[b][: n[b]]:
            g, k, w = (s[m][b, i].double() for m in ("g", "k", "writes"))
            S[b] = g.exp()[:, :, None] * S[b] + k[:, :, None] * w[:, None]
    return {"state": S}
