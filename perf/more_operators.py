"""The attention layers' prompt path and the upkeep of their cache, as they are measured: cases, inputs, plain forms and
exact values.

Five operators work on one paged key/value cache (pages of ``page`` tokens, a table row of page ids per sequence):

* ``attn``     softmax attention of chunks of new tokens over the cache (the context, and the chunk up to each token);
* ``rotate``   norms of queries and keys per head and their rotation by position, keys and values into the cache;
* ``fork``     table rows that share another row's first tokens, and the copy of the page that is not full, in all layers;
* ``release``  table rows cut short, and the pages that nobody holds any more;
* ``keep``     the cache rows of an accepted path of drafts moved to the front of the step's tokens, in all layers.
"""
import math
import random

import numpy as np
import torch

own = False  # True: the framework's kernels; False: the plain forms below

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's short first prompt: only latency
        {"name": "attn_first_b1", "op": "attn", "batch": 1, "new_lo": 129, "new_hi": 129, "lo": 0, "hi": 0, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "bf16": True},
        # a step of a serving batch: single tokens beside chunks of prompts, contexts of all lengths, twelve query heads to a cache head
        {"name": "attn_mixed_b12", "op": "attn", "batch": 12, "new_lo": 1, "new_hi": 2048, "lo": 0, "hi": 16384, "heads": 96, "kv_heads": 8, "dim": 128, "page": 64, "bf16": True},
        # the last chunk of a long prompt: 2048 tokens after 131072
        {"name": "attn_long_b1", "op": "attn", "batch": 1, "new_lo": 2048, "new_hi": 2048, "lo": 131072, "hi": 131072, "heads": 32, "kv_heads": 8, "dim": 128, "page": 128, "bf16": True},
        # the fp32 path: narrow heads, three query heads to a cache head, odd lengths, pages no power of two
        {"name": "attn_f32_b5", "op": "attn", "batch": 5, "new_lo": 1, "new_hi": 701, "lo": 0, "hi": 3001, "heads": 6, "kv_heads": 2, "dim": 64, "page": 24, "bf16": False},
        # one token of each of 64 sequences, some at far positions
        {"name": "rotate_step_t64", "op": "rotate", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": False, "weights": True, "page": 64, "far": 1000000, "bf16": True},
        # the prompts of a batch packed together, 96 heads, the last tokens without a slot
        {"name": "rotate_prompts_t32768", "op": "rotate", "tokens": 32768, "heads": 96, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": False, "weights": True, "page": 128, "far": 131072, "bf16": True},
        # four samples of one prompt in a small cache of one layer
        {"name": "fork_samples_n4", "op": "fork", "forks": 4, "parents": 1, "rows": 8, "lo": 1003, "hi": 1003, "page": 16, "layers": 1, "kv_heads": 8, "dim": 128, "bf16": True},
        # 96 samples of 16 prompts of all lengths, six layers, large pages
        {"name": "fork_batch_n96", "op": "fork", "forks": 96, "parents": 16, "rows": 160, "lo": 1, "hi": 8192, "page": 256, "layers": 6, "kv_heads": 2, "dim": 128, "bf16": True},
        # a small batch: one sequence ends, others give back what a step reserved for drafts
        {"name": "release_step_s16", "op": "release", "rows": 16, "pages_hi": 128, "group": 4, "page": 16, "pool": 4096, "ends": 0.1},
        # a fleet's worth of rows at once, groups of eight that share their first pages
        {"name": "release_many_s2048", "op": "release", "rows": 2048, "pages_hi": 512, "group": 8, "page": 64, "pool": 600000, "ends": 0.5},
        # one step of four users, seven nodes, one layer: only latency
        {"name": "keep_b4", "op": "keep", "batch": 4, "nodes": 7, "layers": 1, "kv_heads": 8, "dim": 128, "page": 16, "bf16": True},
        # the decode workload's 256 sequences, 16 nodes, eight layers
        {"name": "keep_b256", "op": "keep", "batch": 256, "nodes": 16, "layers": 8, "kv_heads": 8, "dim": 128, "page": 16, "bf16": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rotate", "rotate", "fork", "release", "keep"])
    shape = lambda: {"kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]), "page": rng.choice([8, 16, 24, 64, 100, 128, 256]),
                     "bf16": rng.random() < 0.75}
    if op == "attn":
        c = {"op": op, **shape()}
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        new, ctx = _log(rng, 1, 8192), _log(rng, 30, 131072 if c["bf16"] else 20000)
        c["lo"], c["hi"] = rng.choice([(0, 0), (0, ctx), (ctx // 2, ctx), (ctx, ctx)])
        c["new_lo"] = rng.choice([0, 1, new // 2, new])
        most = 4e12 if c["bf16"] else 2e11
        while new > 1 and 4.0 * c["heads"] * c["dim"] * new * (c["hi"] + new) > most:
            new = max(1, new // 2)
        c["new_hi"], c["new_lo"] = new, min(new, c["new_lo"])
        per = 4.0 * c["heads"] * c["dim"] * new * (c["hi"] + new)
        room = 3e9 / (4.0 * c["kv_heads"] * c["dim"] * (c["hi"] + new))
        c["batch"] = _log(rng, 1, max(1, min(48, int(most / per), int(room))))
        return c
    if op == "rotate":
        c = {"op": op, **shape()}
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8, 12])
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4])
        most = int(4e8 / ((c["heads"] + 2 * c["kv_heads"]) * c["dim"]))
        return {**c, "tokens": _log(rng, 1, min(32768, most)), "pairs": rng.random() < 0.4, "weights": rng.random() < 0.8,
                "far": _log(rng, 100, 1000000)}
    if op == "fork":
        c = {"op": op, **shape(), "layers": rng.choice([1, 2, 3, 6])}
        par = _log(rng, 1, 16)
        c["parents"], c["forks"] = par, _log(rng, 1, 96)
        c["rows"] = c["forks"] + par + rng.randint(0, 20)
        most = int(4e8 / (c["layers"] * c["kv_heads"] * c["dim"] * 8))
        c["hi"] = _log(rng, 1, max(2, min(8192, most // par)))
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        return c
    if op == "release":
        rows, hi = _log(rng, 1, 2048), _log(rng, 2, 512)
        return {"op": op, "rows": rows, "pages_hi": hi, "group": rng.choice([1, 2, 5, 8]), "page": rng.choice([1, 16, 24, 64, 256]),
                "pool": rows * hi + rng.randint(0, 60000) if rows * hi < 500000 else 1100000, "ends": rng.choice([0.0, 0.1, 0.5, 1.0])}
    c = {"op": op, **shape(), "layers": rng.choice([1, 2, 5, 8]), "nodes": _log(rng, 1, 64)}
    row = c["layers"] * c["kv_heads"] * c["dim"] * (4 if c["bf16"] else 8)
    return {**c, "batch": _log(rng, 1, max(1, min(256, int(3e8 / (row * (c["nodes"] + 2 * c["page"]))))))}


def _numbers(case, salt):
    """A generator fixed by the case alone, so that work() knows its lengths."""
    return random.Random("%s %s" % (salt, sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, salt, lo, hi, n):
    r = _numbers(case, salt)
    got = [r.randint(lo, hi) for _ in range(n)]
    got[0], got[-1] = lo, hi
    return got


# ------------------------------------------------------------------ inputs
def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _i32(x):
    return _gpu(np.asarray(x, np.int32))


def _dtype(case):
    return torch.bfloat16 if case["bf16"] else torch.float32


def _table(lens, page, r, spare=1, cols_more=1):
    """(table, number of pages): rows of distinct pages in random order, -1 behind them."""
    held = -(-np.asarray(lens, np.int64) // page)
    P = int(held.sum()) + spare
    table = np.full((len(lens), max(1, int(held.max()) + cols_more)), -1, np.int32)
    table[np.arange(table.shape[1])[None] < held[:, None]] = r.permutation(P)[: P - spare].astype(np.int32)
    return table, held, P


def _prepare_attn(case, seed, rnd, r):
    B, H, Hk, D, ps = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    ctx = _lengths(case, "ctx", case["lo"], case["hi"], B)
    new = _lengths(case, "new", case["new_lo"], case["new_hi"], B)
    table, _, P = _table(np.array(ctx) + np.array(new), ps, r)
    kv = rnd(P, 2, ps, Hk, D)  # keys and values of a page side by side
    cu = np.concatenate([[0], np.cumsum(new)])
    return {"q": rnd(int(cu[-1]), H, D), "k": kv[:, 0], "v": kv[:, 1], "table": _gpu(table), "ctx": _i32(ctx), "cu": _i32(cu),
            "host": (ctx, new), "scale": 1.0 / math.sqrt(D)}


def _prepare_rotate(case, seed, rnd, r):
    T, H, Hk, D, ps = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page"))
    qkv = rnd(T, H + 2 * Hk, D)  # the projection's output, used in place
    P = -(-T // ps) + 2
    pages = r.permutation(P)[: -(-T // ps)]
    t = np.arange(T)
    slots = pages[t // ps].astype(np.int64) * ps + t % ps
    slots[T - T // 50:] = -1     # padded tokens
    pos = (r.randint(0, case["far"]) + t) % case["far"]
    s = {"q": qkv[:, :H], "k": qkv[:, H:H + Hk], "v": qkv[:, H + Hk:], "pos": _i32(pos), "slots": _gpu(slots),
         "freq": _gpu((10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])).astype(np.float32)), "pairs": case["pairs"],
         "wq": None, "wk": None}
    kv = rnd(P, 2, ps, Hk, D)
    s["k_cache"], s["v_cache"] = kv[:, 0], kv[:, 1]
    if case["weights"]:
        s["wq"], s["wk"] = (1 + 0.2 * torch.from_numpy(r.standard_normal((2, D)).astype(np.float32)).to(DEV)).unbind(0)
    return s


def _caches(case, rnd, P):
    kv = rnd(case["layers"], P, 2, case["page"], case["kv_heads"], case["dim"])
    return {"k_cache": kv[:, :, 0], "v_cache": kv[:, :, 1]}


def _prepare_fork(case, seed, rnd, r):
    S, n, par, ps = case["rows"], case["forks"], case["parents"], case["page"]
    rows = r.permutation(S)
    lens = _lengths(case, "lens", case["lo"], case["hi"], par)
    whose = [_numbers(case, "whose%d" % i).randrange(par) for i in range(n)]
    table, held, used = _table(lens, ps, r, spare=0)
    pages = used + n + 2
    ids = r.permutation(pages).astype(np.int32)
    full = np.full((S, table.shape[1]), -1, np.int32)
    full[rows[:par]] = np.where(table >= 0, ids[np.maximum(table, 0)] if used else -1, -1)
    all_held = np.zeros(S, np.int64)
    all_held[rows[:par]] = held
    free = ids[used:]
    return {"parents": _i32(rows[np.array(whose)]), "children": _i32(rows[par:par + n]), "lens": _i32([lens[w] for w in whose]),
            "held": _i32(all_held), "table": _gpu(full), "shares": torch.zeros(pages, dtype=torch.int32, device=DEV), "free": _gpu(free),
            "page": ps, **_caches(case, rnd, pages)}


def _held(case):
    """Per row: pages held, pages shared with its group, pages kept, tokens kept."""
    r, ps = _numbers(case, "rows"), case["page"]
    got = []
    for i in range(case["rows"]):
        if i % case["group"] == 0:
            shared = r.randint(0, case["pages_hi"] // 2)
        own_ = r.randint(1, case["pages_hi"] - case["pages_hi"] // 2)
        held = shared + own_
        if r.random() < case["ends"]:
            keep = 0
        else:                     # some pages behind the context, reserved for drafts, or nothing
            keep = (held - min(own_ - 1, r.randint(0, 3))) * ps - r.randint(0, ps - 1)
        got.append((held, shared, -(-keep // ps), keep))
    return got


def _prepare_release(case, seed, rnd, r):
    S, P = case["rows"], case["pool"]
    rows = _held(case)
    ids = r.permutation(P).astype(np.int32)
    table = np.full((S, case["pages_hi"] + 1), -1, np.int32)
    shares = np.zeros(P, np.int32)
    at = 0
    for i, (held, shared, _, _) in enumerate(rows):
        if i % case["group"] == 0:
            common = ids[at:at + shared]
            at += shared
        else:
            shares[common] += 1
        table[i, :shared] = common
        table[i, shared:held] = ids[at:at + held - shared]
        at += held - shared
    return {"keep": _i32([x[3] for x in rows]), "held": _i32([x[0] for x in rows]), "table": _gpu(table), "shares": _gpu(shares),
            "page": case["page"]}


def _paths(case):
    r, K = _numbers(case, "paths"), case["nodes"]
    got = []
    for _ in range(case["batch"]):
        n, node, path = r.randint(0, K), -1, []
        while len(path) < n:
            node += 1 + (r.random() < 0.4) + (r.random() < 0.2)
            if node >= K:
                break
            path.append(node)
        got.append(path)
    return got


def _prepare_keep(case, seed, rnd, r):
    B, K, ps = case["batch"], case["nodes"], case["page"]
    first = np.array(_lengths(case, "first", 0, ps - 1, B))  # where in its page each step began
    table, _, P = _table(first + K, ps, r)
    pos = first[:, None] + np.arange(K)
    slots = np.take_along_axis(table, pos // ps, 1).astype(np.int64) * ps + pos % ps
    path = np.full((B, K), -1, np.int32)
    paths = _paths(case)
    for b, p in enumerate(paths):
        path[b, : len(p)] = p
    return {"slots": _gpu(slots), "path": _gpu(path), "n": _i32([len(p) for p in paths]), **_caches(case, rnd, P)}


_PREPARE = {"attn": _prepare_attn, "rotate": _prepare_rotate, "fork": _prepare_fork, "release": _prepare_release, "keep": _prepare_keep}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _dtype(case) if "bf16" in case else torch.float32
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=dt)
    return {"case": case, **_PREPARE[case["op"]](case, seed, rnd, np.random.RandomState(seed % (1 << 31)))}


# ------------------------------------------------------------------ the plain forms
def _plain_attn(s):
    q, out = s["q"], torch.empty_like(s["q"])
    ps, Hk, D = s["k"].shape[1:]
    H = q.shape[1]
    at = 0
    for b, (n, m) in enumerate(zip(*s["host"])):
        if m == 0:
            continue
        L = n + m
        page = s["table"][b, : -(-L // ps)].long()
        k, v = (s[c][page].reshape(-1, Hk, D)[:L].float().transpose(0, 1) for c in ("k", "v"))    # [Hk, L, D]
        step = max(1, int(5e8 / (H * L)))
        for i in range(0, m, step):
            j = min(m, i + step)
            qq = q[at + i: at + j].float().reshape(j - i, Hk, H // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
            sc = (qq @ k.transpose(1, 2)).mul_(s["scale"]).view(Hk, H // Hk, j - i, L)
            late = torch.arange(L, device=DEV)[None] > n + torch.arange(i, j, device=DEV)[:, None]
            sc.masked_fill_(late, float("-inf"))
            sc.sub_(sc.amax(-1, keepdim=True)).exp_()
            den = sc.sum(-1, keepdim=True)
            o = (sc.view(Hk, -1, L) @ v).view(Hk, H // Hk, j - i, D) / den
            out[at + i: at + j] = o.permute(2, 0, 1, 3).reshape(j - i, H, D).to(out.dtype)
        at += m
    return {"out": out}


def _rotated(x, w, cos, sin, rot, pairs):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if w is not None:
        y = y * w
    if pairs:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _plain_rotate(s):
    rot = 2 * s["freq"].numel()
    angle = s["pos"].double()[:, None, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(s["q"].float(), s["wq"], cos, sin, rot, s["pairs"]).to(s["q"].dtype)
    k = _rotated(s["k"].float(), s["wk"], cos, sin, rot, s["pairs"]).to(s["q"].dtype)
    ps = s["k_cache"].shape[1]
    on = s["slots"] >= 0
    page, at = s["slots"][on] // ps, s["slots"][on] % ps
    s["k_cache"][page, at] = k[on]
    s["v_cache"][page, at] = s["v"][on]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_fork(s):
    ps, F = s["page"], s["free"].numel()
    par, child, lens = s["parents"].long(), s["children"].long(), s["lens"].long()
    full, rest = lens // ps, lens % ps
    need = (rest > 0).long()
    upto = need.cumsum(0)
    ok = (need == 0) | (upto <= F)
    taken = torch.where(ok, upto * need, 0).amax().reshape(1).int()
    col = torch.arange(s["table"].shape[1], device=DEV)
    src = s["table"][par]
    shared = ok[:, None] & (col < full[:, None])
    fresh = (ok & (need > 0))[:, None] & (col == full[:, None])
    page = s["free"][(upto - 1).clamp(0, F - 1)]
    s["table"][child] = torch.where(shared, src, torch.where(fresh, page[:, None], s["table"][child]))
    s["shares"].index_add_(0, torch.where(shared, src, 0).flatten().long(), shared.flatten().int())
    held = s["held"].clone()
    held[child] = torch.where(ok, full + need, s["held"][child]).int()
    on = ok & (need > 0)
    copies = torch.stack([torch.where(on, src.gather(1, full.clamp_max(src.shape[1] - 1)[:, None])[:, 0], -1),
                          torch.where(on, page, -1), torch.where(on, rest, 0)], 1).int()
    a, b, rows = (x[on].long() for x in copies.unbind(1))
    live = (torch.arange(ps, device=DEV) < rows[:, None])[None, :, :, None, None]
    for c in ("k_cache", "v_cache"):
        s[c][:, b] = torch.where(live, s[c][:, a], s[c][:, b])
    return {"held": held, "table": s["table"], "shares": s["shares"], "copies": copies, "taken": taken, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_release(s):
    ps, P = s["page"], s["shares"].numel()
    keep = (s["keep"].long() + ps - 1) // ps
    held = s["held"].long()
    col = torch.arange(s["table"].shape[1], device=DEV)
    last = s["table"].gather(1, (keep - 1).clamp_min(0)[:, None])[:, 0].long().clamp_min(0)
    stays = (s["keep"] % ps > 0) & (s["shares"][last] > 0) & (keep < held)   # others hold the page that would be cut
    gone = (col >= keep[:, None]) & (col < held[:, None]) & ~stays[:, None]
    s["shares"] -= torch.bincount(s["table"][gone], minlength=P).int()
    free = (s["shares"] < 0).nonzero()[:, 0].int()
    s["shares"].clamp_min_(0)
    freed = torch.full((P,), -1, dtype=torch.int32, device=DEV)
    freed[: free.numel()] = free
    return {"held": torch.where(stays, held, torch.minimum(held, keep)).int(), "shares": s["shares"], "freed": freed,
            "n": torch.full((1,), free.numel(), dtype=torch.int32, device=DEV)}


def _plain_keep(s):
    ps = s["k_cache"].shape[2]
    on = torch.arange(s["path"].shape[1], device=DEV) < s["n"][:, None]
    src, dst = s["slots"].gather(1, s["path"].clamp_min(0).long())[on], s["slots"][on]
    for c in ("k_cache", "v_cache"):
        s[c][:, dst // ps, dst % ps] = s[c][:, src // ps, src % ps]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_PLAIN = {"attn": _plain_attn, "rotate": _plain_rotate, "fork": _plain_fork, "release": _plain_release, "keep": _plain_keep}


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    import linear_attention_serving_chunkwise_gb300 as kda
    if op == "attn":
        return {"out": kda.chunk_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cu"], scale=s["scale"])}
    if op == "rotate":
        q = kda.norm_rotate(s["q"], s["k"], s["v"], s["pos"], s["freq"], s["slots"], s["k_cache"], s["v_cache"], q_weight=s["wq"],
                            k_weight=s["wk"], eps=EPS, interleaved=s["pairs"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "fork":
        held, copies, taken = kda.page_fork(s["parents"], s["children"], s["lens"], s["held"], s["table"], s["shares"], s["free"], page_size=s["page"])
        kda.cache_copy(copies, s["k_cache"], s["v_cache"])
        return {"held": held, "table": s["table"], "shares": s["shares"], "copies": copies, "taken": taken, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "release":
        held, freed, n = kda.page_release(s["keep"], s["held"], s["table"], s["shares"], page_size=s["page"])
        return {"held": held, "shares": s["shares"], "freed": freed, "n": n}
    kda.cache_keep_path(s["slots"], s["path"], s["n"], s["k_cache"], s["v_cache"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    e = 2 if case.get("bf16", True) else 4
    if op == "attn":
        B, H, Hk, D = (case[k] for k in ("batch", "heads", "kv_heads", "dim"))
        ctx = _lengths(case, "ctx", case["lo"], case["hi"], B)
        new = _lengths(case, "new", case["new_lo"], case["new_hi"], B)
        seen = sum(m * n + m * (m + 1) // 2 for n, m in zip(ctx, new))
        tokens = sum(n + m for n, m in zip(ctx, new) if m)
        return {"bytes": 2.0 * tokens * Hk * D * e + 2.0 * sum(new) * H * D * e + 4.0 * tokens / case["page"], "flops": 4.0 * H * D * seen}
    if op == "rotate":
        T, D = case["tokens"], case["dim"]
        return {"bytes": 2.0 * T * (case["heads"] + 2 * case["kv_heads"]) * D * e + 12.0 * T, "flops": 6.0 * T * (case["heads"] + case["kv_heads"]) * D}
    if op == "fork":
        par, n, ps = case["parents"], case["forks"], case["page"]
        lens = _lengths(case, "lens", case["lo"], case["hi"], par)
        whose = [lens[_numbers(case, "whose%d" % i).randrange(par)] for i in range(n)]
        row = 2.0 * case["layers"] * case["kv_heads"] * case["dim"] * e
        return {"bytes": 2 * row * sum(m % ps for m in whose) + 16.0 * sum(-(-m // ps) for m in whose) + 24.0 * n + 8.0 * case["rows"], "flops": 0}
    if op == "release":
        gone = sum(held - min(held, keep) for held, _, keep, _ in _held(case))
        return {"bytes": 4.0 * gone + 12.0 * case["rows"] + 8.0 * case["pool"], "flops": 0}
    row = 2.0 * case["layers"] * case["kv_heads"] * case["dim"] * e
    return {"bytes": 2 * row * sum(sum(i != j for i, j in enumerate(p)) for p in _paths(case)) + 12.0 * case["batch"] * case["nodes"], "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "attn":
        return None if work(case)["flops"] > 6e12 else _exact_attn(prepare(case, seed))
    if case["op"] == "rotate":
        return _exact_rotate(prepare(case, seed))
    return None  # whole numbers, and rows that are only moved


def _exact_attn(s):
    T, H, D = s["q"].shape
    ps, Hk = s["k"].shape[1:3]
    out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(*s["host"])):
        t = torch.arange(n + m, device=DEV)
        page = s["table"][b].long()[t // ps]
        for h in range(H):
            if m:
                kk, vv = (s[c][page, t % ps, h * Hk // H].double() for c in ("k", "v"))
            for i in range(0, m, 512):
                j = min(m, i + 512)
                seen = n + j
                logits = s["q"][at + i: at + j, h].double() @ kk[:seen].T * s["scale"]
                logits.masked_fill_(t[:seen] > n + t[i:j, None], -math.inf)
                out[at + i: at + j, h] = torch.softmax(logits, -1) @ vv[:seen]
        at += m
    return {"out": out}


def _exact_rotate(s):
    half = s["freq"].numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None, None] * s["freq"].double())
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        if w is not None:
            y = y * w.double()
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["pairs"] else (slice(0, half), slice(half, 2 * half))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        got.append(y)
    ps = s["k_cache"].shape[1]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    on = s["slots"] >= 0
    where = (s["slots"][on] // ps, s["slots"][on] % ps)
    kc[where], vc[where] = got[1][on], s["v"][on].double()
    return {"q": got[0], "k_cache": kc, "v_cache": vc}
