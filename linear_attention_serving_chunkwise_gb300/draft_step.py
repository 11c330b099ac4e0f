"""One speculative decoding step of a hybrid model, with the library's draft-step calls.

A hybrid model has KDA layers, whose memory is a recurrent state, beside attention layers, whose
memory is a paged key/value cache.  A step takes each sequence's pending token and a tree of drafted
tokens after it, runs the model on all of them at once, keeps the drafts that the target's
probabilities keep, and moves both memories to the end of the kept path:

    page_tables     pages and slots for the step's tokens
    tree_decode     KDA layers: outputs of every node from one read of the state
    tree_attention  attention layers: every node over the cache and its own path
    verify_drafts   kept path and the token after it (the next pending token)
    tree_commit     KDA states at the end of the path;  ``keep_path`` the same for the cache

The pending token is node 0 of the model's tree and drafted node i is node i + 1, so the target's
row 0 is the one after the pending token.  ``HybridLayers`` holds the two memories of one KDA layer and
one attention layer; ``python -m linear_attention_serving_chunkwise_gb300.draft_step`` runs a toy model
with random weights and compares it with decoding token by token.
"""
from __future__ import annotations

import torch

from . import (KDA_PROLOGUE_ALL, KDA_TREE_PAD, page_tables, prefill, tree_attention, tree_commit, tree_decode,
               verify_drafts)


def with_pending(parents: torch.Tensor) -> torch.Tensor:
    """The model's tree [B, K + 1]: the pending token on the context, the drafts ``parents`` [B, K] after it."""
    shifted = torch.where(parents == KDA_TREE_PAD, parents, parents + 1)
    return torch.cat([torch.full_like(parents[:, :1], -1), shifted], 1)


def with_pending_path(path: torch.Tensor, n_accept: torch.Tensor):
    """A kept path of drafts as one of the model's tree: the pending token, then the drafts."""
    full = torch.cat([torch.zeros_like(path[:, :1]), torch.where(path >= 0, path + 1, path)], 1)
    return full, n_accept + 1


def keep_path(cache: torch.Tensor, slots: torch.Tensor, path: torch.Tensor, n: torch.Tensor) -> None:
    """The kept nodes' rows of ``cache`` [pages, 2, page_size, heads, dim] moved to the front of the step's
    tokens.  slots [B, K]: where the nodes were written.  Entry e of a path is node e or a later
    one, so every row moves towards the front; the rows are read before any is written."""
    rows = cache.shape[2]
    on = torch.arange(path.shape[1], device=path.device) < n[:, None]
    src, dst = slots.gather(1, path.clamp_min(0).long())[on], slots[on]
    cache[dst // rows, :, dst % rows] = cache[src // rows, :, src % rows]


class HybridLayers:
    """The memories of one KDA layer (state) and one attention layer (paged cache) for B sequences."""

    def __init__(self, batch: int, heads: int, dim: int, kv_heads: int, num_pages: int, page_size: int, table_cols: int,
                 device="cuda", dtype=torch.bfloat16):
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
        self.state = torch.zeros((batch, heads, dim, dim), dtype=torch.float32, device=device)
        self.cache = torch.empty((num_pages, 2, page_size, kv_heads, dim), dtype=dtype, device=device)
        self.context_lens, self.pages_held = i32(batch), i32(batch)
        self.block_table = torch.full((batch, table_cols), -1, dtype=torch.int32, device=device)
        self.free_pages = torch.arange(num_pages, dtype=torch.int32, device=device)

    def reserve(self, tokens: int) -> torch.Tensor:
        """Slots [B, tokens] for that many tokens after every context.  Where the free pages, or a sequence's
        table row, do not reach for all: RuntimeError, and the sequences they reach for keep their pages."""
        B = self.context_lens.numel()
        new = torch.full_like(self.context_lens, tokens)
        slots, _, self.pages_held, taken = page_tables(self.context_lens, new, self.pages_held, self.block_table, self.free_pages,
                                                       page_size=self.cache.shape[2], max_tokens=B * tokens)
        taken, refused = torch.stack([taken[0], (slots < 0).any().int()]).tolist()      # (one trip to the device)
        self.free_pages = self.free_pages[taken:]
        if refused:
            raise RuntimeError("out of cache pages, or of columns of the block table")
        return slots.view(B, tokens)

    def attend(self, q, k, v, slots, parents) -> torch.Tensor:
        """Keys and values of the nodes into their slots, then the nodes over the cache."""
        rows = self.cache.shape[2]
        page, at = slots // rows, slots % rows
        self.cache[page, 0, at] = k
        self.cache[page, 1, at] = v
        return tree_attention(q, self.cache[:, 0], self.cache[:, 1], self.block_table, self.context_lens, parents)


class ToyHybrid:
    """Embedding, one KDA layer, one attention layer and tied logits, random weights: enough to run the step in earnest."""

    def __init__(self, batch: int, vocab: int = 211, heads: int = 4, dim: int = 128, kv_heads: int = 2, page_size: int = 16,
                 most_tokens: int = 512, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        width = heads * dim
        w = lambda *s: (torch.randn(s, generator=g, device=device) * s[0] ** -0.5).to(torch.bfloat16)
        self.heads, self.dim, self.kv_heads, self.width = heads, dim, kv_heads, width
        self.embed = torch.randn((vocab, width), generator=g, device=device).to(torch.bfloat16)
        self.kda_in, self.kda_out = w(width, 3 * width), w(width, width)
        self.decay, self.beta = w(width, width), w(width, heads)
        self.att_in, self.att_out = w(width, width + 2 * kv_heads * dim), w(width, width)
        cols = -(-most_tokens // page_size)
        self.mem = HybridLayers(batch, heads, dim, kv_heads, batch * cols, page_size, cols, device)

    def _kda_inputs(self, x):
        """q, k, v, g, beta of the KDA layer, raw: the kernels normalise and squash them (input prologue)."""
        heads = lambda y: y.view(*y.shape[:-1], self.heads, self.dim).contiguous()
        q, k, v = (heads(y) for y in (x @ self.kda_in).chunk(3, -1))
        return q, k, v, heads((x @ self.decay).float()), (x @ self.beta).float().contiguous()

    def _attention(self, h, slots, parents):
        B, K, _ = h.shape
        y = h @ self.att_in
        q, k, v = y.split((self.width, self.kv_heads * self.dim, self.kv_heads * self.dim), -1)
        view = lambda t, n: t.reshape(B, K, n, self.dim).contiguous()
        o = self.mem.attend(view(q, self.heads), view(k, self.kv_heads), view(v, self.kv_heads), slots, parents)
        return h + o.view(B, K, self.width) @ self.att_out

    def _probs(self, h):
        h = h.float()
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)
        return torch.softmax(h @ self.embed.float().t() * (4.0 / self.width ** 0.5), -1)

    def prompt(self, tokens: torch.Tensor) -> torch.Tensor:
        """tokens [B, T]: both memories after them; returns the probabilities after each prompt [B, V]."""
        B, T = tokens.shape
        x = self.embed[tokens.long()]
        q, k, v, g, beta = (t.reshape(B * T, *t.shape[2:]) for t in self._kda_inputs(x))
        o, self.mem.state = prefill(q, k, v, g, beta, num_seqs=B, init_state=self.mem.state, prologue=KDA_PROLOGUE_ALL)
        h = x + (o.view(B, T, self.width).to(torch.bfloat16) @ self.kda_out)
        for t in range(0, T, 64):                      # the attention layer takes the prompt in chains of 64
            part = h[:, t:t + 64]
            n = part.shape[1]
            chain = torch.arange(-1, n - 1, dtype=torch.int32, device=h.device).expand(B, n).contiguous()
            last = self._attention(part, self.mem.reserve(n), chain)
            self.mem.context_lens = self.mem.context_lens + n
        return self._probs(last[:, -1])

    def forward(self, tokens: torch.Tensor, parents: torch.Tensor):
        """The model on a tree of tokens [B, K]: probabilities after every node [B, K, V].  The memories do not move;
        ``commit`` moves them."""
        B, K = tokens.shape
        x = self.embed[tokens.long()]
        q, k, v, g, beta = self._kda_inputs(x)
        o, writes = tree_decode(q, k, v, g, beta, parents, self.mem.state, prologue=KDA_PROLOGUE_ALL)
        slots = self.mem.reserve(K)
        h = self._attention(x + o.view(B, K, self.width).to(torch.bfloat16) @ self.kda_out, slots, parents)
        self._step = (k, g, writes, slots)
        return self._probs(h)

    def commit(self, path: torch.Tensor, n: torch.Tensor) -> None:
        """Both memories moved to the end of ``path`` of the last ``forward``'s tree."""
        k, g, writes, slots = self._step
        tree_commit(k, g, writes, path, n, self.mem.state, prologue=KDA_PROLOGUE_ALL)
        keep_path(self.mem.cache, slots, path, n)
        self.mem.context_lens = self.mem.context_lens + n

    def step(self, pending, drafts, parents, uniforms, noise):
        """One speculative step: pending [B], drafts and parents [B, K]; uniforms [B, K] ~ U[0, 1), noise [B, V] ~
        Exp(1).  Returns (kept path [B, K], its length [B], the next pending token [B])."""
        target = self.forward(torch.cat([pending[:, None], drafts], 1), with_pending(parents))
        path, n, nxt = verify_drafts(target, drafts, parents, uniforms, noise)
        self.commit(*with_pending_path(path, n))
        return path, n, nxt


def draft_by_rank(probs: torch.Tensor, parents: torch.Tensor) -> torch.Tensor:
    """A stand-in for a draft model: every node's token by its rank among its siblings in ``probs`` [B, V]."""
    B, K = parents.shape
    same = (parents[:, :, None] == parents[:, None, :]) & torch.ones(K, K, dtype=torch.bool, device=probs.device).tril(-1)
    return probs.topk(K, -1).indices.gather(1, same.sum(-1)).to(torch.int32)


def demo(batch: int = 3, prompt: int = 70, steps: int = 12, seed: int = 0) -> dict:
    """Steps of the toy model, and the same tokens decoded one by one: what was accepted, and the largest
    differences of the states and of the last probabilities."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    tree = torch.tensor([-1, -1, -1, 0, 0, 1, 3], dtype=torch.int32, device=dev).expand(batch, 7).contiguous()
    prompts = torch.randint(0, 211, (batch, prompt), generator=g, device=dev, dtype=torch.int32)
    fast, slow = ToyHybrid(batch, seed=seed), ToyHybrid(batch, seed=seed)
    probs = fast.prompt(prompts)
    slow.prompt(prompts)
    pending = probs.argmax(-1).to(torch.int32)
    done, kept = [[int(t)] for t in pending], 0
    for _ in range(steps):
        drafts = draft_by_rank(probs, tree)
        noise = torch.empty(probs.shape, device=dev).exponential_(generator=g)
        path, n, nxt = fast.step(pending, drafts, tree, torch.rand(tree.shape, generator=g, device=dev), noise)
        for b in range(batch):
            done[b] += drafts[b, path[b, :int(n[b])].long()].tolist() + [int(nxt[b])]
        kept += int(n.sum())
        pending = nxt
    alone, chain = torch.tensor([0], dtype=torch.int32, device=dev), torch.tensor([[-1]], dtype=torch.int32, device=dev)
    worst_state = worst_probs = 0.0
    one = fast.forward(pending[:, None], chain.expand(batch, 1).contiguous())      # probabilities after the pending tokens
    for t in range(max(len(d) for d in done)):          # token by token; sequences that are done stand still
        live = torch.tensor([t < len(d) - 1 for d in done], device=dev)
        tok = torch.tensor([d[min(t, len(d) - 1)] for d in done], dtype=torch.int32, device=dev)
        p = slow.forward(tok[:, None], chain.expand(batch, 1).contiguous())
        for b, d in enumerate(done):
            if t == len(d) - 1:
                worst_probs = max(worst_probs, float((p[b] - one[b]).abs().max()))
                worst_state = max(worst_state, float((slow.mem.state[b] - fast.mem.state[b]).abs().max()))
        slow.commit(alone.expand(batch, 1).contiguous(), live.to(torch.int32))
    return {"tokens": sum(len(d) for d in done), "steps": steps * batch, "kept_drafts": kept, "state": worst_state, "probs": worst_probs}


if __name__ == "__main__":
    r = demo()
    print(f"{r['tokens']} tokens in {r['steps']} sequence steps ({r['kept_drafts']} drafts kept); against token by token: "
          f"state {r['state']:.2e}, probabilities {r['probs']:.2e}")
