"""The attention layers' calls one after another, as a serving loop makes them: prompts in chunks, sequences forked from a
prompt, a step of drafts and its kept path, rows that end and pages that come back.  Two layers share the block tables.
What each sequence holds is kept beside it as plain lists of rows; every chunk's outputs are compared with the
definition over those lists (bounds: those of the single calls)."""
import numpy as np
import pytest
import torch

import _prompt_ref as R
from linear_attention_serving_chunkwise_gb300 import draft_step

pytestmark = pytest.mark.gpu
I32 = torch.int32
LAYERS, HQ, HK, D = 2, 8, 2, 64


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=I32).cuda()


class Loop:
    """Block tables, caches and, per sequence and layer, the rows it has stored."""

    def __init__(self, kda, rows, pages, ps, dtype, seed):
        self.kda, self.rows, self.pages, self.ps, self.dtype = kda, rows, pages, ps, dtype
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.cache = torch.full((LAYERS, pages, 2, ps, HK, D), float("nan"), dtype=dtype, device="cuda")
        self.table = torch.full((rows, 40), -1, dtype=I32, device="cuda")
        self.shares, self.free = _i32(np.zeros(pages)), _i32(np.random.default_rng(seed).permutation(pages))
        self.held, self.ctx = _i32(np.zeros(rows)), _i32(np.zeros(rows))
        self.freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
        self.stored = [[torch.zeros(0, 2, HK, D, dtype=dtype) for _ in range(LAYERS)] for _ in range(rows)]

    def slots(self, new):
        total = sum(new)
        slots, cu, self.held, taken = self.kda.page_tables(self.ctx, _i32(new), self.held, self.table, self.free, page_size=self.ps, max_tokens=total)
        self.free = self.free[int(taken):]
        assert (slots >= 0).all()
        return slots, cu

    def write(self, layer, slots, positions):
        """Random rows of one projection, normed and rotated into the layer's cache."""
        qkv = torch.randn(slots.numel(), HQ + 2 * HK, D, generator=self.gen, device="cuda").to(self.dtype)
        kc, vc = self.cache[layer].unbind(1)
        q = self.kda.norm_rotate(*qkv.split((HQ, HK, HK), 1), positions, self.freq, slots, kc, vc)
        return q, self.cache[layer][slots // self.ps, :, slots % self.ps].cpu()

    def chunk(self, new):
        """new[r] tokens more of every sequence, through both layers."""
        slots, cu = self.slots(new)
        pos = torch.cat([torch.arange(n, dtype=I32) + int(c) for n, c in zip(new, self.ctx)]).cuda()
        ends = cu.tolist()
        for layer in range(LAYERS):
            q, rows = self.write(layer, slots, pos)
            for r in range(self.rows):
                self.stored[r][layer] = torch.cat([self.stored[r][layer], rows[ends[r]:ends[r + 1]]])
            kc, vc = self.cache[layer].unbind(1)
            out = self.kda.chunk_attention(q, kc, vc, self.table, self.ctx, cu)
            # the same sequences, each in one page of its own
            most = max(s[layer].shape[0] for s in self.stored)
            plain = torch.zeros(self.rows, 2, most, HK, D, dtype=self.dtype)
            for r in range(self.rows):
                plain[r, :, :self.stored[r][layer].shape[0]] = self.stored[r][layer].transpose(0, 1)
            ref, bound, mass = R.chunk_attention(q, plain[:, 0], plain[:, 1], torch.arange(self.rows, dtype=I32)[:, None], self.ctx.cpu(), cu.cpu(), D ** -0.5)
            if self.dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
            assert ((out.cpu().double() - ref).abs() <= bound).all(), layer
        self.ctx = self.ctx + _i32(new)
        assert [s[0].shape[0] for s in self.stored] == self.ctx.tolist()

    def fork(self, parents, children, lens):
        self.held, copies, taken = self.kda.page_fork(_i32(parents), _i32(children), _i32(lens), self.held, self.table, self.shares, self.free, page_size=self.ps)
        self.kda.cache_copy(copies, self.cache[:, :, 0], self.cache[:, :, 1])
        self.free = self.free[int(taken):]
        for p, c, n in zip(parents, children, lens):
            self.stored[c] = [x[:n] for x in self.stored[p]]
            self.ctx[c] = n

    def drafts(self, parents, kept):
        """A step of drafts in every sequence: K nodes written, the kept ones' rows moved to the front; the pages behind
        stay reserved."""
        B, K = self.rows, len(parents)
        slots, _ = self.slots([K] * B)
        depth = []
        for p in parents:
            depth.append(0 if p < 0 else depth[p] + 1)
        pos = (self.ctx[:, None] + _i32(depth)).reshape(-1).contiguous()
        path, n = np.full((B, K), -1, np.int32), np.zeros(B, np.int32)
        for r, k in enumerate(kept):
            path[r, :len(k)], n[r] = k, len(k)
        for layer in range(LAYERS):
            q, rows = self.write(layer, slots, pos)
            kc, vc = self.cache[layer].unbind(1)
            out = self.kda.tree_attention(q.view(B, K, HQ, D), kc, vc, self.table, self.ctx, _i32(parents).expand(B, K).contiguous())
            assert torch.isfinite(out).all()
            for r, k in enumerate(kept):
                self.stored[r][layer] = torch.cat([self.stored[r][layer], rows.view(B, K, 2, HK, D)[r, k]])
        self.kda.cache_keep_path(slots.view(B, K), _i32(path), _i32(n), self.cache[:, :, 0], self.cache[:, :, 1])
        self.ctx = self.ctx + _i32(n)

    def release(self, keep):
        self.held, freed, n = self.kda.page_release(_i32(keep), self.held, self.table, self.shares, page_size=self.ps)
        self.free = torch.cat([self.free, freed[:int(n)]])
        for r, k in enumerate(keep):
            k = min(k, self.stored[r][0].shape[0])
            self.stored[r] = [x[:k] for x in self.stored[r]]
            self.ctx[r] = k

    def check_pages(self):
        """Every page is free, or held by one row more than it has shares."""
        holders = np.zeros(self.pages, int)
        for r, h in enumerate(self.held.tolist()):
            for p in self.table[r, :h].tolist():
                holders[p] += 1
        free = self.free.tolist()
        assert len(set(free)) == len(free) and not holders[free].any()
        assert (holders > 0).sum() + len(free) == self.pages
        assert (np.maximum(holders - 1, 0) == self.shares.cpu().numpy()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("ps", [5, 8, 16])
def test_prompts_forks_drafts_and_releases(cuda_lib, ps, dtype):
    loop = Loop(cuda_lib, rows=6, pages=220, ps=ps, dtype=dtype, seed=ps)
    loop.chunk([70, 33, 0, 0, 0, 16])                 # prompts, in two chunks
    loop.chunk([21, 1, 0, 0, 0, 130])
    loop.check_pages()
    loop.fork([0, 0, 5], [2, 3, 4], [91, 40, 16])     # samples of one prompt: all of it, its first tokens; whole pages
    loop.check_pages()
    loop.chunk([1, 1, 1, 1, 1, 1])                    # a token each: nobody writes into another's page
    loop.drafts([-1, -1, 1, 0, 2, 2], [[0, 3], [1, 2, 4], [1], [], [1, 2, 5], [0]])
    loop.chunk([1, 30, 2, 1, 0, 9])                   # single tokens beside chunks
    loop.check_pages()
    loop.release([0, 40, 1000, 1000, 1000, 0])        # two end (one shared by others), one is cut
    loop.check_pages()
    loop.chunk([50, 3, 1, 1, 1, 20])                  # new sequences on pages that came back
    loop.check_pages()
    loop.release([0] * 6)
    assert sorted(loop.free.tolist()) == list(range(220)) and not loop.shares.any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_the_models_forks_go_on_alike(cuda_lib):
    """Two samples forked from one prompt, decoded with the same tokens, give the prompt's own probabilities and states."""
    m = draft_step.ToyHybrid(3, seed=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    m.prompt(torch.randint(0, 211, (3, 45), generator=g, device="cuda", dtype=I32))
    m.mem.release(_i32([1000, 0, 0]))
    m.mem.fork(_i32([0, 0]), _i32([1, 2]), _i32([45, 45]))
    assert m.mem.context_lens.tolist() == [45, 45, 45] and m.mem.shares.sum() == 4
    alone, chain = torch.zeros(3, 1, dtype=I32, device="cuda"), torch.full((3, 1), -1, dtype=I32, device="cuda")
    for t in range(5):
        p = m.forward(_i32([[t], [t], [t]]), chain)
        m.commit(alone, _i32([1, 1, 1]))
        assert torch.equal(p[0], p[1]) and torch.equal(p[0], p[2])
    assert torch.equal(m.mem.state[0], m.mem.state[1]) and torch.equal(m.mem.state[0], m.mem.state[2])
    m.mem.release(_i32([0, 0, 0]))
    assert m.mem.free_pages.numel() == m.mem.shares.numel() and not m.mem.state.any()
    with pytest.raises(RuntimeError):
        m.mem.fork(_i32([0]), _i32([1]), _i32([3]))           # nothing to fork from
    cuda_lib.last_device_status()


def test_the_models_memory_refuses_what_would_break_it(cuda_lib):
    """Rows that do not exist, children that hold pages, cuts inside shared pages: an error, and everything as it was."""
    m = draft_step.HybridLayers(3, 2, 64, 1, 20, 8, 6)
    m.reserve(16)                                             # two pages each
    m.context_lens += 16
    m.state.normal_()
    m.release(_i32([16, 0, 16]))
    m.fork(_i32([0]), _i32([1]), _i32([16]))                  # both pages shared
    before = [t.clone() for t in (m.pages_held, m.context_lens, m.shares, m.free_pages, m.state)]
    same = lambda: all(torch.equal(a, b) for a, b in zip(before, (m.pages_held, m.context_lens, m.shares, m.free_pages, m.state)))
    for parents, children in (([0], [3]), ([-1], [1]), ([7], [1])):
        with pytest.raises(ValueError):
            m.fork(_i32(parents), _i32(children), _i32([3]))
        assert same()
    with pytest.raises(RuntimeError):
        m.fork(_i32([0]), _i32([2]), _i32([16]))              # holds as many pages already
    assert same()
    for keep in ([13, 16, 16], [5, 0, 0], [16, -1, 16]):
        with pytest.raises(RuntimeError):
            m.release(_i32(keep))
        assert same()
    m.release(_i32([8, 16, 3]))
    assert m.context_lens.tolist() == [8, 16, 3] and m.pages_held.tolist() == [1, 2, 1] and m.shares.sum() == 1
    assert cuda_lib.last_device_status() in (cuda_lib.KDA_OK, cuda_lib.KDA_ERR_INVALID_ARG)
