"""The draft step's calls at both sides of what their kernels choose between, and as programs hold
them: prologue words and gates at every node count's form, units dealt in runs, calls captured in a CUDA graph,
one workspace for calls of different shapes."""
import numpy as np
import pytest
import torch

import _draft_ref as R
import kda_workloads as W
import oracle
from _parity import check

pytestmark = pytest.mark.gpu
ORDER = ("q", "k", "v", "g", "beta")


def _draws(B, K, H, D, dtype, seed, raw=False):
    inp = W.make_decode_inputs(W.DecodeConfig("tree", B, H, D, D, dtype, K), seed=seed, raw=raw)
    return {n: inp[n].transpose(0, 1).contiguous() for n in ORDER}, inp["state0"]


@pytest.mark.parametrize("word", [1, 2, 4, 7])
@pytest.mark.parametrize("K", [9, 14, 16, 17, 40, 64])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 128), (torch.bfloat16, 64), (torch.float32, 64)],
                         ids=["bf16-128", "fp32-128", "bf16-64", "fp32-64"])
def test_tree_prologue_words_and_gate(cuda_lib, dtype, D, K, word):
    """Each word's inputs raw, the others as they are; step with and without a gate, then the commit of a path.

    Bars as elsewhere: 1e-4 of the RMS (the fast sigmoid is a few ulp from the exact one), 2e-2 where a
    bf16 normalisation may round the other way."""
    B, H = 2, 2
    raw, s0 = _draws(B, K, H, D, dtype, seed=100 + K, raw=True)
    done, _ = _draws(B, K, H, D, dtype, seed=100 + K)
    bit = {"q": 1, "k": 1, "g": 2, "beta": 4, "v": 0}
    x = {n: raw[n] if word & bit[n] else done[n] for n in ORDER}
    flat = oracle.prologue({n: x[n].reshape(B * K, *x[n].shape[2:]) for n in ORDER}, word)
    ref_in = {n: flat[n].reshape(x[n].shape) for n in ORDER}
    parents = R.trees("ragged" if K % 2 else "random", B, K, seed=K)
    ref_o, ref_w, states = R.kda_tree(ref_in, s0, parents)
    tol = 2e-2 if dtype == torch.bfloat16 and word & 1 else 1e-4
    z = W.make_gate_logits((B, K, H, D), seed=4)
    dev = {n: x[n].cuda() for n in ORDER}
    for gate in (None, z):
        out, writes = cuda_lib.tree_decode(*(dev[n] for n in ORDER), torch.from_numpy(parents).cuda(), s0.cuda(), prologue=word,
                                           gate=None if gate is None else gate.cuda())
        check("out", out, ref_o if gate is None else oracle.output_gate(ref_o, gate), tol)
        check("writes", writes, ref_w, tol)
    path, n = np.full((B, K), -1, np.int32), np.zeros(B, np.int32)
    ends = [max(states[b]) for b in range(B)]
    for b in range(B):
        p = R.path_to(parents[b], ends[b])
        path[b, :len(p)], n[b] = p, len(p)
    state = s0.cuda()
    cuda_lib.tree_commit(dev["k"], dev["g"], writes, torch.from_numpy(path).cuda(), torch.from_numpy(n).cuda(), state, prologue=word)
    check("state", state, np.stack([states[b][ends[b]] for b in range(B)]), tol)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("K", [1, 5, 14])
def test_units_dealt_in_runs(cuda_lib, K):
    """695 x 7 units, the last run one unit short of nothing: the same bits as a few sequences alone, and the oracle's."""
    B, H, D = 695, 7, 128
    g = torch.Generator(device="cuda").manual_seed(K)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1).bfloat16()
    x = {"q": unit(rnd(B, K, H, D)), "k": unit(rnd(B, K, H, D)), "v": rnd(B, K, H, D).bfloat16(),
         "g": -5 * torch.sigmoid(rnd(B, K, H, D)), "beta": torch.sigmoid(rnd(B, K, H))}
    s0 = rnd(B, H, D, D) * 0.02
    parents = R.trees("random", B, K, seed=K)
    run = lambda at: cuda_lib.tree_decode(*(x[n][at].contiguous() for n in ORDER), torch.from_numpy(parents[at]).cuda(), s0[at].contiguous())
    out, writes = run(slice(None))
    some = [0, 1, 2, 173, 346, 520, 692, 693, 694]
    few = run(some)
    assert torch.equal(out[some], few[0]) and torch.equal(writes[some], few[1])
    ends = [0, 346, 694]
    ref_o, ref_w, _ = R.kda_tree({n: x[n][ends].cpu() for n in ORDER}, s0[ends].cpu(), parents[ends])
    check("out", out[ends], ref_o, 1e-4)
    check("writes", writes[ends], ref_w, 1e-4)


@pytest.mark.parametrize("K", [12, 13, 14, 15, 16])
def test_one_sequence_at_the_change_of_groups(cuda_lib, K):
    """One user's 96 heads: fewer units than CTAs, where the second group of a CTA has none."""
    x, s0 = _draws(1, K, 96, 128, torch.bfloat16, seed=K)
    parents = R.trees("random", 1, K, seed=K)
    ref_o, ref_w, _ = R.kda_tree(x, s0, parents)
    out, writes = cuda_lib.tree_decode(*(x[n].cuda() for n in ORDER), torch.from_numpy(parents).cuda(), s0.cuda())
    check("out", out, ref_o, 1e-4)
    check("writes", writes, ref_w, 1e-4)


# ------------------------------------------------------------------ as a program holds them
class _Step:
    """Inputs of all five calls in fixed tensors."""

    def __init__(self, D, dtype, seed, B=3, K=6, H=4, Hk=2, V=1031, ps=8):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.shape = B, K, H, Hk, D, V, ps
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        f = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
        self.x = {"q": f(B, K, H, D, dt=dtype), "k": f(B, K, H, D, dt=dtype), "v": f(B, K, H, D, dt=dtype), "g": f(B, K, H, D), "beta": f(B, K, H)}
        self.state, self.kv, self.aq = f(B, H, D, D), f(40, 2, ps, Hk, D, dt=dtype), f(B, K, H, D, dt=dtype)
        self.ctx, self.new, self.held, self.table, self.free = i32(B), i32(B), i32(B), i32(B, 9), i32(40)
        self.parents, self.tokens, self.u = i32(B, K), i32(B, K), f(B, K)
        self.first, self.one = i32(B, K), i32(B) + 1
        self.target, self.noise = f(B, K + 1, V), f(B, V)
        self.draw(seed)

    def draw(self, seed):
        """Other inputs in the same tensors."""
        B, K, H, Hk, D, V, ps = self.shape
        rnd = lambda t: torch.randn(t.shape, generator=self.gen, device="cuda")
        for n in "qk":
            self.x[n].copy_(torch.nn.functional.normalize(rnd(self.x[n]), dim=-1))
        self.x["v"].copy_(rnd(self.x["v"]))
        self.x["g"].copy_(-5 * torch.sigmoid(rnd(self.x["g"])))
        self.x["beta"].copy_(torch.sigmoid(rnd(self.x["beta"])))
        for t in (self.state, self.kv, self.aq):
            t.copy_(rnd(t))
        r = np.random.default_rng(seed)
        ctx = r.integers(0, 50, B)
        self.ctx.copy_(torch.from_numpy(ctx.astype(np.int32)))
        self.new.fill_(K)
        self.held.copy_(torch.from_numpy((-(-ctx // ps)).astype(np.int32)))
        ids = r.permutation(40).astype(np.int32)
        self.table.copy_(torch.from_numpy(np.resize(ids, (B, 9))))
        self.free.copy_(torch.from_numpy(ids))
        self.parents.copy_(torch.from_numpy(R.trees("random", B, K, seed)))
        self.target.copy_(torch.softmax(2 * rnd(self.target), -1))
        self.tokens.copy_(self.target[:, :1].topk(K, -1).indices[:, 0])
        self.u.copy_(torch.rand(self.u.shape, generator=self.gen, device="cuda"))
        self.noise.exponential_(generator=self.gen).clamp_min_(1e-30)

    def run(self, kda):
        ps = self.shape[-1]
        B, K = self.parents.shape
        tables = kda.page_tables(self.ctx, self.new, self.held, self.table, self.free, page_size=ps, max_tokens=B * K)
        att = kda.tree_attention(self.aq, self.kv[:, 0], self.kv[:, 1], self.table, self.ctx, self.parents)
        out, writes = kda.tree_decode(*(self.x[n] for n in ORDER), self.parents, self.state)
        path, n, nxt = kda.verify_drafts(self.target, self.tokens, self.parents, self.u, self.noise)
        kda.tree_commit(self.x["k"], self.x["g"], writes, path, n, self.state)
        kda.tree_commit(self.x["k"], self.x["g"], writes, self.first, self.one, self.state)    # (and where nothing was kept)
        return [*tables, self.table, att, out, writes, path, n, nxt, self.state]


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float32)], ids=["bf16-128", "fp32-64"])
def test_a_step_in_a_cuda_graph(cuda_lib, D, dtype):
    """Captured once, replayed on other inputs: what the calls give outside a graph."""
    s = _Step(D, dtype, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(cuda_lib)                                  # (each kernel is set up at its first call)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = s.run(cuda_lib)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (2, 3):
        s.draw(seed)
        keep = s.table.clone(), s.state.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        s.table.copy_(keep[0])
        s.state.copy_(keep[1])
        want = s.run(cuda_lib)
        assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        assert not torch.equal(got[-1], keep[1])


def test_one_workspace_for_calls_of_different_shapes(cuda_lib):
    """What a call leaves in the workspace (parts, records of what to join) is not another call's."""
    shapes = [(128, torch.bfloat16, 64, 8, 2, (9000, 40)), (128, torch.bfloat16, 1, 8, 2, (300, 3)), (64, torch.bfloat16, 5, 6, 2, (0, 2000)),
              (64, torch.float32, 5, 6, 2, (700, 0)), (128, torch.float32, 33, 4, 1, (1500, 20)), (128, torch.bfloat16, 64, 8, 2, (9000, 40)),
              (128, torch.bfloat16, 2, 2, 2, (1, 0))]
    g = torch.Generator(device="cuda").manual_seed(3)
    work = torch.full((64 << 20,), 0x7f, dtype=torch.uint8, device="cuda")
    for D, dtype, K, H, Hk, lens in shapes:
        ps, B = 16, len(lens)
        pages = [-(-(n + K) // ps) for n in lens]
        kv = torch.randn(sum(pages), 2, ps, Hk, D, generator=g, device="cuda").to(dtype)
        table = torch.full((B, max(pages)), -1, dtype=torch.int32)
        for b in range(B):
            table[b, :pages[b]] = torch.arange(sum(pages[:b]), sum(pages[:b + 1]))
        q = torch.randn(B, K, H, D, generator=g, device="cuda").to(dtype)
        args = (q, kv[:, 0], kv[:, 1], table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                torch.from_numpy(R.trees("random", B, K, K)).cuda())
        want = cuda_lib.tree_attention(*args)
        assert torch.equal(cuda_lib.tree_attention(*args, workspace=work), want)
        assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
