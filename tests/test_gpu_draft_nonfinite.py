"""Infinities and NaN in the inputs of KDA on draft trees (and of the verification): what they reach, and nothing else.

A NaN has more than one bit pattern: what the GPU's own arithmetic produces is 0x7fffffff, what
torch writes is 0x7fc00000, and any payload may come from elsewhere."""
import numpy as np
import pytest
import torch

import _draft_ref as R
import kda_workloads as W
from _parity import check

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)]
IDS = ["bf16-128", "bf16-64", "fp32-128", "fp32-64"]
ORDER = ("q", "k", "v", "g", "beta")


def _inputs(B, K, H, D, dtype, seed):
    inp = W.make_decode_inputs(W.DecodeConfig("tree", B, H, D, D, dtype, K), seed=seed)
    return {n: inp[n].transpose(0, 1).contiguous().cuda() for n in ORDER}, inp["state0"].cuda()


def _step(kda, x, parents, state, **kw):
    out, writes = kda.tree_decode(*(x[n] for n in ORDER), torch.from_numpy(parents).cuda(), state, **kw)
    torch.cuda.synchronize()
    assert kda.last_device_status() == kda.KDA_OK
    return out.cpu(), writes.cpu()


def _bits(word):
    return torch.tensor([word - (1 << 32) if word >= 1 << 31 else word], dtype=torch.int32, device="cuda").view(torch.float32)


@pytest.mark.parametrize("K", [1, 5, 16, 20])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_tree_decode_shows_a_diverged_state(cuda_lib, dtype, D, K):
    """One NaN or infinite element of a state: its value channel of that head, in every node, and nothing else."""
    B, H, b, h, c, d = 2, 3, 1, 2, 37, 11
    x, s0 = _inputs(B, K, H, D, dtype, seed=5 + K)
    parents = R.trees("random", B, K, seed=K)
    clean = _step(cuda_lib, x, parents, s0)
    inf = torch.full((1,), float("inf"), device="cuda")
    words = {"inf - inf": inf - inf, "inf": inf, "-inf": -inf}
    words.update({hex(w): _bits(w) for w in (0x7fffffff, 0xffffffff, 0x7fc00000, 0x7f800001, 0xff801234)})
    for name, word in words.items():
        state = s0.clone()
        state[b, h, c, d:d + 1] = word
        for what, got, want in zip(("out", "writes"), _step(cuda_lib, x, parents, state), clean):
            hit = torch.zeros(B, K, H, D, dtype=torch.bool)
            hit[b, :, h, d] = True
            assert torch.equal(got[~hit], want[~hit]), (name, what)
            assert not got[hit].isfinite().any(), (name, what)
            if "inf" not in name or name == "inf - inf":
                assert got[hit].isnan().all(), (name, what)


@pytest.mark.parametrize("word", [0x7fffffff, 0xffffffff, 0x7fc00000])
@pytest.mark.parametrize("K,j", [(5, 2), (16, 3), (20, 1), (40, 18)])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_tree_decode_passes_on_a_nodes_nan(cuda_lib, dtype, D, K, j, word):
    """A NaN in one node's row: that node and those below it (q: that node's output alone)."""
    B, H, h, c = 1, 2, 1, 50
    x, s0 = _inputs(B, K, H, D, dtype, seed=9 + K)
    parents = R.trees("random", B, K, seed=K + 1)
    below = torch.tensor([j in R.path_to(parents[0], i) for i in range(K)])
    own = torch.arange(K) == j
    clean = _step(cuda_lib, x, parents, s0)
    for name in ORDER:
        bad = {n: x[n].clone() for n in ORDER}
        at = bad[name][0, j, h]
        (at if name == "beta" else at[c:c + 1]).copy_(_bits(word).to(bad[name].dtype).squeeze(0) if name == "beta" else _bits(word).to(bad[name].dtype))
        got = _step(cuda_lib, bad, parents, s0)
        for what, g, w in zip(("out", "writes"), got, clean):
            hit = torch.zeros(B, K, H, D, dtype=torch.bool)
            nodes = own & (what == "out") if name == "q" else below
            if name == "v":
                hit[0, nodes, h, c] = True
            else:
                hit[0, nodes, h] = True
            assert torch.equal(g[~hit], w[~hit]), (name, what)
            assert g[hit].isnan().all(), (name, what)


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_tree_commit_shows_what_is_on_the_path(cuda_lib, dtype, D):
    """A NaN state element stays; rows that the path does not name are not looked at."""
    B, K, H = 2, 6, 2
    x, s0 = _inputs(B, K, H, D, dtype, seed=3)
    w = torch.randn(B, K, H, D, device="cuda")
    path = torch.tensor([[0, 2, 5, -1, -1, -1]] * B, dtype=torch.int32, device="cuda")
    n = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    clean = cuda_lib.tree_commit(x["k"], x["g"], w, path, n, s0.clone())
    bad = {m: x[m].clone() for m in ("k", "g")}
    for t in (bad["k"], bad["g"], w):
        t[:, [1, 3, 4]] = float("nan")
    state = s0.clone()
    state[1, 1, 7, 9:10] = _bits(0x7fffffff)
    cuda_lib.tree_commit(bad["k"], bad["g"], w, path, n, state)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    hit = torch.zeros(B, H, D, D, dtype=torch.bool, device="cuda")
    hit[1, 1, 7, 9] = True
    assert state[hit].isnan().all() and torch.equal(state[~hit], clean[~hit])


@pytest.mark.parametrize("K", [6, 16, 40])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_absent_nodes_are_zero_whatever_their_rows_hold(cuda_lib, dtype, D, K):
    """NaN in every input row of the absent nodes, the output gate's logits among them."""
    B, H = 3, 2
    x, s0 = _inputs(B, K, H, D, dtype, seed=2 + K)
    parents = R.trees("ragged", B, K, seed=K)
    gone = torch.from_numpy(parents == R.PAD)
    assert gone.any()
    z = torch.randn(B, K, H, D, device="cuda")
    clean = _step(cuda_lib, x, parents, s0, gate=z)
    for t in (*x.values(), z):
        t[gone.cuda()] = float("nan")
    for what, got, want in zip(("out", "writes"), _step(cuda_lib, x, parents, s0, gate=z), clean):
        assert not got[gone].any(), what
        assert torch.equal(got, want), what


def _with_resets(x, seed):
    """g with whole nodes and single channels at what e^g = 0 may look like."""
    r = np.random.default_rng(seed)
    g = x["g"].clone()
    low = torch.tensor([-np.inf, -np.finfo(np.float32).max, -200.0, -1e4], dtype=torch.float32)
    put = torch.from_numpy(r.random(g.shape) < 0.08)
    pick = low[torch.from_numpy(r.integers(0, 4, g.shape))]
    g[put] = pick[put]
    g[0, g.shape[1] // 2] = -np.inf
    return {**x, "g": g}


@pytest.mark.parametrize("kind,K", [("chain", 1), ("chain", 7), ("random", 16), ("binary", 33), ("chain", 33), ("ragged", 64)])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_resets_of_the_state(cuda_lib, dtype, D, kind, K):
    """g = -inf (or any g whose e^g is zero) forgets what lies before the node and nothing after it.

    Bar: 1e-4 of the RMS, as without resets.  A reset counts as some 150 powers of two in G, so a pair's
    factor has a rounding error of 2^-25 |G| ln 2 for each node between the two: 2e-5 for the
    five resets (|G| < 1024) that a path of 33 nodes has in one channel, and the pairs that matter
    (e^g of 1/12 a node on average) have one to three nodes between them."""
    B, H = 2, 2
    x, s0 = _inputs(B, K, H, D, dtype, seed=60 + K)
    x, s0 = {n: x[n].cpu() for n in ORDER}, s0.cpu()
    x = _with_resets(x, K)
    parents = R.trees(kind, B, K, seed=K)
    ref_o, ref_w, states = R.kda_tree(x, s0, parents)
    out, writes = _step(cuda_lib, {n: x[n].cuda() for n in ORDER}, parents, s0.cuda())
    check("out", out, ref_o, 1e-4)
    check("writes", writes, ref_w, 1e-4)
    ends = [max(states[b]) for b in range(B)]
    path = np.full((B, K), -1, np.int32)
    n = np.zeros(B, np.int32)
    for b in range(B):
        p = R.path_to(parents[b], ends[b])
        path[b, :len(p)], n[b] = p, len(p)
    state = s0.cuda()
    cuda_lib.tree_commit(x["k"].cuda(), x["g"].cuda(), writes.cuda(), torch.from_numpy(path).cuda(), torch.from_numpy(n).cuda(), state)
    check("state", state, np.stack([states[b][ends[b]] for b in range(B)]), 1e-4)


@pytest.mark.parametrize("V", [9, 1031, 20011])
@pytest.mark.parametrize("draft", [False, True])
def test_verify_of_probabilities_that_are_none(cuda_lib, draft, V):
    """NaN beside the drafted tokens counts as zero; a whole row of NaN keeps nothing and still names a token."""
    r = np.random.default_rng(V)
    B, K = 6, 2
    target = r.random((B, K + 1, V), dtype=np.float32)
    target /= target.sum(-1, keepdims=True)
    tokens = np.tile(np.array([[1, 2]], np.int32), (B, 1))
    parents = np.tile(np.array([[-1, 0]], np.int32), (B, 1))
    q = r.random((B, K, V), dtype=np.float32) if draft else None
    u, noise = r.random((B, K), dtype=np.float32), r.random((B, V), dtype=np.float32) + np.float32(0.1)
    none = r.random((B, K + 1, V)) < 0.3
    none[:, :, 1:3] = False
    c = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    run = lambda p: [x.tolist() for x in cuda_lib.verify_drafts(c(p), c(tokens), c(parents), c(u), c(noise), draft_probs=c(q))]
    want = R.verify(np.where(none, np.float32(0), target), q, tokens, parents, u, noise)
    assert run(np.where(none, np.float32("nan"), target)) == [x.tolist() for x in want]
    path, n, nxt = run(np.full_like(target, np.float32("nan")))
    assert n == [0] * B and path == [[-1] * K] * B and all(0 <= t < V for t in nxt)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
