"""GPU parity of KDA on draft trees (kda_tree_decode, kda_tree_commit) against the fp64
recurrence run along every node's own path.

Bar: max |error| / RMS <= 1e-4 for both input types (the oracle reads the stored inputs and
the kernels compute in fp32 from them: K <= 64 steps of sums over 128 terms, each within a few
hundred roundings of 2^-24); with the q/k normalisation in bf16, whose rounding may fall the
other way, the bf16 bar of the other kernels, 2e-2."""
import numpy as np
import pytest
import torch

import _draft_ref as R
import kda_workloads as W
import oracle
from _parity import check

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)]
IDS = ["bf16-128", "bf16-64", "fp32-128", "fp32-64"]


def _inputs(B, K, H, D, dtype, seed, raw=False):
    inp = W.make_decode_inputs(W.DecodeConfig("tree", B, H, D, D, dtype, K), seed=seed, raw=raw)
    return {n: inp[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "g", "beta")}, inp["state0"]


def _run(kda, x, parents, s0, **kw):
    state = s0.cuda()
    out, writes = kda.tree_decode(*(x[n].cuda() for n in ("q", "k", "v", "g", "beta")), torch.from_numpy(parents).cuda(),
                                  state, **kw)
    torch.cuda.synchronize()
    assert torch.equal(state.cpu(), s0), "the state was changed"
    return out, writes


@pytest.mark.parametrize("kind", ["chain", "star", "binary", "ragged"])
@pytest.mark.parametrize("K", [1, 2, 7, 16, 33, 64])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_tree_decode_matches_oracle(cuda_lib, dtype, D, K, kind):
    B, H = 3, 2
    x, s0 = _inputs(B, K, H, D, dtype, seed=10 + K)
    parents = R.trees(kind, B, K, seed=K)
    ref_o, ref_w, _ = R.kda_tree(x, s0, parents)
    out, writes = _run(cuda_lib, x, parents, s0)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    check("out", out, ref_o, 1e-4)
    check("writes", writes, ref_w, 1e-4)
    absent = torch.from_numpy(parents == R.PAD)
    assert not out.cpu()[absent].any() and not writes.cpu()[absent].any()


@pytest.mark.parametrize("B,H,K", [(1, 1, 3), (5, 38, 8), (40, 7, 16), (9, 96, 5)])
def test_tree_decode_shapes(cuda_lib, B, H, K):
    x, s0 = _inputs(B, K, H, 128, torch.bfloat16, seed=3)
    parents = R.trees("random", B, K, seed=5)
    ref_o, ref_w, _ = R.kda_tree(x, s0, parents)
    out, writes = _run(cuda_lib, x, parents, s0)
    check("out", out, ref_o, 1e-4)
    check("writes", writes, ref_w, 1e-4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_tree_prologue_gate_and_commit(cuda_lib, dtype):
    """From raw draws: prologue in both calls, the gate on the output only."""
    B, K, H, D = 4, 9, 3, 128
    raw, s0 = _inputs(B, K, H, D, dtype, seed=21, raw=True)
    pro = oracle.prologue({n: raw[n].reshape(B * K, *raw[n].shape[2:]) for n in raw}, cuda_lib.KDA_PROLOGUE_ALL)
    x = {n: torch.as_tensor(np.asarray(pro[n])).reshape(raw[n].shape) if not isinstance(pro[n], torch.Tensor) else pro[n].reshape(raw[n].shape) for n in raw}
    parents = R.trees("random", B, K, seed=2)
    z = W.make_gate_logits((B, K, H, D), seed=4)
    ref_o, ref_w, states = R.kda_tree(x, s0, parents)
    out, writes = _run(cuda_lib, raw, parents, s0, prologue=cuda_lib.KDA_PROLOGUE_ALL, gate=z.cuda())
    tol = 2e-2 if dtype == torch.bfloat16 else 1e-4
    check("gated out", out, oracle.output_gate(ref_o, z), tol)
    check("writes", writes, ref_w, tol)
    path, n, want = _paths(parents, states, s0, [K - 1] * B)
    state = s0.cuda()
    cuda_lib.tree_commit(raw["k"].cuda(), raw["g"].cuda(), writes, path, n, state, prologue=cuda_lib.KDA_PROLOGUE_ALL)
    torch.cuda.synchronize()
    check("state", state, want, tol)


def _paths(parents, states, s0, ends):
    """path, n_accept on the GPU and the states they lead to (ends[b]: last accepted node, -1 = none)."""
    B, K = parents.shape
    path, n, want = np.full((B, K), -1, np.int32), np.zeros(B, np.int32), []
    for b in range(B):
        p = R.path_to(parents[b], ends[b]) if ends[b] >= 0 else []
        path[b, :len(p)], n[b] = p, len(p)
        want.append(states[b][ends[b]] if p else s0[b].double().numpy())
    return torch.from_numpy(path).cuda(), torch.from_numpy(n).cuda(), np.stack(want)


@pytest.mark.parametrize("kind,K", [("chain", 1), ("chain", 8), ("chain", 64), ("random", 16), ("binary", 31), ("ragged", 9)])
@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_tree_commit_matches_oracle(cuda_lib, dtype, D, kind, K):
    B, H = 5, 2
    x, s0 = _inputs(B, K, H, D, dtype, seed=40 + K)
    parents = R.trees(kind, B, K, seed=K)
    _, ref_w, states = R.kda_tree(x, s0, parents)
    ends = [-1 if b == 1 else max(i for i in states[b]) if b % 2 == 0 else min(states[b]) for b in range(B)]
    path, n, want = _paths(parents, states, s0, ends)
    state = s0.cuda()
    cuda_lib.tree_commit(x["k"].cuda(), x["g"].cuda(), torch.from_numpy(ref_w).float().cuda(), path, n, state)
    torch.cuda.synchronize()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    check("state", state, want, 1e-4)
    assert torch.equal(state[1].cpu(), s0[1])


def test_tree_chain_equals_decode_multi(cuda_lib):
    """A chain is decode_multi's drafts: outputs, and the state after n tokens of it."""
    B, K, H, D = 6, 7, 4, 128
    x, s0 = _inputs(B, K, H, D, torch.bfloat16, seed=8)
    parents = R.trees("chain", B, K)
    out, writes = _run(cuda_lib, x, parents, s0)
    n = torch.arange(B, dtype=torch.int32, device="cuda")
    ref = s0.cuda()
    want = cuda_lib.decode_multi(*(x[m].cuda() for m in ("q", "k", "v", "g", "beta")), ref, n_apply=n)
    state = s0.cuda()
    path = torch.arange(K, dtype=torch.int32, device="cuda").expand(B, K).contiguous()
    cuda_lib.tree_commit(x["k"].cuda(), x["g"].cuda(), writes, path, n, state)
    torch.cuda.synchronize()
    check("out", out, want.double().cpu().numpy(), 1e-4)
    check("state", state, ref.double().cpu().numpy(), 1e-4)


@pytest.mark.parametrize("bad", ["self", "forward", "below", "on_absent"])
def test_bad_trees_are_skipped_and_reported(cuda_lib, bad):
    B, K, H, D = 3, 6, 2, 128
    x, s0 = _inputs(B, K, H, D, torch.bfloat16, seed=9)
    good = R.trees("chain", B, K)
    parents = good.copy()
    if bad == "self":
        parents[1, 3] = 3
    elif bad == "forward":
        parents[1, 0] = 4
    elif bad == "below":
        parents[1, 5] = -3
    else:
        parents[1, 2] = R.PAD
    out = torch.full((B, K, H, D), 7.0, device="cuda")
    writes = out.clone()
    _run(cuda_lib, x, parents, s0, out=out, writes=writes)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    ref_o, ref_w, _ = R.kda_tree(x, s0, good)
    for b in (0, 2):
        check("out", out[b], ref_o[b], 1e-4)
        check("writes", writes[b], ref_w[b], 1e-4)
    assert (out[1] == 7).all() and (writes[1] == 7).all()


@pytest.mark.parametrize("n,entry", [(7, 0), (-1, 0), (2, 6), (2, -1)])
def test_bad_paths_leave_the_state(cuda_lib, n, entry):
    B, K, H, D = 2, 6, 2, 64
    x, s0 = _inputs(B, K, H, D, torch.float32, seed=9)
    w = torch.randn(B, K, H, D)
    path = torch.zeros(B, K, dtype=torch.int32)
    path[:, 1] = 1
    path[1, 1] = entry
    count = torch.tensor([1, n], dtype=torch.int32)
    state = s0.cuda()
    cuda_lib.tree_commit(x["k"].cuda(), x["g"].cuda(), w.cuda(), path.cuda(), count.cuda(), state)
    torch.cuda.synchronize()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    assert torch.equal(state[1].cpu(), s0[1]) and not torch.equal(state[0].cpu(), s0[0])


def test_tree_on_another_stream_and_nothing_to_do(cuda_lib):
    B, K, H, D = 4, 5, 3, 128
    x, s0 = _inputs(B, K, H, D, torch.bfloat16, seed=31)
    parents = R.trees("random", B, K)
    ref_o, _, _ = R.kda_tree(x, s0, parents)
    dev = {n: x[n].cuda() for n in x}
    p, state = torch.from_numpy(parents).cuda(), s0.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = cuda_lib.tree_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], p, state, stream=side)
    side.synchronize()
    check("out", out, ref_o, 1e-4)
    none = {n: dev[n][:0] for n in dev}
    out, writes = cuda_lib.tree_decode(none["q"], none["k"], none["v"], none["g"], none["beta"], p[:0], state[:0])
    assert out.shape == (0, K, H, D)
    cuda_lib.tree_commit(none["k"], none["g"], writes, p[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), state[:0])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_deep_decay_does_not_overflow(cuda_lib):
    """g = -5 on a chain of 64: e^{G_j - G_i} of the whole path is e^315, which no fp32 holds."""
    B, K, H, D = 1, 64, 1, 128
    x, s0 = _inputs(B, K, H, D, torch.float32, seed=77)
    x["g"] = torch.full_like(x["g"], -5.0)
    parents = R.trees("chain", B, K)
    ref_o, ref_w, states = R.kda_tree(x, s0, parents)
    out, writes = _run(cuda_lib, x, parents, s0)
    check("out", out, ref_o, 1e-4)
    check("writes", writes, ref_w, 1e-4)
    path, n, want = _paths(parents, states, s0, [K - 1])
    state = s0.cuda()
    cuda_lib.tree_commit(x["k"].cuda(), x["g"].cuda(), writes, path, n, state)
    check("state", state, want, 1e-4)
