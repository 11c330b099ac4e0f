"""GPU parity of kda_tree_attention against the definition in 64 bits.

Bounds, elementwise, from the arithmetic (_draft_ref.attention): a score is a sum of D fp32
products, so it is within (D + 4) 2^-24 of sum |q| |k| times the scale (and a few ulp of itself for the change of base);
its weight's relative error is at most twice that through the softmax's quotient, plus the
exponentials' and the sums' roundings; all of it times sum w |v|.  bf16 adds the rounding of
the weights (2^-9 of sum w |v|, twice: once in the weight, once against the sum that keeps it) and that of the output (2^-8 |out|)."""
import numpy as np
import pytest
import torch

import _draft_ref as R

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)]
IDS = ["bf16-128", "bf16-64", "fp32-128", "fp32-64"]


def _make(lens, K, H, Hk, D, dtype, ps, seed=0, poison=True, fused=True, spare=3):
    """q, caches, table, ctx: every cache row that no sequence owns is NaN (poison)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [-(-(n + K) // ps) for n in lens]
    P, cols = sum(pages) + spare, max(pages) + 1
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((B, cols), 0x7fffffff, dtype=torch.int32)
    kv = torch.full((P, 2, ps, Hk, D), float("nan") if poison else 0.0)
    at = 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        for t in range(n + K):
            kv[int(table[b, t // ps]), :, t % ps] = torch.randn(2, Hk, D, generator=g)
    kv = kv.to(dtype)
    q = torch.randn(B, K, H, D, generator=g).to(dtype)
    return q, kv, table, torch.tensor(lens, dtype=torch.int32)


def _check(kda, q, kv, table, ctx, parents, scale=None, fused=True, status=None, **kw):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    dev = kv.cuda()
    k, v = (dev[:, 0], dev[:, 1]) if fused else (dev[:, 0].contiguous(), dev[:, 1].contiguous())
    out = kda.tree_attention(q.cuda(), k, v, table.cuda(), ctx.cuda(), torch.from_numpy(parents).cuda(), scale=scale, **kw)
    torch.cuda.synchronize()
    assert kda.last_device_status() == (kda.KDA_OK if status is None else status)
    ref, bound, mass = R.attention(q, kv[:, 0], kv[:, 1], table, ctx, parents, scale)
    if q.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    off = (got - ref).abs() - bound
    assert (off <= 0).all(), f"{float(off.max()):.3e} over the bound at {tuple(np.unravel_index(int(off.argmax()), off.shape))}"
    return out


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("K,H,Hk,kind", [(1, 2, 2, "chain"), (1, 8, 1, "chain"), (5, 6, 2, "random"), (8, 4, 4, "ragged"),
                                         (16, 12, 1, "binary"), (33, 5, 1, "random"), (64, 4, 1, "ragged"), (64, 12, 1, "chain")])
def test_attention_matches_definition(cuda_lib, dtype, D, K, H, Hk, kind):
    lens = [0, 1, 63, 64, 130, 391]
    x = _make(lens, K, H, Hk, D, dtype, ps=16, seed=K)
    _check(cuda_lib, *x, R.trees(kind, len(lens), K, seed=K))


@pytest.mark.parametrize("dtype,D", TYPES[:1] + TYPES[3:], ids=IDS[:1] + IDS[3:])
@pytest.mark.parametrize("ps", [1, 7, 8, 24, 64, 100, 128, 256, 1000])
def test_attention_page_sizes(cuda_lib, dtype, D, ps):
    """Pages that end inside a tile, tiles that end inside a page; lengths around both."""
    lens = [ps - 1, ps, ps + 1, 127, 128, 129, 0, 255 + ps]
    x = _make(lens, 3, 6, 2, D, dtype, ps=ps, seed=ps)
    _check(cuda_lib, *x, R.trees("random", len(lens), 3, seed=ps), fused=ps % 2 == 0)


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("lens,K,H,Hk", [([9000], 2, 2, 1), ([5000, 3], 20, 16, 2), ([3, 4000, 1, 2500], 64, 3, 1), ([20000], 1, 1, 1)])
def test_attention_long_contexts_are_split(cuda_lib, dtype, D, lens, K, H, Hk):
    x = _make(lens, K, H, Hk, D, dtype, ps=64, seed=1)
    parents = R.trees("ragged", len(lens), K, seed=1)
    a = _check(cuda_lib, *x, parents)
    b = _check(cuda_lib, *x, parents)
    assert torch.equal(a, b), "two runs differ"


@pytest.mark.parametrize("ps", [16, 20], ids=["boxes", "gathered"])
@pytest.mark.parametrize("ctx", [0, 100, 126, 1000])
def test_attention_passes_on_what_a_node_sees(cuda_lib, ctx, ps):
    """One infinite or NaN value of one node: that channel, in the rows that see the node, and nothing else."""
    K, G, D = 40, 3, 128
    q, kv, table, lens = _make([ctx], K, G, 1, D, torch.bfloat16, ps=ps, seed=ctx)
    parents = R.trees("random", 1, K, seed=1)
    clean = _check(cuda_lib, q, kv, table, lens, parents)
    for node, chan, what in ((2, 5, float("inf")), (30, 127, float("-inf")), (39, 0, float("nan"))):
        bad = kv.clone()
        bad[int(table[0, (ctx + node) // ps]), 1, (ctx + node) % ps, 0, chan] = what
        dev = bad.cuda()
        out = cuda_lib.tree_attention(q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), lens.cuda(), torch.from_numpy(parents).cuda())
        sees = torch.tensor([node in R.path_to(parents[0], i) for i in range(K)])
        hit = torch.zeros(1, K, G, D, dtype=torch.bool)
        hit[0, sees, :, chan] = True
        assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])
        want = torch.full_like(out.cpu()[hit], what)
        assert torch.equal(out.cpu()[hit].isnan(), want.isnan()) and (want.isnan() | (out.cpu()[hit] == want)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_attention_ignores_other_paths_and_absent_nodes(cuda_lib, dtype):
    """NaN and infinities in the rows of nodes that only some nodes may see, and of absent ones."""
    K, lens = 8, [0, 50, 126, 1000]
    q, kv, table, ctx = _make(lens, K, 6, 2, 128, dtype, ps=16, seed=3)
    parents = np.array([[-1, -1, 0, 1, 2, 2, 3, -2]] * 4, np.int32)
    clean = _check(cuda_lib, q, kv, table, ctx, parents)
    bad = kv.clone()
    for b, n in enumerate(lens):
        for node, what in ((1, float("nan")), (3, float("inf")), (6, float("-inf")), (7, float("nan"))):
            bad[int(table[b, (n + node) // 16]), :, (n + node) % 16] = what
    dev = bad.cuda()
    out = cuda_lib.tree_attention(q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), ctx.cuda(), torch.from_numpy(parents).cuda())
    assert torch.equal(out[:, [0, 2, 4, 5, 7]], clean[:, [0, 2, 4, 5, 7]])
    assert out[:, [1, 6]].isnan().all() and not out[:, 3].isfinite().any()      # 6 hangs on 3: inf - inf


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 30.0])
def test_attention_scales(cuda_lib, dtype, scale):
    """Uniform weights, negative ones, and scores of several thousand."""
    x = _make([7, 300], 4, 4, 2, 64, dtype, ps=32, seed=6)
    _check(cuda_lib, *x, R.trees("chain", 2, 4), scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_attention_lowest_scores(cuda_lib, dtype):
    """Every visible score the lowest the type can give: still the mean over what is visible."""
    q, kv, table, ctx = _make([100], 2, 2, 1, 64, dtype, ps=16, seed=6)
    big = 1e30 if dtype == torch.float32 else 1e16
    q = torch.zeros_like(q)
    q[..., 0] = -big
    kv[:, 0] = torch.where(kv[:, 0].isnan(), kv[:, 0], 0.0)
    kv[:, 0, :, :, 0] = torch.where(kv[:, 0, :, :, 0].isnan(), kv[:, 0, :, :, 0], 3e8 if dtype == torch.float32 else 1e16)
    out = cuda_lib.tree_attention(q.cuda(), kv.cuda()[:, 0], kv.cuda()[:, 1], table.cuda(), ctx.cuda(),
                                  torch.from_numpy(R.trees("chain", 1, 2)).cuda())
    rows = lambda n: torch.stack([kv[int(table[0, t // 16]), 1, t % 16, 0].double() for t in range(n)]).mean(0)
    for i in range(2):
        assert (out[0, i].cpu().double() - rows(101 + i)).abs().max() < 2e-2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_attention_reports_bad_input_and_goes_on(cuda_lib, dtype):
    q, kv, table, ctx = _make([40, 200, 30, 90], 4, 4, 2, 128, dtype, ps=16, seed=8)
    parents = R.trees("chain", 4, 4)
    bad = cuda_lib.KDA_ERR_INVALID_ARG
    t = table.clone()
    t[1, 3], t[1, 5] = -1, kv.shape[0]                 # pages that are not there: left out
    _check(cuda_lib, q, kv, t, ctx, parents, status=bad)
    for b, value in ((0, -1), (2, table.shape[1] * 16 - 3)):
        c = ctx.clone()
        c[b] = value
        want = R.attention(q, kv[:, 0], kv[:, 1], table, ctx, parents, 128 ** -0.5)[0]
        dev = kv.cuda()
        out = cuda_lib.tree_attention(q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), c.cuda(), torch.from_numpy(parents).cuda())
        assert cuda_lib.last_device_status() == bad
        assert not out[b].any()
        rest = [i for i in range(4) if i != b]
        assert (out[rest].cpu().double() - want[rest]).abs().max() < 3e-2
    p = parents.copy()
    p[3, 2] = 2
    dev = kv.cuda()
    out = cuda_lib.tree_attention(q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), ctx.cuda(), torch.from_numpy(p).cuda())
    assert cuda_lib.last_device_status() == bad and not out[3].any() and out[:3].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_attention_offsets_past_32_bits(cuda_lib, dtype):
    """A cache of more than 2^31 elements, the sequence's pages at its two ends."""
    ps, Hk, D, K, n = 64, 8, 128, 3, 200
    P = 2 ** 31 // (2 * ps * Hk * D) + 40
    kv = torch.empty((P, 2, ps, Hk, D), dtype=dtype, device="cuda")
    table = torch.tensor([[P - 1, 0, P - 2, P // 2 + 17]], dtype=torch.int32)
    for p in table[0].tolist():
        kv[p].normal_()
    q = torch.randn(1, K, 16, D, device="cuda").to(dtype)
    ctx, parents = torch.tensor([n], dtype=torch.int32), R.trees("chain", 1, K)
    out = cuda_lib.tree_attention(q, kv[:, 0], kv[:, 1], table.cuda(), ctx.cuda(), torch.from_numpy(parents).cuda())
    small = kv[table[0].long().cuda()].cpu()
    ref, bound, mass = R.attention(q, small[:, 0], small[:, 1], torch.tensor([[0, 1, 2, 3]]), ctx, parents, D ** -0.5)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
    assert ((out.cpu().double() - ref).abs() <= bound).all()


def test_attention_many_sequences_and_another_stream(cuda_lib):
    lens = [(37 * i) % 160 for i in range(333)]
    q, kv, table, ctx = _make(lens, 2, 2, 1, 64, torch.bfloat16, ps=32, seed=4)
    parents = R.trees("random", len(lens), 2)
    side = torch.cuda.Stream()
    dev = kv.cuda()
    args = (q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), ctx.cuda(), torch.from_numpy(parents).cuda())
    side.wait_stream(torch.cuda.current_stream())
    out = cuda_lib.tree_attention(*args, stream=side)
    side.synchronize()
    assert torch.equal(out, _check(cuda_lib, q, kv, table, ctx, parents))


def test_attention_nothing_to_do(cuda_lib):
    q, kv, table, ctx = _make([5], 2, 2, 1, 64, torch.bfloat16, ps=32, seed=4)
    out = cuda_lib.tree_attention(q[:0].cuda(), kv.cuda()[:, 0], kv.cuda()[:, 1], table[:0].cuda(), ctx[:0].cuda(),
                                  torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 2, 64)
    empty = kv[:0].cuda()                     # no pages at all: every token is left out
    out = cuda_lib.tree_attention(q.cuda(), empty[:, 0], empty[:, 1], table.cuda(), ctx.cuda(),
                                  torch.tensor([[-1, 0]], dtype=torch.int32, device="cuda"))
    assert not out.any() and cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
