"""GPU parity of kda_chunk_attention against the definition in 64 bits.

Bounds, elementwise, from the arithmetic (_prompt_ref.chunk_attention), as for the tree attention: the scores' fp32 sums, the
exponentials' and the sums' roundings; bf16 adds the rounding of the weights (2^-9 of sum w |v|, twice: once in the weight, once
against the sum that keeps it) and that of the output (2^-8 |out|, or half the least subnormal)."""
import numpy as np
import pytest
import torch

import _prompt_ref as R

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)]
IDS = ["bf16-128", "bf16-64", "fp32-128", "fp32-64"]
I32 = torch.int32


def _make(ctx, new, H, Hk, D, dtype, ps, seed=0, poison=True, behind=0):
    """q (and rows behind the last chunk), cache, table, context lengths, cu_seqlens."""
    kv, table = R.paged([c + n for c, n in zip(ctx, new)], Hk, D, dtype, ps, seed, poison)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=I32)
    q = torch.randn(int(cu[-1]) + behind, H, D, generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
    return q, kv, table, torch.tensor(ctx, dtype=I32), cu


def _run(kda, q, kv, table, ctx, cu, fused=True, **kw):
    dev = kv.cuda()
    k, v = (dev[:, 0], dev[:, 1]) if fused else (dev[:, 0].contiguous(), dev[:, 1].contiguous())
    return kda.chunk_attention(q.cuda(), k, v, table.cuda(), ctx.cuda(), cu.cuda(), **kw)


def _check(kda, q, kv, table, ctx, cu, scale=None, status=None, **kw):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    out = _run(kda, q, kv, table, ctx, cu, scale=scale, **kw)
    torch.cuda.synchronize()
    assert kda.last_device_status() == (kda.KDA_OK if status is None else status)
    ref, bound, mass = R.chunk_attention(q, kv[:, 0], kv[:, 1], table, ctx, cu, scale)
    if q.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
    got = out.cpu().double()
    n = int(cu[-1])
    assert torch.isfinite(got[:n]).all()
    off = ((got - ref).abs() - bound)[:n]
    assert (off <= 0).all(), f"{float(off.max()):.3e} over the bound at {tuple(np.unravel_index(int(off.argmax()), off.shape))}"
    return out


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("H,Hk", [(2, 2), (8, 1), (6, 2), (12, 1), (5, 1), (64, 1), (7, 7)])
def test_chunks_match_the_definition(cuda_lib, dtype, D, H, Hk):
    """Lengths around a tile's and a block's, empty chunks among them, with and without a context."""
    ctx, new = [0, 0, 5, 127, 128, 300, 1, 64], [1, 130, 0, 1, 33, 65, 129, 20]
    _check(cuda_lib, *_make(ctx, new, H, Hk, D, dtype, ps=16, seed=H))


@pytest.mark.parametrize("dtype,D", TYPES[:1] + TYPES[3:], ids=IDS[:1] + IDS[3:])
@pytest.mark.parametrize("ps", [1, 7, 8, 24, 64, 100, 128, 256, 1000])
def test_page_sizes(cuda_lib, dtype, D, ps):
    """Pages that end inside a tile, tiles that end inside a page; lengths around both."""
    ctx, new = [ps - 1, ps, 0, 127, 2, 0], [1, 3, 129, 2, ps, 255 + ps]
    _check(cuda_lib, *_make(ctx, new, 6, 2, D, dtype, ps=ps, seed=ps), fused=ps % 2 == 0)


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("ctx,new,H,Hk", [([9000], [2], 2, 1), ([5000, 3], [20, 700], 16, 2), ([3, 4000, 1, 2500], [64, 1, 0, 257], 3, 1),
                                          ([20000], [1], 1, 1), ([0], [1500], 4, 4), ([700], [900], 12, 1)])
def test_long_work_is_split(cuda_lib, dtype, D, ctx, new, H, Hk):
    x = _make(ctx, new, H, Hk, D, dtype, ps=64, seed=1)
    a = _check(cuda_lib, *x)
    b = _check(cuda_lib, *x)
    assert torch.equal(a, b), "two runs differ"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_many_sequences(cuda_lib, dtype):
    """More sequences than a warp has lanes and than the GPU has SMs; single tokens beside chunks."""
    r = np.random.default_rng(3)
    ctx, new = r.integers(0, 200, 333).tolist(), np.where(r.random(333) < 0.7, 1, r.integers(0, 90, 333)).tolist()
    _check(cuda_lib, *_make(ctx, new, 4, 2, 64, dtype, ps=16, seed=2))


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("ps", [16, 20], ids=["boxes", "gathered"])
def test_a_token_sees_nothing_behind_it(cuda_lib, dtype, D, ps):
    """NaN and infinities in one token's key or value: the rows before it keep their bits, the token's own and later
    ones show it."""
    ctx, new = [70, 0, 250], [150, 130, 9]
    q, kv, table, c, cu = _make(ctx, new, 3, 1, D, dtype, ps, seed=5)
    clean = _check(cuda_lib, q, kv, table, c, cu)
    for b, i in ((0, 1), (0, 60), (0, 149), (1, 1), (1, 129), (2, 4)):
        for part, what in ((0, float("nan")), (1, float("inf")), (1, float("nan"))):
            bad = kv.clone()
            pos = ctx[b] + i
            bad[int(table[b, pos // ps]), part, pos % ps, 0, 3] = what
            out = _run(cuda_lib, q, bad, table, c, cu)
            first = int(cu[b]) + i
            rest = torch.ones(q.shape[0], dtype=torch.bool)
            rest[first:int(cu[b + 1])] = False
            assert torch.equal(out.cpu()[rest], clean.cpu()[rest]), (b, i, part, what)
            hit = out.cpu()[first:int(cu[b + 1])]
            if part == 0:
                assert hit.isnan().all()
            else:
                assert not hit[..., 3].isfinite().any()
                other = [x for x in range(D) if x != 3]
                assert torch.equal(hit[..., other], clean.cpu()[first:int(cu[b + 1])][..., other])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 30.0])
def test_scales(cuda_lib, dtype, scale):
    """Uniform weights, negative ones, and scores of several thousand."""
    _check(cuda_lib, *_make([7, 300], [40, 4], 4, 2, 64, dtype, ps=32, seed=6), scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_lowest_scores(cuda_lib, dtype):
    """Every visible score near the lowest that fp32 holds: still the mean over what is visible."""
    q, kv, table, ctx, cu = _make([100], [3], 2, 1, 64, dtype, ps=16, seed=6)
    q = torch.zeros_like(q)
    q[..., 0] = -1e18
    kv[:, 0] = torch.where(kv[:, 0].isnan(), kv[:, 0], 0.0)
    kv[:, 0, :, :, 0] = torch.where(kv[:, 0, :, :, 0].isnan(), kv[:, 0, :, :, 0], 1e18)
    out = _run(cuda_lib, q, kv, table, ctx, cu).cpu().double()
    rows = lambda n: torch.stack([kv[int(table[0, t // 16]), 1, t % 16, 0].double() for t in range(n)])
    for i in range(3):
        v = rows(101 + i)
        # equal scores: every weight is one; n fp32 additions, and bf16's output rounding
        bound = (101 + i) * 2.0 ** -23 * v.abs().mean(0) + (2.0 ** -8 if dtype == torch.bfloat16 else 0) * v.mean(0).abs()
        assert ((out[i] - v.mean(0)).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_growing_scores(cuda_lib, dtype):
    """The maximum grows with every tile, by more than any fixed margin, and by less."""
    for step in (0.02, 0.5):
        q, kv, table, ctx, cu = _make([600], [200], 2, 1, 128, dtype, ps=16, seed=9)
        for t in range(800):
            kv[int(table[0, t // 16]), 0, t % 16] = step * t / 128 ** 0.5
        q = torch.ones_like(q)
        _check(cuda_lib, q, kv, table, ctx, cu)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_behind_the_last_chunk_stay(cuda_lib, dtype):
    q, kv, table, ctx, cu = _make([3, 40], [20, 0], 4, 2, 64, dtype, ps=16, seed=4, behind=7)
    out = torch.full_like(q, 5.0).cuda()
    got = _check(cuda_lib, q, kv, table, ctx, cu, out=out)
    assert got is out and (out[20:] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_bad_input_is_reported_and_the_rest_goes_on(cuda_lib, dtype):
    ctx, new = [40, 200, 30, 90], [70, 5, 130, 1]
    q, kv, table, c, cu = _make(ctx, new, 4, 2, 128, dtype, ps=16, seed=8)
    bad = cuda_lib.KDA_ERR_INVALID_ARG
    t = table.clone()
    t[1, 3], t[1, 5], t[2, 9] = -1, kv.shape[0], 0x7fffffff      # pages that are not there: left out
    _check(cuda_lib, q, kv, t, c, cu, status=bad)
    t[3, :6] = -1                                                 # and rows that have no other: zero
    out = _check(cuda_lib, q, kv, t, c, cu, status=bad)
    assert not out[205].any()
    ref, bound, mass = R.chunk_attention(q, kv[:, 0], kv[:, 1], table, c, cu, 128 ** -0.5)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
    for b, value in ((0, -1), (2, table.shape[1] * 16 - 129), (1, 0x7fffffff)):
        c2 = c.clone()
        c2[b] = value
        out = _run(cuda_lib, q, kv, table, c2, cu)
        assert cuda_lib.last_device_status() == bad
        mine = torch.zeros(206, dtype=torch.bool)
        mine[int(cu[b]):int(cu[b + 1])] = True
        assert not out.cpu()[mine].any()
        assert ((out.cpu().double() - ref).abs() <= bound)[~mine].all()
    for ends in ([1, 70, 75, 205, 206], [0, 70, 60, 205, 206], [0, 70, 75, 205, 207], [0, -1, 75, 205, 206], [0, 70, 75, 0x7fffffff, 206], [0, 0x7fffffff, -2, 205, 206],
                 [0, 70, -0x80000000, 205, 206]):
        out = torch.full_like(q, 5.0).cuda()
        _run(cuda_lib, q, kv, table, c, torch.tensor(ends, dtype=I32), out=out)
        assert cuda_lib.last_device_status() == bad and (out == 5.0).all(), ends


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_offsets_past_32_bits(cuda_lib, dtype):
    """A cache of more than 2^31 elements, the sequence's pages at its two ends."""
    ps, Hk, D, new, n = 64, 8, 128, 70, 130
    P = 2 ** 31 // (2 * ps * Hk * D) + 40
    kv = torch.empty((P, 2, ps, Hk, D), dtype=dtype, device="cuda")
    table = torch.tensor([[P - 1, 0, P - 2, P // 2 + 17]], dtype=I32)
    for p in table[0].tolist():
        kv[p].normal_()
    q = torch.randn(new, 16, D, device="cuda").to(dtype)
    ctx, cu = torch.tensor([n], dtype=I32), torch.tensor([0, new], dtype=I32)
    out = cuda_lib.chunk_attention(q, kv[:, 0], kv[:, 1], table.cuda(), ctx.cuda(), cu.cuda())
    small = kv[table[0].long().cuda()].cpu()
    ref, bound, mass = R.chunk_attention(q, small[:, 0], small[:, 1], torch.tensor([[0, 1, 2, 3]]), ctx, cu, D ** -0.5)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * mass + 2.0 ** -8 * ref.abs()
    assert ((out.cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_stream_graph_and_workspaces(cuda_lib, dtype):
    """Another stream; a captured and replayed call, with new lengths in the same buffers; a workspace used for one shape, then another."""
    x = _make([37, 500, 0], [100, 1, 260], 8, 2, 128, dtype, ps=16, seed=4)
    want = _check(cuda_lib, *x)
    q, kv, table, ctx, cu = (t.cuda() for t in x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = cuda_lib.chunk_attention(q, kv[:, 0], kv[:, 1], table, ctx, cu, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    desc = cuda_lib.make_chunk_attention_desc(3, q.shape[0], 8, 2, 128, cuda_lib.KDA_BF16 if dtype == torch.bfloat16 else cuda_lib.KDA_F32,
                                              kv.shape[0], 16, table.shape[1], 0.1, kv.stride(0), kv.stride(0))
    ws = torch.full((cuda_lib.chunk_attention_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    held = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        cuda_lib.chunk_attention(q, kv[:, 0], kv[:, 1], table, ctx, cu, out=held, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
    cu2 = torch.tensor([0, 90, 101, 361], dtype=I32)
    ctx2 = torch.tensor([30, 490, 0], dtype=I32)
    cu.copy_(cu2)
    ctx.copy_(ctx2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, _check(cuda_lib, x[0], x[1], x[2], ctx2, cu2, workspace=ws))
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_nothing_to_do(cuda_lib):
    q, kv, table, ctx, cu = _make([5], [2], 2, 1, 64, torch.bfloat16, ps=32, seed=4)
    z = lambda *s: torch.zeros(s, dtype=I32, device="cuda")
    dev = kv.cuda()
    assert cuda_lib.chunk_attention(q[:0].cuda(), dev[:, 0], dev[:, 1], table[:0].cuda(), z(0), z(1)).shape == (0, 2, 64)
    out = torch.full_like(q, 5.0).cuda()
    assert (cuda_lib.chunk_attention(q.cuda(), dev[:, 0], dev[:, 1], table.cuda(), ctx.cuda(), z(2), out=out) == 5.0).all()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    empty = dev[:0]                           # no pages at all: every token is left out
    assert not cuda_lib.chunk_attention(q.cuda(), empty[:, 0], empty[:, 1], table.cuda(), ctx.cuda(), cu.cuda()).any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("D", [64, 128])
def test_one_chunk_equals_its_chain_in_the_tree_attention(cuda_lib, D):
    """The same rows through kda_tree_attention as a chain of nodes: two kernels, one definition."""
    q, kv, table, ctx, cu = _make([100, 0], [40, 40], 8, 2, D, torch.float32, ps=16, seed=3)
    a = _check(cuda_lib, q, kv, table, ctx, cu).cpu().double()
    dev = kv.cuda()
    chain = torch.arange(-1, 39, dtype=I32, device="cuda").expand(2, 40).contiguous()
    b = cuda_lib.tree_attention(q.view(2, 40, 8, D).cuda(), dev[:, 0], dev[:, 1], table.cuda(), ctx.cuda(), chain).cpu().double()
    _, bound, _ = R.chunk_attention(q, kv[:, 0], kv[:, 1], table, ctx, cu, D ** -0.5)
    assert ((a - b.view(80, 8, D)).abs() <= 2 * bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_two_streams_at_once(cuda_lib, dtype):
    """Calls of different shapes on two streams, each with its own workspace; every result is that of the call alone."""
    xs = [[t.cuda() for t in _make([300, 0, 77], [200, 513, 1], 8, 2, 128, dtype, ps=16, seed=1)],
          [t.cuda() for t in _make([50, 900], [1, 1], 6, 2, 64, dtype, ps=20, seed=2)]]
    call = lambda x: cuda_lib.chunk_attention(x[0], x[1][:, 0], x[1][:, 1], *x[2:])
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, call(xs[k])))
    torch.cuda.synchronize()
    assert all(torch.equal(out, want[k]) for k, out in got)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_several_waves(cuda_lib):
    """Keys and values past what the ranges of one wave may share, read by several blocks: the line is cut in two waves (the
    workspace holds as many ranges), and units cross the ranges of both."""
    ctx, new, H, Hk, D, ps = 50000, 300, 16, 4, 128, 64
    x = _make([ctx], [new], H, Hk, D, torch.bfloat16, ps=ps, seed=5, poison=False)
    a = _check(cuda_lib, *x)
    assert torch.equal(a, _run(cuda_lib, *x, scale=D ** -0.5))
    desc = lambda pages: cuda_lib.make_chunk_attention_desc(1, new, H, Hk, D, cuda_lib.KDA_BF16, pages, ps, x[2].shape[1], 0.1, ps * Hk * D, ps * Hk * D)
    assert cuda_lib.chunk_attention_workspace_bytes(desc(x[1].shape[0])) == 2 * cuda_lib.chunk_attention_workspace_bytes(desc(100))
