"""GPU parity of kda_norm_rotate against the definition in 64 bits.  Bounds: _prompt_ref.norm_rotate's for the fp32 arithmetic
(its own roundings counted one by one), and half a step of the type for the one rounding at the end: 2^-8 |y| for bf16, 2^-24 |y|
for fp32."""
import pytest
import torch

import _prompt_ref as R

pytestmark = pytest.mark.gpu
I32, I64 = torch.int32, torch.int64


def _freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


def _make(T, H, Hk, D, dtype, ps, seed=0, far=5000, fused=True, skip=()):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * Hk, D, generator=g) * torch.exp(torch.randn(T, 1, 1, generator=g))).to(dtype).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    if not fused:
        q, k, v = (x.contiguous() for x in (q, k, v))
    P = -(-T // ps) + 2
    slots = torch.randperm(P * ps, generator=g)[:T]
    for t in skip:
        slots[t] = -1
    pos = torch.randint(0, far, (T,), generator=g).to(I32)
    cache = torch.full((P, 2, ps, Hk, D), 7.0, dtype=dtype, device="cuda")
    return q, k, v, pos, slots, cache


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _check(kda, x, freq, wq=None, wk=None, eps=1e-6, norm=True, interleaved=False, status=None, **kw):
    q, k, v, pos, slots, cache = x
    before = cache.clone()
    out = kda.norm_rotate(q, k, v, pos.cuda(), freq.cuda(), slots.cuda(), cache[:, 0], cache[:, 1], eps=eps, norm=norm, interleaved=interleaved,
                          q_weight=None if wq is None else wq.cuda(), k_weight=None if wk is None else wk.cuda(), **kw)
    torch.cuda.synchronize()
    assert kda.last_device_status() == (kda.KDA_OK if status is None else status)
    for got, src, w in ((out, q, wq), (None, k, wk)):
        ref, bound = R.norm_rotate(src, pos, freq, w, eps, norm, interleaved)
        if got is None:
            P, _, ps, Hk, D = cache.shape
            on = (slots >= 0) & (slots < P * ps)
            s = slots[on]
            flat = cache.cpu()
            got, ref, bound = flat[s // ps, 0, s % ps], ref[on], bound[on]
            assert torch.equal(flat[s // ps, 1, s % ps], v.cpu()[on])
            rest = torch.ones(P, ps, dtype=torch.bool)
            rest[s // ps, s % ps] = False
            assert torch.equal(flat.transpose(1, 2)[rest], before.cpu().transpose(1, 2)[rest]), "a row that no slot names was written"
        off = (got.cpu().double() - ref).abs() - (bound * (1 + _half(q.dtype)) + _half(q.dtype) * ref.abs() + 1e-40)
        assert (off <= 0).all(), float(off.max())
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 32), (128, 112), (128, 16), (128, 0), (64, 64), (64, 32), (64, 16), (64, 48), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
def test_norms_and_rotations(cuda_lib, dtype, D, rot, interleaved):
    g = torch.Generator().manual_seed(rot)
    wq, wk = torch.randn(D, generator=g), torch.randn(D, generator=g)
    _check(cuda_lib, _make(37, 6, 2, D, dtype, 16, skip=(3, 36)), _freq(rot), wq, wk, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,H,Hk,ps,fused", [(1, 1, 1, 1, True), (1, 96, 8, 64, True), (2, 5, 5, 7, False), (63, 7, 1, 24, True), (300, 12, 3, 100, False),
                                             (1216, 3, 1, 16, True), (2500, 16, 2, 128, True)])
def test_sizes(cuda_lib, dtype, T, H, Hk, ps, fused):
    """One token to more than the GPU takes at once, a token to a CTA and eight; rows that fill no warp; parts of one projection and not."""
    _check(cuda_lib, _make(T, H, Hk, 128, dtype, ps, seed=T, fused=fused), _freq(128), torch.ones(128) * 1.5, None)


@pytest.mark.parametrize("norm,weight,eps", [(True, False, 1e-6), (True, True, 0.0), (True, True, 0.5), (False, True, 1e-6)])
def test_norm_options(cuda_lib, norm, weight, eps):
    w = torch.linspace(-2, 2, 64) if weight else None
    _check(cuda_lib, _make(20, 4, 2, 64, torch.float32, 16), _freq(64), w, w, eps=eps, norm=norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_far_positions(cuda_lib, dtype):
    """Angles of many whole turns, negative positions and frequencies, frequencies above a turn; past 2^24 the reference's own
    64-bit product is what limits."""
    x = list(_make(64, 4, 1, 128, dtype, 16, seed=2))
    x[3] = torch.cat([torch.tensor([0, 1, -1, -777, 131071, 1000003, 16777215, -16777215]), torch.randint(1 << 20, 1 << 24, (56,))]).to(I32)
    freq = _freq(128, 500000.0)
    freq[:6] = torch.tensor([1.0, 3.14159274, 6.2831855, 100.7, -0.3, 0.0])
    _check(cuda_lib, tuple(x), freq)


def test_rows_of_zeros_and_what_is_not_finite(cuda_lib):
    """Zeros stay zeros with any eps > 0; a NaN or infinity stays in its row."""
    q, k, v, pos, slots, cache = _make(9, 4, 2, 64, torch.float32, 16, fused=False)
    clean = cuda_lib.norm_rotate(q, k, v, pos.cuda(), _freq(64).cuda(), slots.cuda(), cache[:, 0], cache[:, 1])
    q[2, 1] = 0
    q[3, 0, 5] = float("nan")
    q[4, 3, 60] = float("inf")
    out = cuda_lib.norm_rotate(q, k, v, pos.cuda(), _freq(64).cuda(), slots.cuda(), cache[:, 0], cache[:, 1])
    assert not out[2, 1].any() and out[3, 0].isnan().all() and out[4, 3].isnan().any()
    same = torch.ones(9, 4, dtype=torch.bool)
    same[2, 1] = same[3, 0] = same[4, 3] = False
    assert torch.equal(out.cpu()[same], clean.cpu()[same])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_slots_out_of_range_are_reported(cuda_lib):
    x = list(_make(20, 4, 2, 64, torch.bfloat16, 16, skip=(0, 7)))
    x[4][5] = x[5].shape[0] * 16
    x[4][9] = 2 ** 62
    x[4][11] = -2 ** 62                                     # nowhere, and no error
    _check(cuda_lib, tuple(x), _freq(64), status=cuda_lib.KDA_ERR_INVALID_ARG)


def test_other_stream_graph_and_given_out(cuda_lib):
    q, k, v, pos, slots, cache = _make(50, 8, 2, 128, torch.bfloat16, 16, seed=8)
    args = (pos.cuda(), _freq(128).cuda(), slots.cuda())
    want = cuda_lib.norm_rotate(q, k, v, *args, cache[:, 0], cache[:, 1])
    rows = cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.norm_rotate(q, k, v, *args, cache[:, 0], cache[:, 1], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, cache2 = torch.empty_like(want), torch.full_like(cache, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.norm_rotate(q, k, v, *args, cache2[:, 0], cache2[:, 1], out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache2, rows)
    assert cuda_lib.norm_rotate(q[:0], k[:0], v[:0], args[0][:0], args[1], args[2][:0], cache[:, 0], cache[:, 1]).shape == (0, 8, 128)


def test_caches_past_32_bits(cuda_lib):
    ps, Hk, D = 64, 8, 128
    P = 2 ** 31 // (2 * ps * Hk * D) + 40
    kv = torch.empty((P, 2, ps, Hk, D), dtype=torch.bfloat16, device="cuda")
    q, k, v, pos, _, _ = _make(3, 8, Hk, D, torch.bfloat16, 16)
    slots = torch.tensor([P * ps - 1, 5, (P // 2 + 9) * ps + 3])
    cuda_lib.norm_rotate(q, k, v, pos.cuda(), _freq(128).cuda(), slots.cuda(), kv[:, 0], kv[:, 1])
    ref, bound = R.norm_rotate(k, pos, _freq(128), None, 1e-6)
    got = kv[(slots // ps).cuda(), 0, (slots % ps).cuda()].cpu().double()
    assert ((got - ref).abs() <= bound * 1.01 + 2.0 ** -8 * ref.abs()).all()
    assert torch.equal(kv[(slots // ps).cuda(), 1, (slots % ps).cuda()], v)
