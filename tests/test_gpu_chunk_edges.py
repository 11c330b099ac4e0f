"""kda_chunk_attention at the ends of what it takes, against the definition in 64 bits (bounds: _prompt_ref.chunk_attention's, and in bf16
half a step for the weights and half a step for the output)."""
import pytest
import torch

import _prompt_ref as R

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)]
IDS = ["bf16-128", "bf16-64", "fp32-128", "fp32-64"]
I32 = torch.int32


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_one_page_of_any_stride_on_another_stream(cuda_lib, dtype, D):
    """A cache of one page has no distance between pages: what its first stride says is not looked at, on whatever stream."""
    ps, Hk, n = 48, 2, 40
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    q, k, v = rnd(n, 6, D), rnd(ps, 1, Hk, D).transpose(0, 1), rnd(ps, 1, Hk, D).transpose(0, 1)
    assert k.shape == (1, ps, Hk, D) and k.stride(0) < ps * Hk * D
    args = (q, k, v, _i32([[0]]), _i32([0]), _i32([0, n]))
    want = cuda_lib.chunk_attention(*args)
    ref, bound, mass = R.chunk_attention(q, k, v, torch.zeros(1, 1, dtype=I32), [0], [0, n], D ** -0.5)
    more = 2.0 ** -8 * (mass + ref.abs()) if dtype == torch.bfloat16 else 0.0
    assert ((want.cpu().double() - ref).abs() <= bound + more).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.chunk_attention(*args, stream=side)
    out = cuda_lib.chunk_attention(*args, out=torch.empty_like(q), stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want) and cuda_lib.last_device_status() == cuda_lib.KDA_OK


def _paged(kda, k, v, lens, new, ps):
    """Rows of keys and values per sequence (lists of [n, Hk, D]) in a cache whose other rows are NaN: what the call takes behind q."""
    Hk, D = k[0].shape[1:]
    kv, table = R.paged(lens, Hk, D, k[0].dtype, ps)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        where = table[b].long()[t // ps], t % ps
        kv[where[0], 0, where[1]], kv[where[0], 1, where[1]] = k[b], v[b]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    dev = kv.cuda()
    return kv, table, [n - m for n, m in zip(lens, new)], cu, (dev[:, 0], dev[:, 1], table.cuda(), _i32([n - m for n, m in zip(lens, new)]), _i32(cu))


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("H,Hk,ctx,new", [(2, 1, [0, 0, 5], [1, 140, 9]), (16, 2, [300, 129], [20, 1]), (2, 1, [9000, 128], [2, 3]), (3, 1, [6000], [130])])
def test_scores_of_minus_infinity(cuda_lib, dtype, D, H, Hk, ctx, new):
    """Rows all of whose visible scores are -inf are NaN; a single finite score among them is all that counts, wherever it lies."""
    gen = torch.Generator().manual_seed(7)
    lens = [c + n for c, n in zip(ctx, new)]
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)
    q = rnd(sum(new), H, D)
    q[..., 5] = q[..., 5].abs() + 0.5
    k, v = [rnd(n, Hk, D) for n in lens], [rnd(n, Hk, D) for n in lens]
    for x in k:
        x[..., 5] = -float("inf")
    _, _, _, _, args = _paged(cuda_lib, k, v, lens, new, 16)
    out = cuda_lib.chunk_attention(q.cuda(), *args)
    assert out.isnan().all()
    for at in (lambda n, m: 0, lambda n, m: n - m, lambda n, m: n // 2, lambda n, m: n - 1):
        k2 = [x.clone() for x in k]
        for x, n, m in zip(k2, lens, new):
            x[at(n, m), :, 5] = 0.25
        _, _, _, cu, args = _paged(cuda_lib, k2, v, lens, new, 16)
        out = cuda_lib.chunk_attention(q.cuda(), *args).cpu()
        for b, (n, m) in enumerate(zip(lens, new)):
            got, first = out[cu[b]:cu[b + 1]], at(n, m) - (n - m)
            assert got[:max(first, 0)].isnan().all()
            want = v[b][at(n, m)].repeat_interleave(H // Hk, 0).expand(m, H, D)[max(first, 0):]
            # one weight, of 1 or (a maximum kept) up to 2^15: its rounding to bf16 and the quotient's
            assert ((got[max(first, 0):].double() - want.double()).abs() <= (2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -22) * want.double().abs()).all()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
def test_rows_without_a_page_stay_zero_beside_them(cuda_lib, dtype, D):
    """No page that exists: zeros and the error word, also where the part of a split row that has one holds -inf."""
    gen = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)
    lens, new = [7000, 200], [2, 3]
    q, k, v = rnd(5, 2, D).abs() + 0.5, [rnd(n, 1, D) for n in lens], [rnd(n, 1, D) for n in lens]
    k[0][...] = -float("inf")
    _, _, _, _, (kc, vc, table, c, cu) = _paged(cuda_lib, k, v, lens, new, 16)
    table[1] = -1
    out = cuda_lib.chunk_attention(q.to(dtype).cuda(), kc, vc, table, c, cu)
    assert out[:2].isnan().all() and not out[2:].any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    table[0, 1:] = -1                                          # sixteen tokens of -inf are left, the other parts have none
    out = cuda_lib.chunk_attention(q.to(dtype).cuda(), kc, vc, table, c, cu)
    assert out[:2].isnan().all() and not out[2:].any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("H,Hk,ctx,new", [(2, 1, [700] * 200, [1] * 200), (4, 1, [900, 0, 2000], [70, 650, 1]), (1, 1, [40000], [1])])
def test_large_values_under_scores_that_grow_a_little(cuda_lib, dtype, D, H, Hk, ctx, new):
    """Values of the largest size that is promised to stay finite; scores that grow behind the first tile by just less than what renews the
    maximum, so that the weights are as large as they get (bf16: 128 of e^5.5, of 2^15 in all; fp32: 2 or 4 a thread of e^9)."""
    gen = torch.Generator().manual_seed(6)
    lens = [c + n for c, n in zip(ctx, new)]
    q = torch.zeros(sum(new), H, D)
    q[..., 3] = 1
    k = [torch.zeros(n, Hk, D) for n in lens]
    for x in k:
        x[128:, :, 3] = 5.5 if dtype == torch.bfloat16 else 9.0
    v = [(torch.rand(n, Hk, D, generator=gen) + 0.5) * torch.where(torch.rand(D, generator=gen) < 0.5, -1.0, 1.0) * 2.0 ** 81 for n in lens]
    q, k, v = q.to(dtype), [x.to(dtype) for x in k], [x.to(dtype) for x in v]
    kv, table, c, cu, args = _paged(cuda_lib, k, v, lens, new, 16)
    assert max(float(x.abs().max()) for x in v) <= 2.0 ** 82
    out = cuda_lib.chunk_attention(q.cuda(), *args, scale=1.0).cpu().double()
    ref, bound, mass = R.chunk_attention(q, kv[:, 0], kv[:, 1], table, c, cu, 1.0)
    more = 2.0 ** -8 * (mass + ref.abs()) if dtype == torch.bfloat16 else 0.0
    assert ((out - ref).abs() <= bound + more).all() and cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("dtype,D", TYPES, ids=IDS)
@pytest.mark.parametrize("ps", [16, 20], ids=["boxes", "gathered"])
def test_what_a_row_sees_shows_under_a_weight_of_nothing(cuda_lib, dtype, D, ps):
    """An infinite or NaN value whose weight vanishes in fp32 (a score 300 below the others) is seen all the same: the rows from its token on are
    not finite in its channel; all other rows and channels keep their bits."""
    ctx, new = [70, 0, 250], [150, 130, 9]
    lens, gen = [c + n for c, n in zip(ctx, new)], torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)
    q, k, v = rnd(sum(new), 3, D), [rnd(n, 1, D) for n in lens], [rnd(n, 1, D) for n in lens]
    q[..., 3] = 1
    for b, i in ((0, 1), (0, 60), (0, 149), (0, -40), (1, 1), (1, 129), (2, 4), (2, -250)):
        at = ctx[b] + i
        k2, v2 = [x.clone() for x in k], [x.clone() for x in v]
        k2[b][at, :, 3] = -300 * D ** 0.5
        _, _, _, cu, args = _paged(cuda_lib, k2, v2, lens, new, ps)
        clean = cuda_lib.chunk_attention(q.cuda(), *args)
        for what in (float("inf"), float("nan")):
            v2[b][at, 0, 5] = what
            _, _, _, cu, args = _paged(cuda_lib, k2, v2, lens, new, ps)
            out = cuda_lib.chunk_attention(q.cuda(), *args)
            hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
            hit[cu[b] + max(i, 0):cu[b + 1], :, 5] = True
            assert not out[hit].isfinite().any() and torch.equal(out[~hit], clean[~hit]), (b, i, what)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
