"""kda_norm_rotate's angles at the ends of what frequencies and positions may be."""
import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _rotate(kda, x, pos, freq, interleaved=False):
    """x [T, H, D] rotated only: as queries, and as keys through the cache."""
    T, H, D = x.shape
    cache = torch.zeros(T, 2, 1, H, D, dtype=x.dtype, device="cuda")
    slots = torch.arange(T, device="cuda")
    q = kda.norm_rotate(x, x, x, pos.cuda(), freq.cuda(), slots, cache[:, 0], cache[:, 1], norm=False, interleaved=interleaved)
    assert torch.equal(q.nan_to_num(7e7), cache[:, 0, 0].nan_to_num(7e7)) and torch.equal(cache[:, 1, 0], x)
    assert kda.last_device_status() == kda.KDA_OK
    return q


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dtype,D,rot", [(torch.bfloat16, 128, 128), (torch.float32, 64, 32)])
@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
def test_frequencies_that_are_not_finite(cuda_lib, dtype, D, rot, interleaved, what):
    """Their pairs are NaN at every position (the sine of infinity, and of 0 times infinity, is NaN); all others keep their bits."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(12, 3, D, generator=gen, device="cuda").to(dtype)
    pos = torch.arange(12, dtype=I32) * 1001
    freq = 10000.0 ** (-torch.arange(0, rot, 2) / rot)
    clean = _rotate(cuda_lib, x, pos, freq, interleaved)
    assert torch.isfinite(clean).all()
    bad = freq.clone()
    hit = [0, 5, rot // 2 - 1]
    bad[hit] = what
    got = _rotate(cuda_lib, x, pos, bad, interleaved)
    channels = torch.zeros(D, dtype=torch.bool)
    for c in hit:
        channels[[2 * c, 2 * c + 1] if interleaved else [c, c + rot // 2]] = True
    assert got[..., channels].isnan().all() and torch.equal(got[..., ~channels], clean[..., ~channels])
