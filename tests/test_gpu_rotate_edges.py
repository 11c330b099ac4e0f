"""kda_norm_rotate's angles at the ends of what frequencies and positions may be."""
import math

import numpy as np
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


def _per_turn(bits):
    """floor(2^bits / 2 pi), from pi = 16 atan(1/5) - 4 atan(1/239) in integers."""
    one = 1 << (2 * bits + 32)

    def atan(inverse):
        term, total, n = one // inverse, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= inverse * inverse
            n += 2
        return total

    return (one << bits) // (2 * (16 * atan(5) - 4 * atan(239)))


def _turns(pos, freq, bits=400):
    """Fractions of a turn [T, pairs] of pos * freq, exact to 1e-15."""
    per = _per_turn(bits)
    out = np.zeros((len(pos), len(freq)))
    for j, f in enumerate(freq.tolist()):
        m, e = math.frexp(f)
        m, e = int(m * 2 ** 24), e - 24                        # f = m 2^e, an fp32 number
        one = m * per << e if e >= 0 else m * per >> -e        # a token's turns, times 2^bits
        for i, p in enumerate(pos.tolist()):
            out[i, j] = (p * one % (1 << bits) >> (bits - 60)) / 2.0 ** 60
    return out


@pytest.mark.parametrize("low,high", [(1e-6, 1.0), (1.0, 1e3), (1e3, 1e8), (1e8, 2.0 ** 40)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
def test_angles_of_any_position_and_frequency(cuda_lib, low, high, interleaved):
    """Rows of pairs (1, 0) become the cosines and sines.  Bound: two ulp of the functions at 1, a rounding of the sum with what 24 bits of
    the angle leave, and the angle's 1e-9 of a turn: 2^-23 + 2^-24 + 2^-27 < 2^-22."""
    gen = torch.Generator().manual_seed(int(high))
    T, D = 48, 128
    pos = torch.cat([torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24, 16777215, 1000003]), torch.randint(-2 ** 31, 2 ** 31, (20,), generator=gen),
                     torch.randint(0, 1 << 24, (20,), generator=gen)]).to(I32)
    freq = torch.exp(torch.rand(D // 2, generator=gen, dtype=torch.float64) * math.log(high / low) + math.log(low)).float()
    freq[:3] = torch.tensor([low, high, -(low * high) ** 0.5])
    x = torch.zeros(T, 1, D)
    a, b = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    x[..., a] = 1
    got = _rotate(cuda_lib, x.cuda(), pos, freq, interleaved).cpu().double().numpy()[:, 0]
    turns = 2 * np.pi * _turns(pos, freq)
    assert np.abs(got[:, a] - np.cos(turns)).max() <= 2.0 ** -22 and np.abs(got[:, b] - np.sin(turns)).max() <= 2.0 ** -22
