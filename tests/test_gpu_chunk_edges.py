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
