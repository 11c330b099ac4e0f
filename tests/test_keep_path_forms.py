"""``draft_step.keep_path`` on every cache that it is given: the kernel's, and those that the kernel does not take."""
import numpy as np
import pytest
import torch

import _prompt_ref as R
from linear_attention_serving_chunkwise_gb300 import draft_step


def _step(B, K, ps, seed):
    """Slots [B, K], ascending paths of random lengths, pages in all."""
    r = np.random.default_rng(seed)
    pages = -(-(ps - 1 + K) // ps)
    ids = r.permutation(B * pages + 2)
    first = r.integers(0, ps, B)
    pos = first[:, None] + np.arange(K)
    slots = ids[np.arange(B)[:, None] * pages + pos // ps] * ps + pos % ps
    path, n = np.full((B, K), -1, np.int64), r.integers(0, K + 1, B)
    n[0] = K
    for b in range(B):
        path[b, :n[b]] = np.sort(r.choice(K, n[b], replace=False))
    return slots, path, n, B * pages + 2


def _check(device, dtype, K=9, ps=7, H=2, D=64, ints=torch.int32, lay=lambda c: c, B=5):
    slots, path, n, P = _step(B, K, ps, K + H + D)
    cache = torch.randint(-100, 100, (P, 2, ps, H, D), generator=torch.Generator().manual_seed(1)).to(dtype)
    want = R.keep_path(slots, path, n, cache[None])[0]
    got = lay(cache.to(device))
    draft_step.keep_path(got, torch.as_tensor(slots, device=device), torch.as_tensor(path, device=device).to(ints),
                         torch.as_tensor(n, device=device).to(ints))
    assert torch.equal(got.cpu(), want)


def _apart(c):
    """The same values, heads in every other place."""
    wide = torch.zeros(*c.shape[:3], 2 * c.shape[3], c.shape[4], dtype=c.dtype, device=c.device)
    wide[:, :, :, ::2] = c
    return wide[:, :, :, ::2]


def _off_by_one(c):
    """The same values, one element past where they would be aligned."""
    flat = torch.zeros(c.numel() + 1, dtype=c.dtype, device=c.device)
    return flat[1:].view(c.shape).copy_(c)


FORMS = [dict(dtype=torch.bfloat16), dict(dtype=torch.float32), dict(dtype=torch.float16), dict(dtype=torch.int8), dict(dtype=torch.float64),
         dict(dtype=torch.bfloat16, H=1, D=12), dict(dtype=torch.float32, H=3, D=5), dict(dtype=torch.bfloat16, K=70), dict(dtype=torch.bfloat16, K=64),
         dict(dtype=torch.bfloat16, ints=torch.int64), dict(dtype=torch.float32, lay=_apart), dict(dtype=torch.bfloat16, lay=_off_by_one),
         dict(dtype=torch.bfloat16, lay=lambda c: c.transpose(1, 2).contiguous().transpose(1, 2))]


@pytest.mark.parametrize("form", FORMS, ids=range(len(FORMS)))
def test_on_the_cpu(form):
    _check("cpu", **form)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS, ids=range(len(FORMS)))
def test_on_the_gpu(cuda_lib, form):
    _check("cuda", **form)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
