"""The draft step end to end: a toy hybrid model (one KDA layer, one attention layer) decoded
in trees of drafts equals the same tokens decoded one by one."""
import pytest
import torch

from linear_attention_serving_chunkwise_gb300 import draft_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed,prompt", [(0, 70), (1, 3), (2, 129)])
def test_draft_steps_equal_token_by_token(cuda_lib, seed, prompt):
    """The same tokens reach both memories; the bf16 rows between the layers round alike or one step
    apart, which the states (a sum of a hundred writes of size 1) and the probabilities show in the
    third digit at most."""
    r = draft_step.demo(seed=seed, prompt=prompt)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    assert r["kept_drafts"] > 0 and r["tokens"] == r["steps"] + r["kept_drafts"] + 3
    assert r["state"] < 3e-2 and r["probs"] < 3e-2


def test_kept_rows_move_to_the_front(cuda_lib):
    cache = torch.arange(4 * 2 * 4 * 1 * 64, device="cuda", dtype=torch.float32).view(4, 2, 4, 1, 64)
    slots = torch.tensor([[9, 10, 11, 0, 1], [12, 13, 14, 15, 4]], device="cuda")
    path = torch.tensor([[0, 2, 4, -1, -1], [0, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    before = cache.clone()
    draft_step.keep_path(cache, slots, path, n)
    row = lambda c, s: c[s // 4, :, s % 4]
    for dst, src in ((9, 9), (10, 11), (11, 1), (12, 12)):
        assert torch.equal(row(cache, dst), row(before, src))
    for s in (0, 1, 13, 14, 15, 4, 2, 3, 8):
        assert torch.equal(row(cache, s), row(before, s))
