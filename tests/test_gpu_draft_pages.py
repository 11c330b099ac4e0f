"""Pages at their limits: requests that do not fit beside requests that do, and lengths at the ends of 32 bits."""
import numpy as np
import pytest
import torch

from linear_attention_serving_chunkwise_gb300 import draft_step

pytestmark = pytest.mark.gpu


def _layers(num_pages, page_size, cols, context=(0, 0), held=(0, 0)):
    mem = draft_step.HybridLayers(2, 2, 64, 1, num_pages, page_size, cols)
    mem.context_lens[:] = torch.tensor(context)
    taken = 0
    for b, n in enumerate(held):
        mem.block_table[b, :n] = mem.free_pages[taken:taken + n]
        taken += n
    mem.pages_held[:] = torch.tensor(held)
    mem.free_pages = mem.free_pages[taken:]
    return mem


def test_reserve_refuses_when_pages_reach_for_one_sequence_only(cuda_lib):
    mem = _layers(num_pages=3, page_size=4, cols=4)
    with pytest.raises(RuntimeError):
        mem.reserve(8)                                    # two pages each, three there
    # what the first sequence took is its own; the second has nothing
    assert mem.pages_held.tolist() == [2, 0] and mem.free_pages.tolist() == [2]
    assert mem.block_table.tolist() == [[0, 1, -1, -1], [-1] * 4]
    assert mem.reserve(4).tolist() == [[0, 1, 2, 3], [8, 9, 10, 11]]
    assert mem.free_pages.numel() == 0 and cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_reserve_refuses_when_one_table_row_is_full(cuda_lib):
    mem = _layers(num_pages=9, page_size=4, cols=2, context=(0, 6), held=(0, 2))
    with pytest.raises(RuntimeError):
        mem.reserve(4)
    assert mem.pages_held.tolist() == [1, 2] and mem.free_pages.tolist() == [3, 4, 5, 6, 7, 8]
    assert mem.block_table.tolist() == [[2, -1], [0, 1]]


def test_reserve_refuses_when_no_page_is_left(cuda_lib):
    mem = _layers(num_pages=1, page_size=4, cols=4)
    with pytest.raises(RuntimeError):
        mem.reserve(5)
    assert mem.pages_held.tolist() == [0, 0] and mem.free_pages.tolist() == [0]


def _tables(kda, ctx, new, held, table, free, ps, max_tokens):
    c = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    t = c(table)
    slots, cu, out, taken = kda.page_tables(c(ctx), c(new), c(held), t, c(free), page_size=ps, max_tokens=max_tokens)
    return slots.tolist(), out.tolist(), int(taken), t.tolist()


def test_tables_after_a_request_of_two_billion_tokens(cuda_lib):
    """It exceeds its row and is refused; the pages of those behind it are written all the same."""
    slots, held, taken, table = _tables(cuda_lib, [0, 3, 0], [2 ** 31 - 1, 5, 9], [0, 1, 0], [[-1] * 3, [7, -1, -1], [-1] * 3], [40, 41, 42, 43], 4, 6)
    assert held == [0, 2, 3] and taken == 4
    assert table == [[-1] * 3, [7, 40, -1], [41, 42, 43]]
    assert slots == [-1] * 6 and cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG


def test_tables_of_positions_past_31_bits(cuda_lib):
    """A context of 2^31 - 10 tokens and 20 more: the last held page, and a new one."""
    ps, ctx, new = 4096, 2 ** 31 - 10, 20
    held = -(-ctx // ps)
    table = torch.full((1, held + 1), -1, dtype=torch.int32, device="cuda")
    table[0, held - 1] = 77
    c = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    slots, cu, out, taken = cuda_lib.page_tables(c(ctx), c(new), c(held), table, c(123), page_size=ps, max_tokens=new)
    assert slots.tolist() == [77 * ps + ps - 10 + t for t in range(10)] + [123 * ps + t for t in range(10)]
    assert out.tolist() == [held + 1] and int(taken) == 1 and int(table[0, held]) == 123
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("ps", [4096, 4100], ids=["boxes", "gathered"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_attention_of_lengths_at_the_end_of_31_bits(cuda_lib, dtype, ps):
    """Table rows that could hold more than 2^31 tokens (all of them on one page): a sequence that has so many is
    refused, the one beside it is not."""
    K, D = 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, K, 1, D, generator=g, device="cuda").to(dtype)
    kv = torch.randn(1, 2, ps, 1, D, generator=g, device="cuda").to(dtype)
    table = torch.zeros((2, 2 ** 31 // ps + 2), dtype=torch.int32, device="cuda")
    parents = torch.arange(-1, K - 1, dtype=torch.int32, device="cuda").expand(2, K).contiguous()
    lens = lambda a, b: torch.tensor([a, b], dtype=torch.int32, device="cuda")
    small = cuda_lib.tree_attention(q, kv[:, 0], kv[:, 1], table[:, :1].contiguous(), lens(100, 100), parents)
    for long in (2 ** 31 - 1, 2 ** 31 - K, 2 ** 31 - 100, 2 ** 31 - 8191 - K):
        out = cuda_lib.tree_attention(q, kv[:, 0], kv[:, 1], table, lens(100, long), parents)
        assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
        assert not out[1].any() and torch.equal(out[0], small[0])
