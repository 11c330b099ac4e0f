"""The memories of ``draft_step.HybridLayers`` at the ends of what its calls allow: what they refuse leaves everything as it was."""
import pytest
import torch

import _prompt_ref as R
from linear_attention_serving_chunkwise_gb300 import draft_step

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def _kept(m):
    return [t.clone() for t in (m.pages_held, m.context_lens, m.shares, m.free_pages, m.block_table, m.state)]


def _same(m, before):
    return all(torch.equal(a, b) for a, b in zip(before, (m.pages_held, m.context_lens, m.shares, m.free_pages, m.block_table, m.state)))


def _after_a_draft_step():
    """Four sequences, the first of 20 tokens with three pages of 16 held, the others empty; every row's state is its own."""
    m = draft_step.HybridLayers(4, 2, 64, 1, 40, 16, 8)
    m.reserve(20)
    m.context_lens += 20
    m.reserve(28)                                   # a step's nodes: pages up to token 48
    m.release(_i32([48, 0, 0, 0]))
    assert m.context_lens.tolist() == [20, 0, 0, 0] and m.pages_held.tolist() == [3, 0, 0, 0]
    m.state.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    return m


@pytest.mark.parametrize("lens", [21, 32, 48, 49, 2 ** 31 - 1, -1])
def test_no_fork_of_more_than_the_parent_has(cuda_lib, lens):
    """Pages are held past the context: rows that nobody wrote, and a page that the parent still appends to."""
    m = _after_a_draft_step()
    before = _kept(m)
    with pytest.raises(RuntimeError):
        m.fork(_i32([0, 0]), _i32([1, 2]), _i32([20, lens]))
    assert _same(m, before) and cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("parents,children", [([0, 0], [1, 1]), ([0, 1], [1, 2]), ([0, 2], [2, 1]), ([3], [3])])
@pytest.mark.parametrize("lens", [0, 5])
def test_forks_that_contradict_each_other(cuda_lib, parents, children, lens):
    """A child named twice, a parent that is a child: refused whatever the lengths, the empty one among them."""
    m = _after_a_draft_step()
    before = _kept(m)
    with pytest.raises(ValueError):
        m.fork(_i32(parents), _i32(children), _i32([lens if p == 0 else 0 for p in parents]))
    assert _same(m, before) and cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_the_state_of_a_fork(cuda_lib):
    """All of the parent's tokens: its state.  Fewer: an empty one, into which they are replayed (they would count twice in the parent's)."""
    m = _after_a_draft_step()
    whole = m.state[0].clone()
    m.fork(_i32([0, 0, 0]), _i32([1, 2, 3]), _i32([20, 19, 0]))
    assert m.context_lens.tolist() == [20, 20, 19, 0] and m.pages_held.tolist() == [3, 2, 2, 0]
    assert torch.equal(m.state[0], whole) and torch.equal(m.state[1], whole) and not m.state[2].any() and not m.state[3].any()
    assert m.shares.sum() == 2 and cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 1 << 30])
def test_a_release_that_keeps_everything(cuda_lib, most):
    """Lengths up to the largest that int32 holds leave a row as it is, also where its first page is another's too."""
    m = _after_a_draft_step()
    m.fork(_i32([0]), _i32([1]), _i32([20]))
    before = _kept(m)
    m.release(_i32([most, most, most, 1 << 20]))
    assert _same(m, before)
    m.release(_i32([0, most, 0, 0]))
    assert m.context_lens.tolist() == [0, 20, 0, 0] and m.pages_held.tolist() == [0, 2, 0, 0] and not m.shares.any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("pages,cols", [(0, 4), (5, 0), (0, 0)])
def test_a_release_where_nothing_can_be_held(cuda_lib, pages, cols):
    """No pages, or no columns for them: there is no entry to look at."""
    m = draft_step.HybridLayers(3, 2, 64, 1, pages, 16, cols)
    m.release(_i32([0, 5, 2 ** 31 - 1]))
    assert m.pages_held.tolist() == [0, 0, 0] and m.free_pages.numel() == pages
    with pytest.raises(RuntimeError):
        m.release(_i32([0, -1, 0]))
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def _off(t):
    """The same values, one element past where they would be aligned."""
    return torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape).copy_(t)


# keys and values [B, K, heads, dim] as a model may have them
LAYOUTS = {"heads outside": lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), "channels outside": lambda t: t.transpose(2, 3).contiguous().transpose(2, 3),
           "unaligned": _off, "parts of odd rows": lambda t: torch.cat([t.flatten(2), t[..., 0, :1]], 2)[..., :-1].unflatten(2, t.shape[2:]),
           "one row for all": lambda t: t[:, :1].expand(t.shape), "tokens outside": lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,K", [(1, 5), (3, 4), (2, 1)])
def test_keys_and_values_of_any_layout(cuda_lib, layout, B, K):
    """Strides and alignments that norm_rotate does not take are the memory's to mend."""
    H, D, ps = 2, 64, 4
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda h: torch.randn(B, K, h, D, generator=gen, device="cuda").to(torch.bfloat16)
    m = draft_step.HybridLayers(B, 4, D, H, 20, ps, 6)
    q, k, v = rnd(4), LAYOUTS[layout](rnd(H)), LAYOUTS[layout](rnd(H))
    slots = m.reserve(K)
    chain = torch.arange(-1, K - 1, dtype=I32, device="cuda").expand(B, K).contiguous()
    out = m.attend(q, k, v, slots.to(torch.int32) if K == 4 else slots, chain)
    rows = m.cache[slots // ps, :, slots % ps]
    assert torch.equal(rows[:, :, 0], k) and torch.equal(rows[:, :, 1], v)
    s = torch.einsum("bihd,bjhd->bhij", q.double(), k.double().repeat_interleave(2, 2)) * D ** -0.5
    w = torch.softmax(s.masked_fill(torch.ones(K, K, device="cuda", dtype=torch.bool).triu(1), float("-inf")), -1)
    want = torch.einsum("bhij,bjhd->bihd", w, v.double().repeat_interleave(2, 2))
    mass = torch.einsum("bhij,bjhd->bihd", w, v.double().abs().repeat_interleave(2, 2))
    # bf16: the weights' rounding and that of the output, half a step each, and fp32's share
    assert ((out.double() - want).abs() <= 2.0 ** -8 * (mass + want.abs()) + 2.0 ** -16 * mass).all()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("heads,kv_heads,dim", [(96, 1, 64), (130, 2, 64), (128, 1, 128)])
def test_prompts_of_more_heads_to_a_cache_head_than_one_call_takes(cuda_lib, heads, kv_heads, dim):
    """The tree attention has no such limit, and the model's prompts went through it before."""
    gen = torch.Generator(device="cuda").manual_seed(heads)
    rnd = lambda h: torch.randn(90, h, dim, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = rnd(heads), rnd(kv_heads), rnd(kv_heads)
    new, ends = [41, 0, 49], _i32([0, 41, 41, 90])
    m = draft_step.HybridLayers(3, heads, 64, kv_heads, 30, 16, 8)
    m.cache = torch.empty((30, 2, 16, kv_heads, dim), dtype=torch.bfloat16, device="cuda")
    slots, _, m.pages_held, _ = cuda_lib.page_tables(m.context_lens, _i32(new), m.pages_held, m.block_table, m.free_pages, page_size=16, max_tokens=90)
    got = m.attend_chunks(q, k, v, slots, ends)
    ref, bound, mass = R.chunk_attention(q, m.cache[:, 0], m.cache[:, 1], m.block_table.cpu(), m.context_lens.cpu(), ends.cpu(), dim ** -0.5)
    # bf16: the weights' rounding and that of the output, half a step each
    assert ((got.cpu().double() - ref).abs() <= bound + 2.0 ** -8 * (mass + ref.abs())).all()
    m = draft_step.ToyHybrid(2, heads=heads, dim=64, kv_heads=kv_heads, most_tokens=96)
    assert torch.isfinite(m.prompt(torch.randint(0, 211, (2, 70), generator=gen, device="cuda", dtype=I32))).all()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
