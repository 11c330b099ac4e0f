"""GPU tests of kda_verify_drafts and kda_page_tables: whole numbers, equal to the references
(every step of the verification is one IEEE fp32 operation per element, in the same order)."""
import numpy as np
import pytest
import torch

import _draft_ref as R

pytestmark = pytest.mark.gpu


def _case(B, K, V, kind, seed, draft, sharp=3.0):
    r = np.random.default_rng(seed)
    soft = lambda z: (np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)
    z = r.standard_normal((B, K + 1, V)) * sharp
    parents = R.trees(kind, B, K, seed)
    target = soft(z)
    q = None
    if draft:
        q = soft(z[:, :K] + 0.7 * r.standard_normal((B, K, V)))
        tokens = np.array([[r.choice(V, p=q[b, i].astype(np.float64) / q[b, i].astype(np.float64).sum()) for i in range(K)] for b in range(B)])
    else:
        rows = np.take_along_axis(target, np.maximum(parents + 1, 0)[..., None].astype(np.int64), 1)
        top = np.argsort(-rows, -1)
        tokens = np.take_along_axis(top, r.integers(0, min(3, V), (B, K, 1)), -1)[..., 0]   # siblings may repeat a token
    u = r.random((B, K), dtype=np.float32)
    noise = r.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)
    return target, q, tokens.astype(np.int32), parents, u, noise


def _run(kda, target, q, tokens, parents, u, noise, **kw):
    c = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    got = kda.verify_drafts(c(target), c(tokens), c(parents), c(u), c(noise), draft_probs=c(q), **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got]


def _same(got, want):
    for name, g, w in zip(("path", "n_accept", "next"), got, want):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("V", [1, 2, 37, 1000, 4099, 50001])
@pytest.mark.parametrize("K,kind,draft", [(1, "chain", True), (4, "chain", True), (9, "chain", True), (1, "chain", False),
                                          (7, "star", False), (31, "random", False), (64, "ragged", False), (64, "chain", False)])
def test_verify_matches_the_rule(cuda_lib, V, K, kind, draft):
    B = 5 if V * K > 100000 else 23
    x = _case(B, K, V, kind, seed=V + K, draft=draft)
    got = _run(cuda_lib, *x)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    _same(got, R.verify(*x))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("u", [0.0, 0.99999994])
def test_verify_all_kept_and_all_turned_down(cuda_lib, draft, u):
    target, q, tokens, parents, us, noise = _case(6, 5, 300, "chain", 4, draft)
    us[:] = u
    x = (target, q, tokens, parents, us, noise)
    got = _run(cuda_lib, *x)
    _same(got, R.verify(*x))
    assert u > 0 or (got[1] == 5).all()


def _offset(x, by, guard):
    """x on the GPU, `by` elements into a buffer whose other elements are `guard`."""
    flat = torch.full((x.size + 8,), guard, dtype=torch.from_numpy(x).dtype, device="cuda")
    flat[by:by + x.size] = torch.from_numpy(x).cuda().flatten()
    return flat[by:by + x.size].view(x.shape)


@pytest.mark.parametrize("by", [(0, 0, 0), (1, 2, 3), (3, 1, 2), (2, 0, 1)])
@pytest.mark.parametrize("V", [5, 8, 9, 70, 1031, 8200, 40003])
def test_verify_any_entry_can_win_whatever_the_alignment(cuda_lib, V, by):
    """One entry of each row stands out, at the ends of the row, of slices and of copies; what lies next
    to the arrays would win if it were read.  Rows 1 on: a turned-down draft, so that its row counts."""
    at = sorted({v for e in (0, V // 8 & ~3, V // 4 & ~3, V // 2, 1028, 2052, V) for v in range(e - 6, e + 7) if 0 <= v < V})
    r = np.random.default_rng(V)
    B = len(at)
    target = r.random((B, 2, V), dtype=np.float32) * np.float32(1e-3)
    target[np.arange(B), 0, at] = 1.0
    noise = r.random((B, V), dtype=np.float32) + np.float32(0.5)
    q = r.random((B, 1, V), dtype=np.float32) * np.float32(1e-4)
    tokens = np.array([[(v + 1) % V] for v in at], np.int32)
    q[np.arange(B), 0, tokens[:, 0]] = 1.0
    parents = np.full((B, 1), -1, np.int32)
    parents[0] = -2
    u = np.full((B, 1), 0.5, np.float32)
    c = lambda x: torch.from_numpy(x).cuda()
    got = cuda_lib.verify_drafts(_offset(target, by[0], 1e30), c(tokens), c(parents), c(u), _offset(noise, by[1], 1e-30),
                                 draft_probs=_offset(q, by[2], -1e30))
    torch.cuda.synchronize()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    assert np.array_equal(got[2].cpu().numpy(), np.array(at, np.int32))
    _same([x.cpu().numpy() for x in got], R.verify(target, q, tokens, parents, u, noise))


def test_verify_nothing_left_and_ties(cuda_lib):
    """p = q where p(x) = 0: nothing is left after the turned-down token, the row itself is drawn from;
    equal scores go to the lowest index."""
    V = 1003
    target = np.zeros((2, 2, V), np.float32)
    target[:, :, 5] = target[:, :, 700] = 0.5
    q = target[:, :1].copy()
    tokens = np.array([[9], [9]], np.int32)
    parents = np.full((2, 1), -1, np.int32)
    x = (target, q, tokens, parents, np.full((2, 1), 0.5, np.float32), np.ones((2, V), np.float32))
    got = _run(cuda_lib, *x)
    _same(got, R.verify(*x))
    assert got[2].tolist() == [5, 5] and got[1].tolist() == [0, 0]
    tokens[:] = 5                                        # without a draft: token 5 turned down leaves 700
    x = (target, None, tokens, parents, np.full((2, 1), 0.9, np.float32), np.ones((2, V), np.float32))
    got = _run(cuda_lib, *x)
    assert got[2].tolist() == [700, 700]
    target[:, 0] = 0
    target[:, 0, 5] = 1                                  # all mass on the turned-down token (u * 1 < 1 keeps it, so u = 1 here)
    x = (target, None, tokens, parents, np.ones((2, 1), np.float32), np.ones((2, V), np.float32))
    _same(_run(cuda_lib, *x), R.verify(*x))


@pytest.mark.parametrize("mode", ["chain", "tree"])
def test_verify_keeps_the_targets_distribution(cuda_lib, mode):
    """The first token out (kept draft or next token) is the target's: 60000 sequences over 8 tokens.
    A count of n p has a standard deviation of at most sqrt(n p); 5 of them, and 3 more counts, is the bar."""
    n, V = 60000, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    p0 = torch.tensor([0.3, 0.02, 0.18, 0.1, 0.05, 0.05, 0.25, 0.05], device="cuda")
    q0 = torch.tensor([0.05, 0.3, 0.1, 0.2, 0.05, 0.1, 0.1, 0.1], device="cuda")
    K = 1 if mode == "chain" else 3
    target = p0.expand(n, K + 1, V).contiguous()
    rnd = lambda *s: torch.rand(s, generator=g, device="cuda")
    noise = torch.empty(n, V, device="cuda").exponential_(generator=g)
    if mode == "chain":
        draft = q0.expand(n, 1, V).contiguous()
        tokens = torch.multinomial(q0.expand(n, V), 1, generator=g).to(torch.int32)
    else:
        draft, tokens = None, torch.tensor([6, 1, 0], dtype=torch.int32, device="cuda").expand(n, 3).contiguous()
    parents = torch.full((n, K), -1, dtype=torch.int32, device="cuda")
    path, count, nxt = cuda_lib.verify_drafts(target, tokens, parents, rnd(n, K), noise, draft_probs=draft)
    first = torch.where(count > 0, tokens.gather(1, path[:, :1].clamp_min(0).long())[:, 0], nxt)
    seen = torch.bincount(first.long(), minlength=V).double().cpu()
    want = p0.double().cpu() * n
    assert ((seen - want).abs() <= 5 * want.sqrt() + 3).all(), (seen, want)


def test_verify_reports_bad_input_and_goes_on(cuda_lib):
    target, q, tokens, parents, u, noise = _case(5, 6, 500, "chain", 9, False)
    bad = [x.copy() for x in (tokens, parents)]
    bad[0][1, 2] = 500                                    # a token outside the vocabulary
    bad[1][2, 1] = 3                                      # a parent that comes later
    bad[1][3, 2] = R.PAD                                  # node 3 hangs on an absent node
    got = _run(cuda_lib, target, None, bad[0], bad[1], u, noise)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    want = R.verify(target, None, tokens, parents, u, noise)
    for b in (0, 4):
        assert all(np.array_equal(g[b], w[b]) for g, w in zip(got, want))
    for b in (1, 2, 3):
        assert (got[0][b] == -1).all() and got[1][b] == 0 and got[2][b] == -1
    target, q, tokens, parents, u, noise = _case(2, 3, 50, "star", 9, False)     # siblings with a draft
    got = _run(cuda_lib, target, target[:, :3].copy(), tokens, parents, u, noise)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG and (got[2] == -1).all()


def test_verify_feeds_decode_multi(cuda_lib):
    """n_accept of a chain is decode_multi's n_apply."""
    x = _case(7, 4, 100, "chain", 2, True)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    side = torch.cuda.Stream()
    ins = [c(x[0]), c(x[2]), c(x[3]), c(x[4]), c(x[5])]
    dr = c(x[1])
    side.wait_stream(torch.cuda.current_stream())
    path, n, nxt = cuda_lib.verify_drafts(*ins, draft_probs=dr, stream=side)
    side.synchronize()
    want = R.verify(*x)
    assert np.array_equal(n.cpu().numpy(), want[1])
    B, K, H, D = 7, 4, 2, 128
    rnd = lambda *s: torch.randn(*s, device="cuda")
    k = torch.nn.functional.normalize(rnd(B, K, H, D), dim=-1)
    state = rnd(B, H, D, D)
    before = state.clone()
    cuda_lib.decode_multi(k, k, rnd(B, K, H, D), -rnd(B, K, H, D).abs(), torch.rand(B, K, H, device="cuda"), state, n_apply=n)
    moved = [not torch.equal(state[b], before[b]) for b in range(B)]
    assert moved == [int(m) > 0 for m in want[1]]


# ------------------------------------------------------------------ page tables
def _tables(kda, ctx, new, held, table, free, ps, max_tokens):
    c = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    t = c(table)
    slots, cu, out, taken = kda.page_tables(c(ctx), c(new), c(held), t, c(free), page_size=ps, max_tokens=max_tokens)
    torch.cuda.synchronize()
    return slots.cpu().numpy(), cu.cpu().numpy(), out.cpu().numpy(), int(taken), t.cpu().numpy()


def _requests(B, seed, ps, most_ctx, most_new):
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, most_ctx + 1, B), r.integers(0, most_new + 1, B)
    held = -(-ctx // ps) + r.integers(0, 3, B)
    cols = int((-(-(ctx + new) // ps)).max() if B else 0) + 3
    table = r.integers(0, 10 ** 6, (B, cols)).astype(np.int32)
    return ctx, new, held, table, r.permutation(10 ** 5).astype(np.int32)


@pytest.mark.parametrize("B,ps,most_ctx,most_new", [(1, 16, 0, 1), (1, 1, 5, 7), (7, 64, 1000, 16), (33, 24, 300, 900), (256, 16, 50, 5),
                                                    (257, 128, 4000, 64), (1500, 8, 100, 9), (13000, 4, 20, 3)])
@pytest.mark.parametrize("share", [1.0, 0.6, 0.0])
def test_tables_match_the_loop(cuda_lib, B, ps, most_ctx, most_new, share):
    """share: of the free pages that are needed; the rest of the requests is refused."""
    ctx, new, held, table, free = _requests(B, B + ps, ps, most_ctx, most_new)
    need = int(np.maximum(-(-(ctx + new) // ps) - held, 0).sum())
    free = free[:int(need * share)]
    total = int(new.sum()) + 5
    got = _tables(cuda_lib, ctx, new, held, table, free, ps, total)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
    for g, w in zip(got, R.page_tables(ctx, new, held, table, free, ps, total)):
        assert np.array_equal(g, w)


def test_tables_refuse_what_exceeds_a_row(cuda_lib):
    ctx, new, held = [10, 30, 4], [5, 3, 4], [1, 2, 1]
    table, free = np.zeros((3, 2), np.int32), np.arange(40, 50, dtype=np.int32)
    got = _tables(cuda_lib, ctx, new, held, table, free, 16, 12)
    want = R.page_tables(ctx, new, held, table, free, 16, 12)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert (got[0][5:8] == -1).all() and cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("what", ["negative", "uncovered", "too_many"])
def test_tables_report_bad_input_and_go_on(cuda_lib, what):
    ctx, new, held = [10, 20, 4], [5, 3, 4], [1, 2, 1]
    table, free = np.arange(12, dtype=np.int32).reshape(3, 4), np.arange(40, 50, dtype=np.int32)
    bad = {"negative": ([10, -20, 4], [1, 2, 1]), "uncovered": ([10, 20, 4], [1, 1, 1]), "too_many": ([10, 20, 4], [1, 5, 1])}[what]
    got = _tables(cuda_lib, bad[0], new, bad[1], table, free, 16, 9)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    want = R.page_tables([10, 16, 4], [5, 0, 4], [1, 1, 1], table, free, 16, 9)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[2].tolist() == [1, bad[1][1], 1]


def test_tables_short_slot_map_and_no_requests(cuda_lib):
    got = _tables(cuda_lib, [3], [10], [1], [[7, -1]], [9], 8, 6)
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    assert got[0].tolist() == [59, 60, 61, 62, 63, 72] and got[4].tolist() == [[7, 9]]
    got = _tables(cuda_lib, [], [], [], np.zeros((0, 4)), [], 8, 3)
    assert got[0].tolist() == [-1] * 3 and got[1].tolist() == [0] and got[3] == 0


def test_tables_give_prefill_its_cu_seqlens(cuda_lib):
    """Prompts paged from nothing: cu_seqlens is what kda_prefill takes."""
    lens = np.array([70, 1, 130], np.int32)
    c = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    _, cu, _, _ = cuda_lib.page_tables(c([0, 0, 0]), c(lens), c([0, 0, 0]), c(np.full((3, 9), -1)), c(np.arange(20)),
                                       page_size=16, max_tokens=int(lens.sum()))
    T, H, D = int(lens.sum()), 2, 64
    rnd = lambda *s: torch.randn(*s, device="cuda")
    k = torch.nn.functional.normalize(rnd(T, H, D), dim=-1)
    args = (k, k, rnd(T, H, D), -rnd(T, H, D).abs().clamp_max(5), torch.rand(T, H, device="cuda"))
    a, _ = cuda_lib.prefill(*args, cu)
    b, _ = cuda_lib.prefill(*args, torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and cuda_lib.last_device_status() == cuda_lib.KDA_OK
