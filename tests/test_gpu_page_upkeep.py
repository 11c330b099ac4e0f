"""kda_page_fork, kda_page_release, kda_cache_copy and kda_cache_keep_path against loops over the same lists: whole numbers
and moved rows, equal to the last bit."""
import numpy as np
import pytest
import torch

import _prompt_ref as R

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _gpu(x, dtype=I32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def _rows(r, rows, cols, ps, held, spare=20):
    """(table, shares, free): rows of distinct pages in random order, some pages shared with an earlier row."""
    P = int(sum(held)) + spare
    ids = r.permutation(P).astype(np.int32)
    table = np.full((rows, cols), -7, np.int32)
    shares, at = np.zeros(P, np.int32), 0
    for i, h in enumerate(held):
        j = int(r.integers(0, i)) if i and r.random() < 0.5 else -1
        common = int(r.integers(0, min(h, held[j]) + 1)) if j >= 0 else 0
        table[i, :common] = table[j, :common]
        shares[table[i, :common]] += 1
        table[i, common:h] = ids[at:at + h - common]
        at += h - common
    return table, shares, ids[at:]


# ------------------------------------------------------------------ forks
def _fork(kda, parents, children, lens, held, table, shares, free, ps, status=None):
    t, s = _gpu(table), _gpu(shares)
    out, copies, taken = kda.page_fork(_gpu(parents), _gpu(children), _gpu(lens), _gpu(held), t, s, _gpu(free), page_size=ps)
    torch.cuda.synchronize()
    h, tab, sh, cop, used, bad = R.page_fork(parents, children, lens, held, table, shares, free, ps)
    assert kda.last_device_status() == (kda.KDA_ERR_INVALID_ARG if bad else kda.KDA_OK)
    assert out.tolist() == h and taken.tolist() == [used] and copies.tolist() == [list(c) for c in cop]
    assert np.array_equal(t.cpu().numpy(), tab) and s.tolist() == list(sh)
    return bad


@pytest.mark.parametrize("ps", [1, 7, 16, 256])
@pytest.mark.parametrize("rows,cols,n", [(2, 3, 1), (9, 40, 5), (70, 300, 64), (700, 9, 500), (40, 1100, 30)])
def test_forks(cuda_lib, ps, rows, cols, n):
    r = np.random.default_rng(ps * rows)
    held = [0] * rows
    order = r.permutation(rows)
    kids, rest = order[:n], order[n:]
    for p in rest:
        held[p] = int(r.integers(0, cols + 1))
    table, shares, free = _rows(r, rows, cols, ps, held, spare=n + 3)
    parents = r.choice(rest, n)
    lens = [int(r.integers(0, held[p] * ps + 1)) for p in parents]
    assert not _fork(cuda_lib, parents.tolist(), kids.tolist(), lens, held, table, shares, free, ps)


def test_forks_of_all_lengths_around_a_page(cuda_lib):
    held, ps = [4] + [0] * 9, 5
    table, shares, free = _rows(np.random.default_rng(0), 10, 6, ps, held)
    assert not _fork(cuda_lib, [0] * 9, list(range(1, 10)), [0, 1, 4, 5, 6, 9, 10, 19, 20], held, table, shares, free, ps)


@pytest.mark.parametrize("free", [0, 1, 3])
def test_forks_when_pages_run_out(cuda_lib, free):
    """First come, first served; forks of whole pages go on."""
    held, ps = [3] + [0] * 7, 4
    table, shares, ids = _rows(np.random.default_rng(0), 8, 3, ps, held)
    assert not _fork(cuda_lib, [0] * 7, [3, 1, 7, 2, 5, 4, 6], [5, 8, 0, 9, 12, 1, 11], held, table, shares, ids[:free], ps)


def test_forks_that_do_nothing(cuda_lib):
    """Rows out of range, children twice or parents too, lengths that are not covered, children that hold pages, pages held out of range; the
    others go on.  Page ids out of range."""
    held, ps = [3, 2, 0, 0, 0, 0, 9, -1, 0, 0], 4
    table, shares, free = _rows(np.random.default_rng(0), 10, 6, ps, [3, 2, 0, 0, 0, 0, 0, 0, 0, 0])
    parents = [0, -1, 10, 0, 0, 0, 1, 0, 6, 7, 2]
    kids = [2, 3, 3, -1, 10, 4, 5, 1, 8, 8, 9]
    lens = [13, 1, 1, 1, 1, 6, 8, 2, 1, 1, 0]
    for pick in ([0, 5, 6], [1, 5, 7, 9], [2, 3, 4, 5, 8], [5, 10, 0, 6], [5, 5, 6], [6, 10]):
        _fork(cuda_lib, [parents[i] for i in pick], [kids[i] for i in pick], [lens[i] for i in pick], held, table, shares, free, ps)
    assert _fork(cuda_lib, [0, 0], [2, 3], [4, -1], held, table, shares, free, ps)
    table[0, :3] = [-1, 5, len(shares)]
    assert _fork(cuda_lib, [0, 0, 0], [2, 3, 4], [12, 10, 8], held, table, shares, free, ps)
    table[0, :3] = [1, 5, 2]
    assert _fork(cuda_lib, [0], [2], [3], held, table, shares, [-4], ps)


def test_a_fork_of_many_rows_and_nothing(cuda_lib):
    rows = cuda_lib.KDA_PAGE_TABLES_MAX_BATCH
    held = [2] + [0] * (rows - 1)
    table, shares, free = _rows(np.random.default_rng(0), rows, 2, 3, held, spare=rows)
    t, s = _gpu(table), _gpu(shares)
    n = rows - 1
    out, copies, taken = cuda_lib.page_fork(_gpu([0] * n), _gpu(np.arange(1, rows)), _gpu([4] * n), _gpu(held), t, s, _gpu(free), page_size=3)
    assert taken.item() == n and (out == 2).all() and s[int(table[0, 0])].item() == n
    assert torch.equal(t[1:, 1].cpu(), torch.as_tensor(free[:n])) and torch.equal(copies[:, 1].cpu(), torch.as_tensor(free[:n]))
    e = _gpu(np.zeros(0))
    out, copies, taken = cuda_lib.page_fork(e, e, e, _gpu([1, 0]), _gpu(np.zeros((2, 3))), _gpu([0]), e, page_size=3)
    assert out.tolist() == [1, 0] and copies.shape == (0, 3) and taken.item() == 0
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


# ------------------------------------------------------------------ releases
def _release(kda, keep, held, table, shares, ps):
    s = _gpu(shares)
    out, freed, n = kda.page_release(_gpu(keep), _gpu(held), _gpu(table), s, page_size=ps)
    torch.cuda.synchronize()
    h, sh, free, bad = R.page_release(keep, held, table, shares, ps)
    assert kda.last_device_status() == (kda.KDA_ERR_INVALID_ARG if bad else kda.KDA_OK)
    assert out.tolist() == h and s.tolist() == list(sh) and n.item() == len(free)
    assert freed.tolist() == free + [-1] * (len(shares) - len(free))
    return bad


@pytest.mark.parametrize("ps", [1, 7, 64])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (40, 300), (600, 20), (5, 3000)])
def test_releases(cuda_lib, ps, rows, cols):
    r = np.random.default_rng(ps + rows)
    held = [int(r.integers(0, cols + 1)) for _ in range(rows)]
    table, shares, _ = _rows(r, rows, cols, ps, held, spare=77)
    for kind in range(3):
        if kind == 0:
            keep = [0] * rows
        elif kind == 1:            # whole pages: nothing is refused
            keep = [int(r.integers(0, h + 2)) * ps for h in held]
        else:
            keep = [int(r.integers(0, h * ps + 3)) for h in held]
        bad = _release(cuda_lib, keep, held, table, shares, ps)
        assert not bad or (kind == 2 and ps > 1)


def test_a_page_that_others_hold_is_not_cut(cuda_lib):
    table = np.array([[0, 1, 2], [0, 1, 3], [0, 4, -1]], np.int32)
    shares = [2, 1, 0, 0, 0, 0]
    assert _release(cuda_lib, [5, 8, 4], [3, 3, 2], table, shares, 4)        # row 0 inside page 1
    assert not _release(cuda_lib, [9, 8, 5], [3, 3, 2], table, shares, 4)    # inside their own last pages
    assert not _release(cuda_lib, [0, 0, 0], [3, 3, 2], table, shares, 4)
    table = np.array([[0, 1], [0, 1], [2, 3]], np.int32)                     # inside the last page that is held: no page goes, but what
    assert _release(cuda_lib, [7, 8, 8], [2, 2, 2], table, [1, 1, 0, 0], 4)  # the row appends there would be row 1's
    assert not _release(cuda_lib, [8, 9, 7], [2, 2, 2], table, [1, 1, 0, 0], 4)


def test_releases_of_bad_rows(cuda_lib):
    table = np.array([[0, 1, 2], [3, -1, 9], [1, 1, 4], [5, 6, 7]], np.int32)
    for keep, held in (([-1, 0, 0, 0], [3, 1, 0, 3]), ([0, 0, 0, 0], [4, 3, 0, -2]), ([0, 0, 0, 4], [3, 0, 3, 3]), ([0, 5, 0, 0], [0, 3, 0, 0])):
        assert _release(cuda_lib, keep, held, table, [0] * 9, 4)


def test_release_of_a_large_pool_and_nothing(cuda_lib):
    """More pages than the threads take in one round; a long row; no rows, no pages."""
    P, cols = 300001, 9000
    r = np.random.default_rng(1)
    ids = r.permutation(P).astype(np.int32)
    table = np.stack([ids[i * cols:(i + 1) * cols] for i in range(30)])
    keep = [0 if i % 3 else 5000 * 16 for i in range(30)]
    s = torch.zeros(P, dtype=I32, device="cuda")
    held, freed, n = cuda_lib.page_release(_gpu(keep), _gpu([cols] * 30), _gpu(table), s, page_size=16)
    want = np.sort(np.concatenate([table[i, (0 if i % 3 else 5000):] for i in range(30)]))
    assert n.item() == len(want) and np.array_equal(freed.cpu().numpy()[:len(want)], want) and (freed[len(want):] == -1).all() and not s.any()
    assert held.tolist() == [0 if i % 3 else 5000 for i in range(30)]
    e = torch.zeros(0, dtype=I32, device="cuda")
    held, freed, n = cuda_lib.page_release(e, e, torch.zeros((0, 4), dtype=I32, device="cuda"), e, page_size=16)
    assert held.numel() == 0 and freed.numel() == 0 and n.item() == 0
    held, freed, n = cuda_lib.page_release(_gpu([0]), _gpu([0]), torch.zeros((1, 0), dtype=I32, device="cuda"), s[:5], page_size=16)
    assert held.tolist() == [0] and freed.tolist() == [-1] * 5 and n.item() == 0
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


# ------------------------------------------------------------------ copies and kept paths
def _cache(L, P, ps, Hk, D, dtype, seed=0):
    return torch.randn(L, P, 2, ps, Hk, D, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("L,ps,Hk,D", [(1, 16, 8, 128), (3, 7, 2, 64), (2, 300, 4, 128), (5, 1, 1, 8)])
def test_copies(cuda_lib, dtype, L, ps, Hk, D):
    cache = _cache(L, 20, ps, Hk, D, dtype)
    copies = [(3, 4, ps), (3, 5, 1), (19, 0, ps - 1), (-1, -1, 0), (7, 7, ps), (2, 6, max(1, ps // 2))]
    got = cache.cuda()
    cuda_lib.cache_copy(_gpu(copies), got[:, :, 0], got[:, :, 1])
    assert torch.equal(got.cpu(), R.cache_copy(copies, cache, ps)) and cuda_lib.last_device_status() == cuda_lib.KDA_OK
    one = cache[0].cuda()                                      # one layer's, and separate caches
    cuda_lib.cache_copy(_gpu(copies), one[:, 0], one[:, 1])
    assert torch.equal(one.cpu(), R.cache_copy(copies, cache, ps)[0])
    k, v = cache[:, :, 0].contiguous().cuda(), cache[:, :, 1].contiguous().cuda()
    cuda_lib.cache_copy(_gpu(copies), k, v)
    want = R.cache_copy(copies, cache, ps)
    assert torch.equal(k.cpu(), want[:, :, 0]) and torch.equal(v.cpu(), want[:, :, 1])
    swapped = cache.transpose(0, 1).contiguous().cuda()        # pages outside, layers inside
    kv = swapped.transpose(0, 1)
    cuda_lib.cache_copy(_gpu(copies), kv[:, :, 0], kv[:, :, 1])
    assert torch.equal(kv.cpu(), want)


def test_copies_out_of_range_are_left_out(cuda_lib):
    cache = _cache(2, 5, 4, 2, 64, torch.float32)
    copies = [(0, 1, 4), (-1, 2, 3), (0, 5, 1), (5, 0, 1), (0, 2, 5), (0, 2, -1), (3, 4, 2)]
    got = cache.cuda()
    cuda_lib.cache_copy(_gpu(copies), got[:, :, 0], got[:, :, 1])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    assert torch.equal(got.cpu(), R.cache_copy([copies[0], copies[6]], cache, 4))
    cuda_lib.cache_copy(_gpu(np.zeros((0, 3))), got[:, :, 0], got[:, :, 1])
    cuda_lib.cache_copy(_gpu([(0, 0, 0)]), got[:, :0, 0], got[:, :0, 1])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def _step(r, B, K, ps, spare=2):
    first = r.integers(0, ps, B)
    pages = [-(-(int(f) + K) // ps) for f in first]
    P = sum(pages) + spare
    ids, at, slots = r.permutation(P), 0, np.zeros((B, K), np.int64)
    for b in range(B):
        mine = ids[at:at + pages[b]]
        at += pages[b]
        pos = first[b] + np.arange(K)
        slots[b] = mine[pos // ps] * ps + pos % ps
    path, n = np.full((B, K), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n[b] = r.integers(0, K + 1)
        path[b, :n[b]] = np.sort(r.choice(K, n[b], replace=False))
    return slots, path, n, P


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,K,ps,L,Hk,D", [(1, 1, 16, 1, 8, 128), (4, 7, 16, 1, 8, 128), (33, 64, 7, 2, 2, 64), (70, 16, 1, 3, 1, 128), (3, 40, 128, 2, 16, 128)])
def test_kept_paths(cuda_lib, dtype, B, K, ps, L, Hk, D):
    slots, path, n, P = _step(np.random.default_rng(B), B, K, ps)
    cache = _cache(L, P, ps, Hk, D, dtype)
    got = cache.cuda()
    cuda_lib.cache_keep_path(_gpu(slots, torch.int64), _gpu(path), _gpu(n), got[:, :, 0], got[:, :, 1])
    assert torch.equal(got.cpu(), R.keep_path(slots, path, n, cache)) and cuda_lib.last_device_status() == cuda_lib.KDA_OK
    one = cache[0].cuda()
    cuda_lib.cache_keep_path(_gpu(slots, torch.int64), _gpu(path), _gpu(n), one[:, 0], one[:, 1])
    assert torch.equal(one.cpu(), R.keep_path(slots, path, n, cache)[0])


def test_bad_paths_leave_their_sequence(cuda_lib):
    slots, path, n, P = _step(np.random.default_rng(1), 6, 40, 16)
    path[:], n[:] = -1, 0
    for b in range(6):
        path[b, :20], n[b] = np.arange(20) * 2, 20
    path[0, 5] = path[0, 4]             # not ascending
    path[1, 19] = 40
    path[2, 0] = -1
    n[3] = 41
    slots[4, 38] = P * 16
    cache = _cache(2, P, 16, 2, 64, torch.float32)
    got = cache.cuda()
    cuda_lib.cache_keep_path(_gpu(slots, torch.int64), _gpu(path), _gpu(n), got[:, :, 0], got[:, :, 1])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_ERR_INVALID_ARG
    n[:5] = 0
    assert torch.equal(got.cpu(), R.keep_path(slots, path, n, cache))
    slots[:, 0] = -1                    # a slot from and to which nothing moves is not looked at
    got = cache.cuda()
    cuda_lib.cache_keep_path(_gpu(slots, torch.int64), _gpu(path), _gpu(n), got[:, :, 0], got[:, :, 1])
    assert torch.equal(got.cpu(), R.keep_path(slots[:, 1:], np.array([[p - 1 for p in row[1:]] for row in path]), np.maximum(n - 1, 0), cache))
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_offsets_past_32_bits(cuda_lib):
    P = 2 ** 31 // (2 * 64 * 8 * 128) + 5
    kv = torch.empty((P, 2, 64, 8, 128), dtype=torch.bfloat16, device="cuda")
    kv[P - 1].normal_()
    kv[1].normal_()
    kv[P - 2].normal_()
    before = kv[[1, P - 2, P - 1]].clone()
    cuda_lib.cache_copy(_gpu([(P - 1, 0, 64), (1, P - 3, 7)]), kv[:, 0], kv[:, 1])
    assert torch.equal(kv[0], before[2]) and torch.equal(kv[P - 3, :, :7], before[0, :, :7])
    slots = torch.tensor([[64, (P - 2) * 64 + 5]], device="cuda")
    cuda_lib.cache_keep_path(slots, _gpu([[1, -1]]), _gpu([1]), kv[:, 0], kv[:, 1])
    assert torch.equal(kv[1, :, 0], before[1, :, 5]) and torch.equal(kv[1, :, 1:], before[0, :, 1:])


def test_upkeep_in_graphs_and_on_another_stream(cuda_lib):
    """Fork, copy, release and kept path captured together and replayed twice: every replay starts from the buffers as they are."""
    r = np.random.default_rng(5)
    held = [3, 0, 0, 2]
    table, shares, free = _rows(r, 4, 5, 4, held)
    cache = _cache(2, len(shares), 4, 2, 64, torch.bfloat16)
    t, s, got = _gpu(table), _gpu(shares), cache.cuda()
    args = [_gpu(x) for x in ([0, 0], [1, 2], [10, 5], held)]
    fr, keep = _gpu(free), _gpu([12, 0, 0, 8])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, copies, taken = cuda_lib.page_fork(*args, t, s, fr, page_size=4)
        cuda_lib.cache_copy(copies, got[:, :, 0], got[:, :, 1])
        back, freed, count = cuda_lib.page_release(keep, out, t, s, page_size=4)
    h, tab, sh, cop, used, _ = R.page_fork([0, 0], [1, 2], [10, 5], held, table, shares, free, 4)
    h2, sh2, free2, _ = R.page_release([12, 0, 0, 8], h, tab, sh, 4)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == h and copies.tolist() == [list(c) for c in cop] and taken.item() == used
        assert back.tolist() == h2 and s.tolist() == list(sh2) and freed.tolist()[:count.item()] == free2
        assert torch.equal(got.cpu(), R.cache_copy(cop, cache, 4))
    with torch.cuda.stream(side):
        o2, c2, _ = cuda_lib.page_fork(*args, t, s, fr, page_size=4)
        b2, f2, n2 = cuda_lib.page_release(keep, o2, t, s, page_size=4)
    side.synchronize()
    assert o2.tolist() == h and b2.tolist() == h2 and f2.tolist()[:n2.item()] == free2
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_releases_of_large_pools_in_graphs_and_on_two_streams(cuda_lib):
    """The form with a barrier of the whole grid: captured and replayed, then two calls on two streams at once."""
    P, cols, rows = 50000, 700, 60
    r = np.random.default_rng(3)
    ids = r.permutation(P).astype(np.int32)
    tables = [_gpu(ids[:rows * cols].reshape(rows, cols)), _gpu(ids[-rows * cols:].reshape(rows, cols))]
    keep, held = _gpu([0 if i % 4 else 320 * 16 for i in range(rows)]), _gpu([cols] * rows)
    want = [np.sort(np.concatenate([t[i, (0 if i % 4 else 320):] for i in range(rows)])) for t in (x.cpu().numpy() for x in tables)]
    shares = torch.zeros(P, dtype=I32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, freed, n = cuda_lib.page_release(keep, held, tables[0], shares, page_size=16)
    for _ in range(2):
        freed.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert n.item() == len(want[0]) and np.array_equal(freed.cpu().numpy()[:n.item()], want[0]) and (freed[n.item():] == -1).all() and not shares.any()
        assert h.tolist() == [0 if i % 4 else 320 for i in range(rows)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, cuda_lib.page_release(keep, held, tables[k], torch.zeros(P, dtype=I32, device="cuda"), page_size=16)))
    torch.cuda.synchronize()
    for k, (_, freed, n) in got:
        assert n.item() == len(want[k]) and np.array_equal(freed.cpu().numpy()[:n.item()], want[k])
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


def test_forks_and_copies_on_two_streams(cuda_lib):
    """Two tables and caches at once; each call's shared memory and outputs are its own."""
    r = np.random.default_rng(8)
    cases = []
    for k in range(2):
        held = [5, 0, 0, 0]
        table, shares, free = _rows(r, 4, 6, 8, held, spare=9)
        cases.append((table, shares, free, held, _cache(3, len(shares), 8, 2, 64, torch.bfloat16, seed=k)))
    streams, done = [torch.cuda.Stream() for _ in range(2)], []
    for (table, shares, free, held, cache), s in zip(cases, streams):
        with torch.cuda.stream(s):
            t, sh, c = _gpu(table), _gpu(shares), cache.cuda()
            out, copies, taken = cuda_lib.page_fork(_gpu([0, 0, 0]), _gpu([1, 3, 2]), _gpu([33, 8, 39]), _gpu(held), t, sh, _gpu(free), page_size=8)
            cuda_lib.cache_copy(copies, c[:, :, 0], c[:, :, 1])
            done.append((out, copies, t, sh, c))
    torch.cuda.synchronize()
    for (table, shares, free, held, cache), (out, copies, t, sh, c) in zip(cases, done):
        h, tab, want, cop, _, bad = R.page_fork([0, 0, 0], [1, 3, 2], [33, 8, 39], held, table, shares, free, 8)
        assert not bad and out.tolist() == h and copies.tolist() == [list(x) for x in cop] and np.array_equal(t.cpu().numpy(), tab) and sh.tolist() == list(want)
        assert torch.equal(c.cpu(), R.cache_copy(cop, cache, 8))
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK
