"""Host-side checks of the draft-step entry points: every refusal comes before anything
reaches a GPU, from the C calls and from the Python binding (CPU only)."""
import ctypes

import pytest
import torch

import linear_attention_serving_chunkwise_gb300 as kda
from linear_attention_serving_chunkwise_gb300.build import build

BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return kda.load()


def _p(a):
    return None if a is None else ctypes.c_void_p(a)


def test_page_tables_refusals(lib):
    names = ("ctx", "new", "held", "table", "free", "slots", "cu", "out", "taken")
    base = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    call = lambda B=4, cols=8, F=10, ps=16, T=64, **kw: lib.kda_page_tables(
        B, cols, F, ps, T, *[_p(kw.get(n, base[n])) for n in names], None)
    for kw in (dict(B=-1), dict(cols=-1), dict(F=-1), dict(ps=0), dict(T=-1), dict(B=16000, cols=1 << 20)):
        assert call(**kw) == BAD
    assert call(B=kda.KDA_PAGE_TABLES_MAX_BATCH + 1) == UNSUP
    for n in names:
        assert call(**{n: None}) == BAD
        assert call(**{n: base[n] + 2}) == BAD
    assert call(slots=base["slots"] + 4) == BAD
    assert call(table=base["free"]) == BAD              # the table is written
    assert call(out=base["held"]) == BAD
    assert call(slots=base["cu"]) == BAD
    assert call(taken=base["cu"] + 16) == BAD


def _desc(**kw):
    d = dict(batch=2, nodes=4, num_heads=8, num_kv_heads=2, dim=128, dtype=kda.KDA_BF16, num_pages=10, page_size=16,
             table_cols=5, scale=0.1, k_page_stride=16 * 2 * 128, v_page_stride=16 * 2 * 128)
    d.update(kw)
    return kda.make_tree_attention_desc(**d)


def test_tree_attention_refusals(lib):
    names = ("q", "k", "v", "table", "ctx", "par", "out", "ws")
    base = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}

    def call(desc=None, nbytes=1 << 40, **kw):
        d = _desc() if desc is None else desc
        return lib.kda_tree_attention(ctypes.byref(d), *[_p(kw.get(n, base[n])) for n in names], nbytes, None)

    for kw in (dict(batch=-1), dict(nodes=0), dict(nodes=65), dict(num_heads=0), dict(num_kv_heads=3), dict(num_kv_heads=0),
               dict(page_size=0), dict(num_pages=-1), dict(table_cols=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(k_page_stride=16 * 2 * 128 - 8), dict(v_page_stride=16 * 2 * 128 + 4), dict(k_page_stride=1 << 62)):
        assert call(_desc(**kw)) == BAD, kw
        assert kda.tree_attention_workspace_bytes(_desc(**kw)) == 0
    for kw in (dict(dim=96), dict(dtype=5)):
        assert call(_desc(**kw)) == UNSUP
    assert lib.kda_tree_attention(None, *[_p(base[n]) for n in names], 1 << 40, None) == BAD
    need = kda.tree_attention_workspace_bytes(_desc())
    assert need > 0
    assert call(nbytes=need - 1) == kda.KDA_ERR_WORKSPACE
    for n in names:
        assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    assert call(out=base["q"]) == BAD
    assert call(out=base["v"] + 16 * 2 * 128 * 2 * 9) == BAD       # inside the last page of the cache
    assert call(nbytes=need, out=base["ws"] + 16) == BAD
    assert call(_desc(batch=0), q=None, ctx=None) == kda.KDA_OK
    assert kda.tree_attention_workspace_bytes(_desc(batch=0)) == 0


@pytest.mark.parametrize("dtype", [kda.KDA_BF16, kda.KDA_F32])
def test_tree_attention_refuses_more_tiles_than_it_counts(lib, dtype):
    """2^21 pages of 64 tokens: 16 sequences x 2 heads fit 32-bit tile numbers, 4096 do not."""
    wide = dict(dtype=dtype, page_size=64, table_cols=1 << 21, k_page_stride=64 * 2 * 128, v_page_stride=64 * 2 * 128)
    assert kda.tree_attention_workspace_bytes(_desc(batch=16, **wide)) > 0
    d = _desc(batch=4096, **wide)
    assert kda.tree_attention_workspace_bytes(d) == 0
    assert lib.kda_tree_attention(ctypes.byref(d), *[_p(0x10000000 * (i + 1)) for i in range(8)], 1 << 40, None) == UNSUP


def test_tree_decode_and_commit_refusals(lib):
    names = ("q", "k", "v", "g", "beta", "par", "gate", "state", "out", "w")
    base = {n: 0x1000000 * (i + 1) for i, n in enumerate(names)}
    call = lambda B=2, K=4, H=2, d=64, dv=64, dt=0, pro=0, **kw: lib.kda_tree_decode(
        B, K, H, d, dv, dt, pro, *[_p(kw.get(n, base[n])) for n in names], None)
    for kw in (dict(B=-1), dict(K=0), dict(K=65), dict(H=0), dict(pro=8), dict(pro=-1), dict(B=1 << 24, K=64, H=64)):
        assert call(**kw) == BAD, kw
    for kw in (dict(d=96, dv=96), dict(d=128), dict(dt=3)):
        assert call(**kw) == UNSUP, kw
    for n in names:
        if n != "gate":
            assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    assert call(out=base["state"]) == BAD and call(w=base["out"]) == BAD and call(out=base["gate"] + 64) == BAD
    assert call(B=0) == kda.KDA_OK

    names2 = ("k", "g", "w", "path", "n", "state")
    base2 = {n: 0x1000000 * (i + 1) for i, n in enumerate(names2)}
    com = lambda B=2, K=4, H=2, d=64, dv=64, dt=0, pro=0, **kw: lib.kda_tree_commit(
        B, K, H, d, dv, dt, pro, *[_p(kw.get(n, base2[n])) for n in names2], None)
    for kw in (dict(B=-1), dict(K=65), dict(pro=8)):
        assert com(**kw) == BAD
    assert com(d=32, dv=32) == UNSUP
    for n in names2:
        assert com(**{n: None}) == BAD and com(**{n: base2[n] + 2}) == BAD
    assert com(state=base2["w"]) == BAD and com(B=0) == kda.KDA_OK


def test_verify_refusals(lib):
    names = ("target", "draft", "tok", "par", "u", "noise", "path", "n", "next")
    base = {n: 0x1000000 * (i + 1) for i, n in enumerate(names)}
    call = lambda B=2, K=4, V=100, **kw: lib.kda_verify_drafts(B, K, V, *[_p(kw.get(n, base[n])) for n in names], None)
    for kw in (dict(B=-1), dict(K=0), dict(K=65), dict(V=0), dict(B=1 << 25)):
        assert call(**kw) == BAD, kw
    for n in names:
        if n != "draft":
            assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    assert call(path=base["tok"]) == BAD and call(n=base["path"]) == BAD
    assert call(B=0) == kda.KDA_OK


def test_binding_refuses_wrong_tensors():
    """Shapes and types that the C calls cannot see."""
    i32 = torch.int32
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    with pytest.raises(TypeError):
        kda.verify_drafts(z(2, 4, 9), z(2, 3, dt=torch.int64), z(2, 3, dt=i32), z(2, 3), z(2, 9))
    with pytest.raises(ValueError):
        kda.verify_drafts(z(2, 4, 9), z(2, 3, dt=i32), z(2, 3, dt=i32), z(2, 3), z(2, 8))
    with pytest.raises(ValueError):
        kda.verify_drafts(z(2, 4, 9), z(2, 3, dt=i32), z(2, 3, dt=i32), z(2, 3), z(2, 9), draft_probs=z(2, 4, 9))
    with pytest.raises(ValueError):
        kda.page_tables(z(3, dt=i32), z(2, dt=i32), z(3, dt=i32), z(3, 4, dt=i32), z(5, dt=i32), page_size=4, max_tokens=3)
    q, k = z(2, 3, 4, 64), z(5, 8, 2, 64)
    with pytest.raises(TypeError):
        kda.tree_attention(q, k.bfloat16(), k, z(2, 2, dt=i32), z(2, dt=i32), z(2, 3, dt=i32))
    with pytest.raises(ValueError):
        kda.tree_attention(q, k, k, z(1, 2, dt=i32), z(2, dt=i32), z(2, 3, dt=i32))
    with pytest.raises(ValueError):                                  # pages that are not contiguous
        kda.tree_attention(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, z(2, 2, dt=i32), z(2, dt=i32), z(2, 3, dt=i32))
    x = z(2, 3, 4, 64)
    with pytest.raises(ValueError):
        kda.tree_decode(x, x, x, x, z(2, 3, 4), z(2, 3, dt=i32), z(2, 4, 64, 32))
    with pytest.raises(TypeError):
        kda.tree_decode(x, x, x, x, z(2, 3, 4), z(2, 3), z(2, 4, 64, 64))
    with pytest.raises(ValueError):
        kda.tree_commit(x, x, x, z(2, 2, dt=i32), z(2, dt=i32), z(2, 4, 64, 64))
