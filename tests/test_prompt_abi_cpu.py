"""Host-side checks of the prompt path's and the cache upkeep's entry points: every refusal comes before anything
reaches a GPU, from the C calls and from the Python binding (CPU only)."""
import ctypes

import pytest
import torch

import linear_attention_serving_chunkwise_gb300 as kda
from linear_attention_serving_chunkwise_gb300 import _lib
from linear_attention_serving_chunkwise_gb300.build import build

BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return kda.load()


def _p(a):
    return None if a is None else ctypes.c_void_p(a)


def _chunk(**kw):
    d = dict(batch=2, total_tokens=40, num_heads=8, num_kv_heads=2, dim=128, dtype=kda.KDA_BF16, num_pages=10, page_size=16,
             table_cols=5, scale=0.1, k_page_stride=16 * 2 * 128, v_page_stride=16 * 2 * 128)
    d.update(kw)
    return kda.make_chunk_attention_desc(**d)


def test_chunk_attention_refusals(lib):
    names = ("q", "k", "v", "table", "ctx", "cu", "out", "ws")
    base = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}

    def call(desc=None, nbytes=1 << 40, **kw):
        d = _chunk() if desc is None else desc
        return lib.kda_chunk_attention(ctypes.byref(d), *[_p(kw.get(n, base[n])) for n in names], nbytes, None)

    for kw in (dict(batch=-1), dict(total_tokens=-1), dict(total_tokens=1 << 29), dict(num_heads=0), dict(num_kv_heads=3), dict(num_kv_heads=0),
               dict(page_size=0), dict(page_size=1 << 30), dict(num_pages=-1), dict(table_cols=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(k_page_stride=16 * 2 * 128 - 8), dict(v_page_stride=16 * 2 * 128 + 4), dict(k_page_stride=1 << 62)):
        assert call(_chunk(**kw)) == BAD, kw
        assert kda.chunk_attention_workspace_bytes(_chunk(**kw)) == 0
    for kw in (dict(dim=96), dict(dtype=5), dict(num_heads=130)):
        assert call(_chunk(**kw)) == UNSUP
    assert lib.kda_chunk_attention(None, *[_p(base[n]) for n in names], 1 << 40, None) == BAD
    need = kda.chunk_attention_workspace_bytes(_chunk())
    assert need > 0
    assert call(nbytes=need - 1) == kda.KDA_ERR_WORKSPACE
    for n in names:
        assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    assert call(out=base["q"]) == BAD
    assert call(out=base["v"] + 16 * 2 * 128 * 2 * 9) == BAD       # inside the last page of the cache
    assert call(nbytes=need, out=base["ws"] + 16) == BAD
    for kw in (dict(batch=0), dict(total_tokens=0)):
        assert call(_chunk(**kw), nbytes=0, q=None, ctx=None, ws=None) == kda.KDA_OK
        assert kda.chunk_attention_workspace_bytes(_chunk(**kw)) == 0


@pytest.mark.parametrize("dtype", [kda.KDA_BF16, kda.KDA_F32])
def test_chunk_attention_refuses_more_work_than_it_counts(lib, dtype):
    """Tables of 2^31 tokens a row: 100 sequences are counted, 2^24 are not."""
    wide = dict(dtype=dtype, page_size=64, table_cols=1 << 25, k_page_stride=64 * 2 * 128, v_page_stride=64 * 2 * 128)
    assert kda.chunk_attention_workspace_bytes(_chunk(batch=100, **wide)) > 0
    d = _chunk(batch=1 << 24, **wide)
    assert kda.chunk_attention_workspace_bytes(d) == 0
    assert lib.kda_chunk_attention(ctypes.byref(d), *[_p(0x10000000 * (i + 1)) for i in range(8)], 1 << 40, None) == UNSUP


def _rotate(**kw):
    d = dict(total_tokens=20, num_heads=8, num_kv_heads=2, dim=128, dtype=kda.KDA_BF16, rot_dim=64, flags=0, num_pages=10, page_size=16, eps=1e-6,
             q_stride=12 * 128, k_stride=12 * 128, v_stride=12 * 128, k_page_stride=16 * 2 * 128, v_page_stride=16 * 2 * 128)
    d.update(kw)
    return kda.NormRotateDesc(*[d[n] for n, _ in kda.NormRotateDesc._fields_])


def test_norm_rotate_refusals(lib):
    names = ("q", "k", "v", "wq", "wk", "freq", "pos", "slots", "out", "kc", "vc")
    base = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}
    call = lambda desc=None, **kw: lib.kda_norm_rotate(ctypes.byref(_rotate() if desc is None else desc), *[_p(kw.get(n, base[n])) for n in names], None)
    for kw in (dict(total_tokens=-1), dict(num_heads=0), dict(num_kv_heads=0), dict(num_pages=-1), dict(page_size=0), dict(rot_dim=-16), dict(rot_dim=144),
               dict(flags=4), dict(flags=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_stride=8 * 128 - 8), dict(k_stride=128),
               dict(v_stride=12 * 128 + 4), dict(q_stride=1 << 62), dict(k_page_stride=16 * 2 * 128 - 8), dict(v_page_stride=16 * 2 * 128 + 1),
               dict(total_tokens=1 << 29), dict(num_heads=1 << 21, total_tokens=1, q_stride=1 << 40)):
        assert call(_rotate(**kw)) == BAD, kw
    for kw in (dict(dim=96), dict(dtype=5), dict(rot_dim=24)):
        assert call(_rotate(**kw)) == UNSUP, kw
    assert lib.kda_norm_rotate(None, *[_p(base[n]) for n in names], None) == BAD
    for n in names:
        if n not in ("wq", "wk"):
            assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    assert call(slots=base["slots"] + 4) == BAD
    assert call(out=base["q"]) == BAD and call(out=base["kc"]) == BAD and call(vc=base["v"]) == BAD and call(kc=base["freq"] - 4096) == BAD
    assert call(_rotate(total_tokens=0), q=None, slots=None) == kda.KDA_OK


def test_page_fork_refusals(lib):
    names = ("par", "chi", "lens", "held", "table", "shares", "free", "out", "copies", "taken")
    base = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    call = lambda n=3, rows=6, cols=8, pages=50, frees=10, ps=16, **kw: lib.kda_page_fork(
        n, rows, cols, pages, frees, ps, *[_p(kw.get(x, base[x])) for x in names], None)
    for kw in (dict(n=-1), dict(n=7), dict(rows=-1), dict(cols=-1), dict(pages=-1), dict(frees=-1), dict(ps=0), dict(rows=16000, cols=1 << 20)):
        assert call(**kw) == BAD, kw
    assert call(rows=kda.KDA_PAGE_TABLES_MAX_BATCH + 1) == UNSUP
    for n in names:
        assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    for n in ("table", "shares", "out", "copies", "taken"):
        for other in names:
            if n != other:
                assert call(**{n: base[other]}) == BAD, (n, other)


def test_page_release_refusals(lib):
    names = ("keep", "held", "table", "shares", "out", "freed", "count")
    base = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    call = lambda rows=6, cols=8, pages=50, ps=16, **kw: lib.kda_page_release(rows, cols, pages, ps, *[_p(kw.get(x, base[x])) for x in names], None)
    for kw in (dict(rows=-1), dict(cols=-1), dict(pages=-1), dict(ps=0), dict(rows=1 << 20, cols=1 << 20)):
        assert call(**kw) == BAD, kw
    for n in names:
        assert call(**{n: None}) == BAD, n
        assert call(**{n: base[n] + 2}) == BAD, n
    for n in ("shares", "out", "freed", "count"):
        for other in names:
            if n != other:
                assert call(**{n: base[other]}) == BAD, (n, other)


def _layers(**kw):
    d = dict(num_layers=2, num_pages=10, page_size=16, num_kv_heads=2, dim=64, dtype=kda.KDA_BF16, k_layer_stride=20 * 2048, v_layer_stride=20 * 2048,
             k_page_stride=2048, v_page_stride=2048)
    d.update(kw)
    return kda.CacheDesc(*[d[n] for n, _ in kda.CacheDesc._fields_])


def test_cache_moves_refusals(lib):
    copy = lambda desc=None, n=3, c=0x1000, k=0x1000000, v=0x2000000: lib.kda_cache_copy(
        ctypes.byref(_layers() if desc is None else desc), n, _p(c), _p(k), _p(v), None)
    base = dict(slots=0x1000, path=0x4000, n=0x8000, k=0x1000000, v=0x2000000)
    keep = lambda desc=None, B=3, K=5, **kw: lib.kda_cache_keep_path(
        ctypes.byref(_layers() if desc is None else desc), B, K, *[_p({**base, **kw}[x]) for x in base], None)
    for call in (copy, keep):
        for kw in (dict(num_layers=-1), dict(num_pages=-1), dict(page_size=0), dict(num_kv_heads=0), dict(dim=0), dict(page_size=1 << 30),
                   dict(k_page_stride=2040), dict(v_page_stride=2052), dict(k_layer_stride=1024), dict(v_layer_stride=20 * 2048 + 4),
                   dict(k_layer_stride=1 << 62), dict(v_page_stride=-2048)):
            assert call(_layers(**kw)) == BAD, kw
        assert call(_layers(dtype=7)) == UNSUP and call(_layers(dim=3, num_kv_heads=1)) == UNSUP
        for x in ("k", "v"):
            assert call(**{x: None}) == BAD and call(**{x: 0x1000008}) == BAD
        assert call(_layers(num_layers=0)) == kda.KDA_OK
    assert copy(n=-1) == BAD and copy(c=None) == BAD and copy(c=0x1002) == BAD and copy(c=0x1000000) == BAD and copy(n=0, c=None) == kda.KDA_OK
    assert copy(n=(1 << 31) - 1, k=1 << 40, v=1 << 41) == UNSUP      # more pieces than a grid has blocks
    for kw in (dict(B=-1), dict(K=0), dict(K=65), dict(B=1 << 25), dict(slots=None), dict(path=None), dict(n=None), dict(slots=0x1004), dict(path=0x4002),
               dict(n=0x8002), dict(slots=0x1000000), dict(path=0x2000000)):
        assert keep(**kw) == BAD, kw
    assert keep(B=0, slots=None) == kda.KDA_OK


# ------------------------------------------------------------------ the binding
def _z(*s, dt=torch.float32):
    return torch.zeros(*s, dtype=dt)


def _calls(**over):
    def arg(name, value):
        return over.get(name, value)

    lens, table = _z(2, dt=I32), _z(2, 2, dt=I32)
    q, k = arg("q", _z(6, 4, 64)), arg("k", _z(6, 2, 64))
    kc, vc = arg("kc", _z(5, 8, 2, 64)), arg("vc", _z(5, 8, 2, 64))
    return {
        "chunk_attention": lambda **kw: kda.chunk_attention(q, kc, vc, arg("table", table), arg("lens", lens), arg("cu", _z(3, dt=I32)), **kw),
        "norm_rotate": lambda **kw: kda.norm_rotate(q, k, arg("v", _z(6, 2, 64)), arg("pos", _z(6, dt=I32)), arg("freq", _z(32)),
                                                    arg("slots", _z(6, dt=I64)), kc, vc, **kw),
        "page_fork": lambda **kw: kda.page_fork(arg("lens", lens), lens, lens, arg("held", _z(4, dt=I32)), arg("table", _z(4, 2, dt=I32)),
                                                arg("shares", _z(9, dt=I32)), _z(3, dt=I32), page_size=8, **kw),
        "page_release": lambda **kw: kda.page_release(lens, arg("held", lens), arg("table", table), arg("shares", _z(9, dt=I32)), page_size=8, **kw),
        "cache_copy": lambda **kw: kda.cache_copy(arg("copies", _z(2, 3, dt=I32)), kc, vc, **kw),
        "cache_keep_path": lambda **kw: kda.cache_keep_path(arg("slots", _z(2, 3, dt=I64)), arg("path", _z(2, 3, dt=I32)), arg("n", lens), kc, vc, **kw),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_tensors_on_the_cpu_are_refused(name):
    with pytest.raises(ValueError, match="CUDA device"):
        _calls()[name]()


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_given_stream_is_looked_at_first(monkeypatch, name):
    """Its handle reaches the call by way of the check of its device only."""
    asked = []
    monkeypatch.setattr(_lib, "_stream_on", lambda stream, device: asked.append((stream, device)) or 0)
    more = {"workspace": _z(64, dt=torch.uint8)} if name == "chunk_attention" else {}
    with pytest.raises(ValueError, match="CUDA device"):
        _calls()[name](stream="one", **more)
    assert asked == [("one", -1)]


WRONG = [("chunk_attention", dict(q=_z(6, 4, 64).half()), TypeError), ("chunk_attention", dict(kc=_z(5, 8, 2, 64).bfloat16()), TypeError),
         ("chunk_attention", dict(cu=_z(2, dt=I32)), ValueError), ("chunk_attention", dict(lens=_z(3, dt=I32)), ValueError),
         ("chunk_attention", dict(table=_z(2, 2)), TypeError), ("chunk_attention", dict(q=_z(4, 6, 64).transpose(0, 1)), ValueError),
         ("chunk_attention", dict(vc=_z(5, 2, 8, 64).transpose(1, 2)), ValueError),
         ("norm_rotate", dict(k=_z(6, 2, 64).bfloat16()), TypeError), ("norm_rotate", dict(v=_z(6, 3, 64)), ValueError),
         ("norm_rotate", dict(q=_z(6, 64, 4).transpose(1, 2)), ValueError), ("norm_rotate", dict(slots=_z(6, dt=I32)), TypeError),
         ("norm_rotate", dict(pos=_z(6, dt=I64)), TypeError), ("norm_rotate", dict(freq=_z(32).double()), TypeError),
         ("page_fork", dict(lens=_z(2, dt=I64)), TypeError), ("page_fork", dict(held=_z(5, dt=I32)), ValueError),
         ("page_fork", dict(table=_z(2, 4, dt=I32).t()), ValueError), ("page_fork", dict(shares=_z(18, dt=I32)[::2]), ValueError),
         ("page_release", dict(held=_z(3, dt=I32)), ValueError), ("page_release", dict(table=_z(2, 2, dt=I64)), TypeError),
         ("cache_copy", dict(copies=_z(2, 2, dt=I32)), ValueError), ("cache_copy", dict(vc=_z(5, 8, 2, 64).bfloat16()), TypeError),
         ("cache_copy", dict(vc=_z(5, 8, 2, 32)), ValueError), ("cache_copy", dict(kc=_z(8, 2, 64)), ValueError),
         ("cache_keep_path", dict(path=_z(2, 4, dt=I32)), ValueError), ("cache_keep_path", dict(slots=_z(2, 3, dt=I32)), TypeError),
         ("cache_keep_path", dict(kc=_z(5, 2, 8, 64).transpose(1, 2)), ValueError)]


@pytest.mark.parametrize("name,over,error", WRONG, ids=[f"{n}-{next(iter(o))}-{i}" for i, (n, o, _) in enumerate(WRONG)])
def test_wrong_tensors_are_refused(name, over, error):
    """Shapes, types and strides that the C calls cannot see."""
    with pytest.raises(error) as e:
        _calls(**over)[name]()
    assert "CUDA device" not in str(e.value)


def test_wrong_arguments_are_refused():
    calls = _calls()
    lens, table, shares = _z(2, dt=I32), _z(2, 2, dt=I32), _z(9, dt=I32)
    for bad, error in ((1 << 40, ValueError), (-1 << 40, ValueError), (1 << 80, ValueError), (2.5, TypeError), (None, TypeError)):
        with pytest.raises(error):
            kda.page_release(lens, lens, table, shares, page_size=bad)
    with pytest.raises(TypeError):
        kda.page_release(None, lens, table, shares, page_size=8)
    with pytest.raises(TypeError):
        kda.cache_copy([[0, 1, 2]], _z(5, 8, 2, 64), _z(5, 8, 2, 64))
    for kw, error in (({"scale": "x"}, TypeError), ({"out": _z(5, 4, 64)}, ValueError), ({"out": _z(6, 4, 64).bfloat16()}, TypeError),
                      ({"workspace": _z(64, 2, dt=torch.uint8)[:, 0]}, ValueError), ({"workspace": 5}, TypeError)):
        with pytest.raises(error) as e:
            calls["chunk_attention"](**kw)
        assert "CUDA device" not in str(e.value)
    for kw, error in (({"eps": None}, TypeError), ({"q_weight": _z(63)}, ValueError), ({"k_weight": _z(64).double()}, TypeError), ({"out": _z(6, 4, 32)}, ValueError)):
        with pytest.raises(error) as e:
            calls["norm_rotate"](**kw)
        assert "CUDA device" not in str(e.value)
