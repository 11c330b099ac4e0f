"""What the binding of the draft-step calls refuses before anything reaches a GPU: tensors that are on no
GPU, or on another than the current one (CPU only)."""
import pytest
import torch

import linear_attention_serving_chunkwise_gb300 as kda
from linear_attention_serving_chunkwise_gb300 import _lib
from linear_attention_serving_chunkwise_gb300.build import build

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return kda.load()


def _z(*s, dt=torch.float32):
    return torch.zeros(*s, dtype=dt)


def _calls():
    x, k = _z(2, 3, 4, 64), _z(5, 8, 2, 64)
    lens = _z(2, dt=I32)
    return {
        "page_tables": lambda **kw: kda.page_tables(lens, lens, lens, _z(2, 4, dt=I32), _z(5, dt=I32), page_size=4, max_tokens=3, **kw),
        "tree_attention": lambda **kw: kda.tree_attention(x, k, k, _z(2, 2, dt=I32), lens, _z(2, 3, dt=I32), **kw),
        "tree_decode": lambda **kw: kda.tree_decode(x, x, x, x, _z(2, 3, 4), _z(2, 3, dt=I32), _z(2, 4, 64, 64), **kw),
        "tree_commit": lambda **kw: kda.tree_commit(x, x, x, _z(2, 3, dt=I32), lens, _z(2, 4, 64, 64), **kw),
        "verify_drafts": lambda **kw: kda.verify_drafts(_z(2, 4, 9), _z(2, 3, dt=I32), _z(2, 3, dt=I32), _z(2, 3), _z(2, 9), **kw),
    }


class _Never:
    """Stands in for the library: any call of it is a failure."""

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 64

        def called(*a):
            raise AssertionError(f"{name} was called")
        return called


@pytest.mark.parametrize("name", sorted(_calls()))
def test_tensors_on_the_cpu_are_refused(monkeypatch, name):
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(_lib, "_lib", _Never())
    with pytest.raises(ValueError, match="CUDA device"):
        _calls()[name]()


class _Stream:
    device_index, cuda_stream = 1, 77


def test_the_tensors_gpu_has_to_be_the_current_one(monkeypatch):
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 5)
    assert _lib._stream_on(None, 0) == 5
    with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
        _lib._stream_on(None, 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _lib._stream_on(_Stream(), 0)
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    assert _lib._stream_on(_Stream(), 1) == 77


@pytest.mark.parametrize("name", sorted(_calls()))
def test_every_call_asks_for_its_stream_that_way(monkeypatch, name):
    """With the check taken for passed, the library is reached: no call goes there without it."""
    asked = []
    monkeypatch.setattr(_lib, "_stream_on", lambda stream, device: asked.append((stream, device)) or 0)
    monkeypatch.setattr(_lib, "_lib", _Never())
    with pytest.raises(AssertionError, match=f"kda_{name} was called"):
        _calls()[name]()
    assert asked == [(None, -1)]


def test_a_workspace_with_gaps_is_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_stream_on", lambda stream, device: 0)
    monkeypatch.setattr(_lib, "_lib", _Never())
    with pytest.raises(ValueError, match="workspace"):
        _calls()["tree_attention"](workspace=_z(64, 2, dt=torch.uint8)[:, 0])


@pytest.mark.parametrize("vocab,status", [(kda.KDA_VERIFY_MAX_VOCAB + 1, kda.KDA_ERR_UNSUPPORTED), (2 ** 31 - 1, kda.KDA_ERR_UNSUPPORTED),
                                          (0, kda.KDA_ERR_INVALID_ARG)])
def test_verify_refuses_a_vocabulary_past_its_indexes(lib, vocab, status):
    """The ends of the vocabulary's slices are 32-bit; rows of 2^30 entries are 4 GB each."""
    at = [None if i == 1 else (i + 1) << 40 for i in range(9)]           # no draft
    assert kda.load().kda_verify_drafts(1, 1, vocab, *at, None) == status


@pytest.mark.parametrize("dim,nodes,rows,ctas", [(128, 16, 16, 304), (128, 17, 64, 152), (64, 16, 16, 304), (64, 17, 64, 304)])
def test_fp32_attention_cuts_its_work_for_the_ctas_that_run_at_once(dim, nodes, rows, ctas):
    """The workspace holds a record and two parts for each CTA: two to an SM, one where two do not fit its shared memory."""
    page = 16 * 2 * dim
    desc = kda.make_tree_attention_desc(2, nodes, 2, 2, dim, kda.KDA_F32, 10, 16, 5, 0.1, page, page)
    assert kda.tree_attention_workspace_bytes(desc) == ctas * (16 + 2 * rows * (dim + 2) * 4)
