"""ctypes binding of the KDA C ABI (include/kda.h).

Argument marshalling only: every step of prefill and decode runs in the CUDA
library ``libkda_gb300.so``.  PyTorch supplies device memory and streams.  There
is no fallback: if the library is missing or fails to load, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda_gb300.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = -1
KDA_ERR_UNSUPPORTED = -2
KDA_ERR_WORKSPACE = -3
KDA_ERR_CUDA = -4
KDA_ERR_TIMEOUT = -5
KDA_F32 = 0
KDA_BF16 = 1
KDA_ABI_VERSION = 3
# input prologue bits (include/kda.h): q/k L2 normalisation, g = -5 sigmoid(z), beta = sigmoid(y)
KDA_PROLOGUE_QK_L2NORM = 1
KDA_PROLOGUE_G_LOGITS = 2
KDA_PROLOGUE_BETA_LOGITS = 4
KDA_PROLOGUE_ALL = 7

# Every symbol include/kda.h declares.
EXPORTED = ("kda_abi_version", "kda_status_string", "kda_prefill_workspace_bytes", "kda_prefill_query",
            "kda_prefill", "kda_prefill_gated", "kda_prefill_checkpointed", "kda_prefill_host_workspace_bytes",
            "kda_prefill_host", "kda_prefill_host_static", "kda_decode", "kda_decode_gated", "kda_decode_multi",
            "kda_decode_multi_gated", "kda_state_combine", "kda_last_device_status", "kda_page_tables",
            "kda_tree_attention_workspace_bytes", "kda_tree_attention", "kda_tree_decode", "kda_tree_commit",
            "kda_verify_drafts")
KDA_DECODE_MULTI_MAX_TOKENS = 64
KDA_STATIC_SCRATCH_BYTES = 64 << 20
KDA_TREE_MAX_NODES = 64
KDA_TREE_PAD = -2          # parents entry of an absent node
KDA_PAGE_TABLES_MAX_BATCH = 16384
KDA_VERIFY_MAX_VOCAB = 1 << 30


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class PrefillDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("qkv_dtype", ctypes.c_int32),
                ("prologue", ctypes.c_int32)]


class TreeAttentionDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "nodes", "num_heads", "num_kv_heads", "dim", "dtype", "num_pages",
                                              "page_size", "table_cols")] + \
               [("scale", ctypes.c_float), ("k_page_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64)]


class PrefillPlan(ctypes.Structure):
    _fields_ = [("kernel_launches", ctypes.c_int32), ("tensor_cores", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the CUDA library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"KDA CUDA library not built ({p} missing): run "
                           "`python -m linear_attention_serving_chunkwise_gb300.build`")
    lib = ctypes.CDLL(p)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.kda_abi_version.restype = i32
    lib.kda_abi_version.argtypes = []
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_prefill_workspace_bytes.restype = sz
    lib.kda_prefill_workspace_bytes.argtypes = [ctypes.POINTER(PrefillDesc)]
    lib.kda_prefill_query.restype = ctypes.c_int
    lib.kda_prefill_query.argtypes = [ctypes.POINTER(PrefillDesc), ctypes.POINTER(PrefillPlan)]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = [ctypes.POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_prefill_gated.restype = ctypes.c_int
    lib.kda_prefill_gated.argtypes = [ctypes.POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_prefill_checkpointed.restype = ctypes.c_int
    lib.kda_prefill_checkpointed.argtypes = [ctypes.POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                             i32, i32, vp, vp, sz, vp]
    lib.kda_prefill_host_workspace_bytes.restype = sz
    lib.kda_prefill_host_workspace_bytes.argtypes = [ctypes.POINTER(PrefillDesc), i32]
    lib.kda_prefill_host.restype = ctypes.c_int
    lib.kda_prefill_host.argtypes = [ctypes.POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz,
                                     vp]
    lib.kda_prefill_host_static.restype = ctypes.c_int
    lib.kda_prefill_host_static.argtypes = [ctypes.POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                            vp]
    lib.kda_decode.restype = ctypes.c_int
    lib.kda_decode.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_decode_gated.restype = ctypes.c_int
    lib.kda_decode_gated.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_decode_multi.restype = ctypes.c_int
    lib.kda_decode_multi.argtypes = [i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_decode_multi_gated.restype = ctypes.c_int
    lib.kda_decode_multi_gated.argtypes = [i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           vp]
    lib.kda_state_combine.restype = ctypes.c_int
    lib.kda_state_combine.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp]
    lib.kda_page_tables.restype = ctypes.c_int
    lib.kda_page_tables.argtypes = [i32] * 5 + [vp] * 10
    lib.kda_tree_attention_workspace_bytes.restype = sz
    lib.kda_tree_attention_workspace_bytes.argtypes = [ctypes.POINTER(TreeAttentionDesc)]
    lib.kda_tree_attention.restype = ctypes.c_int
    lib.kda_tree_attention.argtypes = [ctypes.POINTER(TreeAttentionDesc)] + [vp] * 8 + [sz, vp]
    lib.kda_tree_decode.restype = ctypes.c_int
    lib.kda_tree_decode.argtypes = [i32] * 7 + [vp] * 11
    lib.kda_tree_commit.restype = ctypes.c_int
    lib.kda_tree_commit.argtypes = [i32] * 7 + [vp] * 7
    lib.kda_verify_drafts.restype = ctypes.c_int
    lib.kda_verify_drafts.argtypes = [i32] * 3 + [vp] * 10
    lib.kda_last_device_status.restype = ctypes.c_int
    lib.kda_last_device_status.argtypes = [vp]
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("KDA tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() > 0 else None


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _keep_until_done(tensor: torch.Tensor, stream) -> None:
    """A scratch tensor this module allocated on the current stream and the library uses on
    ``stream``: tell the caching allocator, so that the memory is not handed to another
    allocation before that stream's work is done."""
    if stream is not None and stream != torch.cuda.current_stream(tensor.device):
        tensor.record_stream(stream)


def make_desc(num_seqs: int, total_tokens: int, num_heads: int, dk: int, dv: int, qkv_dtype: int,
              prologue: int = 0) -> PrefillDesc:
    return PrefillDesc(int(num_seqs), int(total_tokens), int(num_heads), int(dk), int(dv), int(qkv_dtype),
                       int(prologue))


def prefill_workspace_bytes(desc: PrefillDesc) -> int:
    return int(load().kda_prefill_workspace_bytes(ctypes.byref(desc)))


def prefill_query(desc: PrefillDesc) -> dict:
    """What one kda_prefill call for ``desc`` will launch (host only)."""
    plan = PrefillPlan()
    st = load().kda_prefill_query(ctypes.byref(desc), ctypes.byref(plan))
    if st != KDA_OK:
        raise KDAError(st, "kda_prefill_query")
    return {"kernel_launches": plan.kernel_launches, "tensor_cores": plan.tensor_cores,
            "workspace_bytes": plan.workspace_bytes}


def prefill(q, k, v, g, beta, cu_seqlens=None, init_state=None, out=None, final_state=None, *,
            num_seqs: Optional[int] = None, want_final: bool = True, workspace=None, stream=None, check=True,
            checkpoint_interval: int = 0, checkpoint_slots: int = 0, checkpoints=None, prologue: int = 0,
            gate=None):
    """KDA prefill through ``kda_prefill`` (``kda_prefill_gated`` when ``gate`` is given).

    q, k [T,H,dk], v [T,H,dv] (fp32 or bf16); g [T,H,dk] fp32; beta [T,H] fp32;
    cu_seqlens [N+1] int32 on the device, or None with ``num_seqs`` equal
    sequences (default 1); init_state [N,H,dk,dv] fp32 or None.
    ``out``/``final_state`` are allocated if not given (``final_state`` may be
    ``init_state`` for in-place chaining).  ``prologue``: KDA_PROLOGUE_* bits (q, k, g and
    beta then hold the raw values of the input recipe).  ``gate``: output gate logits
    [T,H,dv] fp32 (out = o * sigmoid(gate)), not combined with checkpoints.  Returns
    (out, final_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (1 if num_seqs is None else int(num_seqs))
    desc = make_desc(N, T, H, dk, dv, _dtype_code(q), prologue)
    if out is None:
        out = torch.empty((T, H, dv), dtype=torch.float32, device=q.device)
        _keep_until_done(out, stream)
    if final_state is None and want_final:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
        _keep_until_done(final_state, stream)
    need = prefill_workspace_bytes(desc)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _keep_until_done(workspace, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if checkpoint_interval:
        if gate is not None:
            raise ValueError("the output gate is not offered with checkpoints")
        if checkpoints is None:
            checkpoints = torch.zeros((N, H, checkpoint_slots, dk, dv), dtype=torch.float32, device=q.device)
            _keep_until_done(checkpoints, stream)
        st = load().kda_prefill_checkpointed(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                             _ptr(cu_seqlens), _ptr(init_state), _ptr(out), _ptr(final_state),
                                             int(checkpoint_interval), int(checkpoint_slots), _ptr(checkpoints),
                                             _ptr(workspace), ws_bytes, _stream_handle(stream))
        if check and st != KDA_OK:
            raise KDAError(st, "kda_prefill_checkpointed")
        return out, final_state, checkpoints
    if gate is not None:
        st = load().kda_prefill_gated(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate),
                                      _ptr(cu_seqlens), _ptr(init_state), _ptr(out), _ptr(final_state),
                                      _ptr(workspace), ws_bytes, _stream_handle(stream))
        if check and st != KDA_OK:
            raise KDAError(st, "kda_prefill_gated")
        return out, final_state
    st = load().kda_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                            _ptr(init_state), _ptr(out), _ptr(final_state), _ptr(workspace), ws_bytes,
                            _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_prefill")
    return out, final_state


def prefill_host_workspace_bytes(desc: PrefillDesc, segment_tokens: int) -> int:
    return int(load().kda_prefill_host_workspace_bytes(ctypes.byref(desc), int(segment_tokens)))


def prefill_host(q, k, v, g, beta, cu_seqlens=None, init_state=None, out=None, final_state=None, *,
                 segment_tokens: int = 1024, num_seqs: Optional[int] = None, want_final: bool = True,
                 workspace=None, stream=None, check=True, device=None, prologue: int = 0):
    """KDA prefill through ``kda_prefill_host``: every tensor is a CPU tensor (pinned for
    the copies to overlap the kernels); ``workspace`` is a CUDA uint8 tensor, allocated if
    not given.  Asynchronous like the other entry points: the results are in ``out`` /
    ``final_state`` once ``stream`` (default: the current stream) has been synchronised.
    Returns (out, final_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (1 if num_seqs is None else int(num_seqs))
    desc = make_desc(N, T, H, dk, dv, _dtype_code(q), prologue)
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((T, H, dv), dtype=torch.float32, pin_memory=pin)
    if final_state is None and want_final:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    if workspace is None:
        need = prefill_host_workspace_bytes(desc, segment_tokens)
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _keep_until_done(workspace, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().kda_prefill_host(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                 _ptr(cu_seqlens), _ptr(init_state), _ptr(out), _ptr(final_state),
                                 int(segment_tokens), ctypes.c_void_p(workspace.data_ptr()), ws_bytes,
                                 _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_prefill_host")
    return out, final_state


def prefill_host_static(q, k, v, g, beta, cu_seqlens=None, init_state=None, out=None, final_state=None, *,
                        segment_tokens: int = 128, num_seqs: Optional[int] = None, want_final: bool = True,
                        stream=None, check=True, prologue: int = 0):
    """``prefill_host`` through ``kda_prefill_host_static``: the device staging is the
    library's own scratch (no workspace, no device allocation).  Returns (out, final_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (1 if num_seqs is None else int(num_seqs))
    desc = make_desc(N, T, H, dk, dv, _dtype_code(q), prologue)
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((T, H, dv), dtype=torch.float32, pin_memory=pin)
    if final_state is None and want_final:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    st = load().kda_prefill_host_static(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                        _ptr(cu_seqlens), _ptr(init_state), _ptr(out), _ptr(final_state),
                                        int(segment_tokens), _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_prefill_host_static")
    return out, final_state


def decode(q, k, v, g, beta, state, out=None, *, stream=None, check=True, prologue: int = 0, gate=None):
    """One KDA decode step through ``kda_decode`` (``kda_decode_gated`` with ``gate``);
    ``state`` [B,H,dk,dv] fp32 is updated in place.

    q, k [B,H,dk], v [B,H,dv] (fp32 or bf16); g [B,H,dk] fp32; beta [B,H] fp32;
    ``prologue``: KDA_PROLOGUE_* bits; ``gate``: output gate logits [B,H,dv] fp32.
    Returns out [B,H,dv] fp32."""
    B, H, dk = q.shape
    dv = v.shape[2]
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
        _keep_until_done(out, stream)
    if gate is not None:
        st = load().kda_decode_gated(B, H, dk, dv, _dtype_code(q), int(prologue), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                     _ptr(beta), _ptr(gate), _ptr(state), _ptr(out), _stream_handle(stream))
        if check and st != KDA_OK:
            raise KDAError(st, "kda_decode_gated")
        return out
    st = load().kda_decode(B, H, dk, dv, _dtype_code(q), int(prologue), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                           _ptr(state), _ptr(out), _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_decode")
    return out


def decode_multi(q, k, v, g, beta, state, out=None, n_apply=None, *, want_out=True, stream=None, check=True,
                 prologue: int = 0, gate=None):
    """K tokens per sequence through ``kda_decode_multi``: q, k [B,K,H,dk], v [B,K,H,dv]
    (fp32 or bf16); g [B,K,H,dk] fp32; beta [B,K,H] fp32; ``state`` [B,H,dk,dv] fp32 is
    replaced by the state after the first ``n_apply[b]`` tokens (int32 [B] on the device;
    None = all K); ``prologue``: KDA_PROLOGUE_* bits.  Returns out [B,K,H,dv] fp32 (None
    when ``want_out`` is False).  ``gate``: output gate logits [B,K,H,dv] fp32 (through
    ``kda_decode_multi_gated``)."""
    B, K, H, dk = q.shape
    dv = v.shape[3]
    if out is None and want_out:
        out = torch.empty((B, K, H, dv), dtype=torch.float32, device=q.device)
        _keep_until_done(out, stream)
    if gate is not None:
        st = load().kda_decode_multi_gated(B, K, H, dk, dv, _dtype_code(q), int(prologue), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(g), _ptr(beta), _ptr(gate), _ptr(n_apply), _ptr(state), _ptr(out),
                                           _stream_handle(stream))
        if check and st != KDA_OK:
            raise KDAError(st, "kda_decode_multi_gated")
        return out
    st = load().kda_decode_multi(B, K, H, dk, dv, _dtype_code(q), int(prologue), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(beta),
                                 _ptr(n_apply), _ptr(state), _ptr(out), _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_decode_multi")
    return out


def state_combine(transition, state_in, state_add, out=None, *, stream=None, check=True):
    """out = transition @ state_in + state_add per (sequence, head), through
    ``kda_state_combine``: transition [..., dk, dk], states [..., dk, dv] fp32 on the device
    (state_in or state_add may be None = zero; ``out`` may be ``state_add``).  Returns out."""
    ref = state_add if state_add is not None else state_in
    dk, dv = ref.shape[-2], ref.shape[-1]
    count = ref.numel() // (dk * dv)
    if out is None:
        out = torch.empty_like(ref)
        _keep_until_done(out, stream)
    st = load().kda_state_combine(count, dk, dv, _ptr(transition), _ptr(state_in), _ptr(state_add), _ptr(out),
                                  _stream_handle(stream))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_state_combine")
    return out


# ---- the draft step (include/kda.h) -----------------------------------------------------
# These calls take a few microseconds on the GPU, so the marshalling is kept lean: pointers go
# to ctypes as plain integers and the stream comes as its raw handle (outputs are allocations of
# their own: a view of a fresh tensor costs three times an allocation).
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _stream_on(stream, device: int) -> int:
    """Handle of the stream for tensors on ``device``, which has to be the GPU that the library will use: the current one."""
    if device < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if device != _current_device():
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{_current_device()}")
    if stream is None:
        return _raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _expect(name: str, t: torch.Tensor, dtype, shape, device: int) -> int:
    """Address of ``t``.  The C calls know pointers only: a wrong type, shape, layout, or device other than
    the others' is found here, a device that is not the current GPU by ``_stream_on``, before anything is launched."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the device of the other tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _fresh(shape, dtype, device, stream) -> torch.Tensor:
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        _keep_until_done(t, stream)
    return t


def page_tables(context_lens, new_lens, pages_held, block_table, free_pages, *, page_size: int, max_tokens: int,
                stream=None, check=True):
    """Pages and slots for the tokens a step appends to a paged cache, through ``kda_page_tables``:
    context_lens, new_lens, pages_held [B] int32; block_table [B, cols] int32, updated in place;
    free_pages [F] int32, taken from index 0 on; ``max_tokens``: length of the slot map (>= the sum
    of new_lens).  Returns (slot_map [max_tokens] int64, cu_seqlens [B+1] int32, pages_held after
    the call [B] int32, pages_taken [1] int32)."""
    dev, (B, cols) = block_table.device, block_table.shape
    at, F = block_table.get_device(), free_pages.numel()
    ctx = _expect("context_lens", context_lens, _I32, (B,), at)
    new = _expect("new_lens", new_lens, _I32, (B,), at)
    had = _expect("pages_held", pages_held, _I32, (B,), at)
    table = _expect("block_table", block_table, _I32, (B, cols), at)
    free = _expect("free_pages", free_pages, _I32, (F,), at)
    queue = _stream_on(stream, at)
    slots = _fresh((max_tokens,), torch.int64, dev, stream)
    cu, held, taken = _fresh((B + 1,), _I32, dev, stream), _fresh((B,), _I32, dev, stream), _fresh((1,), _I32, dev, stream)
    st = load().kda_page_tables(B, cols, F, page_size, max_tokens, ctx, new, had, table, free, slots.data_ptr(),
                                cu.data_ptr(), held.data_ptr(), taken.data_ptr(), queue)
    if check and st != KDA_OK:
        raise KDAError(st, "kda_page_tables")
    return slots, cu, held, taken


def _cache(name: str, c: torch.Tensor, dtype, shape, device: int):
    """(address, elements from page to page) of a cache [pages, page_size, heads, dim] whose pages are contiguous."""
    if c.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {c.dtype}")
    if c.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(c.shape)}")
    if c.get_device() != device:
        raise ValueError(f"{name} is on {c.device}, not on the device of the other tensors")
    P, ps, h, d = shape
    stride = c.stride()
    if stride[1:] != (h * d, d, 1) and P > 0 and not c[0].is_contiguous():
        raise ValueError(f"{name}: each page must be contiguous")
    return c.data_ptr(), stride[0] if P > 1 else ps * h * d


def make_tree_attention_desc(batch, nodes, num_heads, num_kv_heads, dim, dtype, num_pages, page_size, table_cols,
                             scale, k_page_stride, v_page_stride) -> TreeAttentionDesc:
    return TreeAttentionDesc(batch, nodes, num_heads, num_kv_heads, dim, dtype, num_pages, page_size, table_cols,
                             scale, k_page_stride, v_page_stride)


def tree_attention_workspace_bytes(desc: TreeAttentionDesc) -> int:
    return int(load().kda_tree_attention_workspace_bytes(ctypes.byref(desc)))


def tree_attention(q, k_cache, v_cache, block_table, context_lens, parents, out=None, *, scale: Optional[float] = None,
                   workspace=None, stream=None, check=True):
    """Attention of draft trees over a paged cache, through ``kda_tree_attention``.

    q [B,K,Hq,D] (fp32 or bf16); k_cache, v_cache [pages, page_size, Hk, D] of q's type, each page
    contiguous (the pages themselves may be strided, as in views of one [pages, 2, ...] tensor);
    block_table [B, cols] int32; context_lens [B] int32; parents [B,K] int32; ``scale`` defaults
    to 1 / sqrt(D).  Node j's key and value lie at logical position context_lens + j.  ``workspace``:
    uint8 scratch of ``tree_attention_workspace_bytes``, allocated if not given.  Returns out
    [B,K,Hq,D] of q's type."""
    B, K, H, D = q.shape
    P, ps, Hk, _ = k_cache.shape
    dt, dev, at = q.dtype, q.device, q.get_device()
    code = _dtype_code(q)
    qp = _expect("q", q, dt, (B, K, H, D), at)
    kp, ks = _cache("k_cache", k_cache, dt, (P, ps, Hk, D), at)
    vp, vs = _cache("v_cache", v_cache, dt, (P, ps, Hk, D), at)
    cols = block_table.shape[-1]
    table = _expect("block_table", block_table, _I32, (B, cols), at)
    ctx = _expect("context_lens", context_lens, _I32, (B,), at)
    par = _expect("parents", parents, _I32, (B, K), at)
    queue = _stream_on(stream, at)
    desc = ctypes.byref(TreeAttentionDesc(B, K, H, Hk, D, code, P, ps, cols, D ** -0.5 if scale is None else scale, ks, vs))
    if out is None:
        out = _fresh((B, K, H, D), dt, dev, stream)
        op = out.data_ptr()
    else:
        op = _expect("out", out, dt, (B, K, H, D), at)
    lib = load()
    if workspace is None:
        workspace = _fresh((lib.kda_tree_attention_workspace_bytes(desc),), torch.uint8, dev, stream)
    elif workspace.get_device() != at or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    st = lib.kda_tree_attention(desc, qp, kp, vp, table, ctx, par, op, workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), queue)
    if check and st != KDA_OK:
        raise KDAError(st, "kda_tree_attention")
    return out


def tree_decode(q, k, v, g, beta, parents, state, out=None, writes=None, *, stream=None, check=True,
                prologue: int = 0, gate=None):
    """KDA for every node of draft trees through ``kda_tree_decode``: q, k [B,K,H,dk], v
    [B,K,H,dv] (fp32 or bf16); g [B,K,H,dk], beta [B,K,H] fp32; parents [B,K] int32; ``state``
    [B,H,dk,dv] fp32 is only read; ``prologue``: KDA_PROLOGUE_* bits; ``gate``: output gate logits
    [B,K,H,dv] fp32.  Returns (out, writes), both [B,K,H,dv] fp32; ``tree_commit`` takes writes.  A sequence
    whose tree is bad (``last_device_status``) is skipped: its rows are not written, so in tensors allocated here
    they are undefined."""
    B, K, H, dk = q.shape
    dv, dt, dev, at = v.shape[3], q.dtype, q.device, q.get_device()
    code = _dtype_code(q)
    wide = (B, K, H, dv)
    ins = (_expect("q", q, dt, (B, K, H, dk), at), _expect("k", k, dt, (B, K, H, dk), at), _expect("v", v, dt, wide, at),
           _expect("g", g, _F32, (B, K, H, dk), at), _expect("beta", beta, _F32, (B, K, H), at),
           _expect("parents", parents, _I32, (B, K), at), None if gate is None else _expect("gate", gate, _F32, wide, at),
           _expect("state", state, _F32, (B, H, dk, dv), at))
    queue = _stream_on(stream, at)
    if out is None:
        out = _fresh(wide, _F32, dev, stream)
    if writes is None:
        writes = _fresh(wide, _F32, dev, stream)
    st = load().kda_tree_decode(B, K, H, dk, dv, code, prologue, *ins, _expect("out", out, _F32, wide, at),
                                _expect("writes", writes, _F32, wide, at), queue)
    if check and st != KDA_OK:
        raise KDAError(st, "kda_tree_decode")
    return out, writes


def tree_commit(k, g, writes, path, n_accept, state, *, stream=None, check=True, prologue: int = 0):
    """``state`` [B,H,dk,dv] fp32 moved in place to the end of each accepted path, through
    ``kda_tree_commit``: k, g and ``prologue`` as given to ``tree_decode``, ``writes`` as it returned
    them; path [B,K] and n_accept [B] int32 as ``verify_drafts`` returns them.  Returns state."""
    B, K, H, dk = k.shape
    dv, at = state.shape[3], k.get_device()
    st = load().kda_tree_commit(B, K, H, dk, dv, _dtype_code(k), prologue, _expect("k", k, k.dtype, (B, K, H, dk), at),
                                _expect("g", g, _F32, (B, K, H, dk), at), _expect("writes", writes, _F32, (B, K, H, dv), at),
                                _expect("path", path, _I32, (B, K), at), _expect("n_accept", n_accept, _I32, (B,), at),
                                _expect("state", state, _F32, (B, H, dk, dv), at), _stream_on(stream, at))
    if check and st != KDA_OK:
        raise KDAError(st, "kda_tree_commit")
    return state


def verify_drafts(target_probs, tokens, parents, uniforms, noise, draft_probs=None, *, stream=None, check=True):
    """Which drafted tokens are kept and what follows them, through ``kda_verify_drafts``:
    target_probs [B,K+1,V] fp32 (row 0 after the context, row i+1 after node i); tokens, parents
    [B,K] int32; uniforms [B,K] fp32 in [0, 1); noise [B,V] fp32 ~ Exp(1); ``draft_probs``
    [B,K,V] fp32 for chains drawn from a draft model, None for drafts picked by any other rule.
    Returns (path [B,K] int32 with -1 after the kept nodes, n_accept [B] int32, next_token [B]
    int32)."""
    B, K1, V = target_probs.shape
    K, dev, at = K1 - 1, target_probs.device, target_probs.get_device()
    target = _expect("target_probs", target_probs, _F32, (B, K1, V), at)
    tok = _expect("tokens", tokens, _I32, (B, K), at)
    par = _expect("parents", parents, _I32, (B, K), at)
    uni = _expect("uniforms", uniforms, _F32, (B, K), at)
    noi = _expect("noise", noise, _F32, (B, V), at)
    dra = None if draft_probs is None else _expect("draft_probs", draft_probs, _F32, (B, K, V), at)
    queue = _stream_on(stream, at)
    path = _fresh((B, K), _I32, dev, stream)
    n_accept, next_token = _fresh((B,), _I32, dev, stream), _fresh((B,), _I32, dev, stream)
    st = load().kda_verify_drafts(B, K, V, target, dra, tok, par, uni, noi, path.data_ptr(), n_accept.data_ptr(),
                                  next_token.data_ptr(), queue)
    if check and st != KDA_OK:
        raise KDAError(st, "kda_verify_drafts")
    return path, n_accept, next_token


def last_device_status(stream=None) -> int:
    return int(load().kda_last_device_status(_stream_handle(stream)))
