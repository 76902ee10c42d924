"""ctypes binding of the C ABI in ``include/attn.h``.

Argument marshalling only: torch tensors supply device pointers, shapes and
the current CUDA stream; every step of the computation runs in the library's
CUDA kernels. If the library is missing the import fails loudly; there is no
fallback of any kind.
"""

from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

from ._build import CALLS_PATH, LIB_PATH, calls_current

ATTN_OK = 0
ATTN_F32 = 0
ATTN_BF16 = 1

_STATUS_NAMES = {
    0: "ATTN_OK", -1: "ATTN_ERR_INVALID_ARG", -2: "ATTN_ERR_UNSUPPORTED",
    -3: "ATTN_ERR_MISALIGNED", -4: "ATTN_ERR_WORKSPACE", -5: "ATTN_ERR_CUDA",
    -6: "ATTN_ERR_DEVICE_TIMEOUT", -7: "ATTN_ERR_DEVICE_INDEX",
}


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS_NAMES.get(status, status)} "
                         f"({lib().attn_status_string(status).decode()})")


_LIB = None


class AttnMask(ctypes.Structure):
    """The C ``attn_mask``: window (left, right; -1 = unbounded), n_global
    keys visible to every row, optional per-row key ranges [B, Nq] int32."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("n_global", ctypes.c_int), ("row_kv_start", ctypes.c_void_p),
                ("row_kv_end", ctypes.c_void_p)]


class AttnStrides(ctypes.Structure):
    """The C ``attn_strides``: element strides of a [B, H, N, d] tensor."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong),
                ("token", ctypes.c_longlong)]


_SIGNATURES = {
    "attn_fwd": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 6 +
                 [ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "attn_fwd_masked": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 6 +
                        [ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "attn_bwd_masked": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int] * 6 +
                        [ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                         ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd_workspace_size": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "attn_bwd_workspace_size_dt": (ctypes.c_size_t, [ctypes.c_int] * 7),
    "attn_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_uint, ctypes.c_void_p]),
    "attn_bwd": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_int] * 6 +
                 [ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                  ctypes.c_void_p]),
    "attn_decode_workspace_size": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "attn_decode_splitkv": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 5 +
                            [ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_void_p]),
    "attn_decode_paged": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int] * 7 +
                          [ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                           ctypes.c_void_p]),
    "attn_decode_sparse": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int] * 7 +
                           [ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                            ctypes.c_void_p]),
    "attn_merge_partials": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 +
                            [ctypes.c_void_p]),
    "attn_decode_splitkv_noalloc": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 5 +
                                    [ctypes.c_float, ctypes.c_int, ctypes.c_void_p]),
    "attn_rope": (ctypes.c_int, [ctypes.c_void_p] * 9 + [ctypes.c_longlong, ctypes.c_void_p] +
                  [ctypes.c_int] * 7 + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p]),
    "attn_cache_evict": (ctypes.c_int, [ctypes.c_void_p] * 10 + [ctypes.c_int] * 13 +
                         [ctypes.c_void_p]),
    "attn_decode_shared_workspace_size": (ctypes.c_size_t, [ctypes.c_int] * 11),
    "attn_decode_shared": (ctypes.c_int, [ctypes.c_void_p] * 12 + [ctypes.c_int] * 11 +
                           [ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                            ctypes.c_size_t, ctypes.c_void_p]),
    "attn_key_weights_workspace_size": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "attn_key_weights": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_int] * 10 +
                         [ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                          ctypes.c_size_t, ctypes.c_void_p]),
    "attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "attn_sync_status": (ctypes.c_int, [ctypes.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """Load the in-tree library (built by ``__graft_entry__.build()``)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library not built ({LIB_PATH} missing): run "
                "`python -c 'import __graft_entry__ as g; g.build()'` first")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


# ------------------------------------------------------------------ helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return ATTN_F32
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _device_contig(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on the GPU (device pointers)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


_CALLS = None


def _calls():
    """The Python calls of the cache operators (csrc/py_cache.cpp), which check
    their tensors and launch on the tensors' device."""
    global _CALLS
    if _CALLS is None:
        lib()                       # built, and loaded before what links against it
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} missing: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        if not calls_current():
            raise RuntimeError(f"{CALLS_PATH} was built for another Python or torch: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` again")
        spec = importlib.util.spec_from_file_location("_cache_calls", CALLS_PATH)
        calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(calls)
        calls.set_error(AttnError)
        _CALLS = calls
    return _CALLS


def _handle(stream):
    """Handle of a stream; None: the current stream of the call's device."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _allocating_on(stream, t: torch.Tensor):
    """Context for a call that allocates: what it allocates (workspaces above
    all) must belong to the stream it runs on, or the allocator may hand it
    out again while the call still runs."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    return torch.cuda.stream(stream)


def _check(status: int, what: str):
    if status != ATTN_OK:
        raise AttnError(status, what)


# ------------------------------------------------ the C entry points by name

def attn_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None):
    """attn_fwd on torch tensors: q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d], o like q,
    lse [B,Hq,Nq] float32 or None."""
    _device_contig(q, k, v, o, lse)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    st = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                        float(scale), int(bool(causal)), _dt(q), _stream(stream))
    _check(st, "attn_fwd")


def make_mask(window_left=-1, window_right=-1, n_global=0, row_kv_start=None,
              row_kv_end=None) -> AttnMask:
    """An ``attn_mask``; the row ranges are int32 device tensors [B, Nq]
    kept alive by the caller for as long as the call runs."""
    for t in (row_kv_start, row_kv_end):
        if t is not None and (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous()):
            raise ValueError("row ranges must be contiguous int32 device tensors")
    return AttnMask(int(window_left), int(window_right), int(n_global),
                    None if row_kv_start is None else row_kv_start.data_ptr(),
                    None if row_kv_end is None else row_kv_end.data_ptr())


def attn_fwd_masked(q, k, v, o, lse, scale: float, mask, stream=None):
    """attn_fwd under an ``attn_mask`` (``make_mask``; None: no mask)."""
    _device_contig(q, k, v, o, lse)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    m = None if mask is None else ctypes.byref(mask)
    st = lib().attn_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq,
                               Nk, d, float(scale), m, _dt(q), _stream(stream))
    _check(st, "attn_fwd_masked")


def attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, dtype=None) -> int:
    """Workspace bytes of attn_bwd: for ``dtype`` (torch.float32 or
    torch.bfloat16) the exact need, else the largest over dtypes."""
    if dtype is None:
        return int(lib().attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, d))
    dt = ATTN_F32 if dtype == torch.float32 else ATTN_BF16 if dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError(f"unsupported dtype {dtype}: float32 or bfloat16")
    return int(lib().attn_bwd_workspace_size_dt(B, Hq, Hkv, Nq, Nk, d, dt))


def attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace,
             stream=None):
    _device_contig(q, k, v, o, do, lse, dq, dk, dv, workspace)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    st = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                        _ptr(dk), _ptr(dv), B, Hq, Hkv, Nq, Nk, d, float(scale),
                        int(bool(causal)), _dt(q), _ptr(workspace),
                        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "attn_bwd")


def attn_bwd_masked(q, k, v, o, do, lse, dq, dk, dv, scale: float, mask, workspace,
                    stream=None):
    """attn_bwd under an ``attn_mask`` (``make_mask``; None: no mask)."""
    _device_contig(q, k, v, o, do, lse, dq, dk, dv, workspace)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    m = None if mask is None else ctypes.byref(mask)
    st = lib().attn_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), B, Hq, Hkv, Nq, Nk, d, float(scale), m, _dt(q),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    _check(st, "attn_bwd_masked")


def attn_decode_workspace_size(B, Hq, d, num_splits) -> int:
    return int(lib().attn_decode_workspace_size(B, Hq, d, num_splits))


def attn_decode_splitkv(q, k_cache, v_cache, o, lse, scale: float, num_splits: int, workspace,
                        stream=None):
    """q [B,Hq,d], caches [B,Hkv,L,d] bf16; o [B,Hq,d] bf16; lse [B,Hq] or None."""
    _device_contig(q, k_cache, v_cache, o, lse, workspace)
    B, Hq, d = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    st = lib().attn_decode_splitkv(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), B,
                                   Hq, Hkv, L, d, float(scale), int(num_splits), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "attn_decode_splitkv")


def attn_decode_splitkv_noalloc(q, k_cache, v_cache, o, lse, scale: float, num_splits: int,
                                stream=None):
    """Split-KV decode whose partials live in the library's fixed scratch array
    (no workspace argument): for callers that cannot allocate device memory
    when they decode. Same shapes and results as attn_decode_splitkv."""
    _device_contig(q, k_cache, v_cache, o, lse)
    B, Hq, d = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    st = lib().attn_decode_splitkv_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o),
                                           _ptr(lse), B, Hq, Hkv, L, d, float(scale),
                                           int(num_splits), _stream(stream))
    _check(st, "attn_decode_splitkv_noalloc")


def attn_decode_paged(q, k_pages, v_pages, block_table, seq_lens, o, lse, scale: float,
                      num_splits: int, workspace, stream=None):
    """q [B,Hq,d] bf16; pages [num_pages,Hkv,page_size,d] bf16; block_table
    [B,max_pages] and seq_lens [B] int32 on the device; o [B,Hq,d] bf16;
    lse [B,Hq] float32 or None."""
    _device_contig(q, k_pages, v_pages, block_table, seq_lens, o, lse, workspace)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    B, Hq, d = q.shape
    num_pages, Hkv, page_size = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    st = lib().attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                 _ptr(seq_lens), _ptr(o), _ptr(lse), B, Hq, Hkv, num_pages,
                                 page_size, block_table.shape[1], d, float(scale),
                                 int(num_splits), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "attn_decode_paged")


def attn_decode_sparse(q, k_cache, v_cache, indices, counts, o, lse, scale: float,
                       num_splits: int, workspace, stream=None):
    """q [B,Hq,T,d] bf16; caches [B,Hkv,L,d] bf16; indices [B,max_idx] and
    counts [B] int32 on the device; o [B,Hq,T,d] bf16; lse [B,Hq,T] or None."""
    _device_contig(q, k_cache, v_cache, indices, counts, o, lse, workspace)
    if indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise TypeError("indices and counts must be int32")
    B, Hq, T, d = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    st = lib().attn_decode_sparse(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(indices),
                                  _ptr(counts), _ptr(o), _ptr(lse), B, Hq, Hkv, T, L,
                                  indices.shape[1], d, float(scale), int(num_splits),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check(st, "attn_decode_sparse")


def attn_merge_partials(o_part, m_part, l_part, o, lse, stream=None):
    """o_part [rows,S,d], m_part/l_part [rows,S] float32 -> o [rows,d], lse [rows]."""
    _device_contig(o_part, m_part, l_part, o, lse)
    rows, S, d = o_part.shape
    st = lib().attn_merge_partials(_ptr(o_part), _ptr(m_part), _ptr(l_part), _ptr(o), _ptr(lse),
                                   rows, S, d, _dt(o), _stream(stream))
    _check(st, "attn_merge_partials")


def attn_rope(q, k, q_out, k_out, positions, inv_freq, interleaved: bool = False,
              magnitude: float = 1.0, inverse: bool = False, stream=None):
    """attn_rope on torch tensors: q, q_out [B,Hq,N,d] (or [B,Hq,d]: one
    token), k, k_out [B,Hkv,N,d] or None, last dimension contiguous, other
    strides free; positions int32 [B,N] (or [N], [1,N]: shared; [B] with one
    token); inv_freq float64 [rot_dim / 2]."""
    _calls().rope(q, k, positions, inv_freq, interleaved, magnitude, inverse, q_out, k_out,
                  _handle(stream))


def attn_decode_shared_workspace_size(q, k_prefix, prefix_table, k_pages, block_table,
                                      num_prefix_splits: int = 0, num_splits: int = 0) -> int:
    """Workspace bytes of attn_decode_shared for these tensors."""
    B, Hq, d = q.shape
    with torch.cuda.device(q.device):
        return lib().attn_decode_shared_workspace_size(
            B, Hq, k_pages.shape[1], d, prefix_table.shape[0], k_prefix.shape[2],
            prefix_table.shape[1], k_pages.shape[2], block_table.shape[1], num_prefix_splits,
            num_splits)


def attn_decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start, k_pages,
                       v_pages, block_table, seq_lens, o, lse, scale: float,
                       num_prefix_splits: int, num_splits: int, workspace, stream=None):
    """q [B,Hq,d] bf16; k_prefix, v_prefix [num_prefix_pages,Hkv,prefix_page,d]
    bf16 behind prefix_table [n_prefix,max_prefix_pages], prefix_lens
    [n_prefix] and prefix_start [n_prefix+1] int32; own pages, block_table and
    seq_lens as for attn_decode_paged; o like q; lse [B,Hq] float32 or None."""
    _calls().decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start, k_pages,
                           v_pages, block_table, seq_lens, o, lse, scale, num_prefix_splits,
                           num_splits, workspace, False, _handle(stream))


def attn_key_weights_workspace_size(B, Hq, Hkv, T, capacity, out_len) -> int:
    """Workspace bytes of attn_key_weights on the current device (0 while
    T * Hq / Hkv <= 256)."""
    return int(lib().attn_key_weights_workspace_size(B, Hq, Hkv, T, capacity, out_len))


def attn_key_weights(q, k, lse, prev, out, scale: float, decay: float = 1.0, causal: bool = True,
                     seq_lens=None, block_table=None, workspace=None, stream=None):
    """q [B,Hq,T,d] bf16 (or [B,Hq,d]: one token), lse [B,Hq,T] (or [B,Hq])
    float32; k [B,Hkv,L,d] bf16 (or pages [num_pages,Hkv,page_size,d] behind
    block_table [B,max_pages], with seq_lens [B]); prev (None: absent; may be
    out) and out [B,Hkv,out_len] float32."""
    _calls().key_weights(q, k, lse, prev, out, scale, decay, causal, seq_lens, block_table,
                         workspace, False, _handle(stream))


def attn_cache_evict(k, v, scores, k_out, v_out, scores_out, kept, new_lens, n_sink: int = 0,
                     n_recent: int = 0, seq_lens=None, block_table=None, stream=None):
    """k, v [B,Hkv,L,d] (or pages [num_pages,Hkv,page_size,d] behind
    block_table [B,max_pages], with seq_lens [B]); scores [B,Hkv,score_len]
    float32; k_out, v_out [B,Hkv,out_len,d]; scores_out [B,Hkv,out_len] or
    None; kept [B,Hkv,n_keep] and new_lens [B] int32."""
    _calls().evict(k, v, scores, k_out, v_out, scores_out, kept, new_lens, n_sink, n_recent,
                   seq_lens, block_table, _handle(stream))


def attn_status_string(status: int) -> str:
    return lib().attn_status_string(status).decode()


def attn_sync_status(stream=None) -> int:
    return int(lib().attn_sync_status(_stream(stream)))


def attn_selftest_bounded_wait(limit_us: int, stream=None):
    """Launch the bounded-wait self-test (a wait that runs out after
    ``limit_us``); the next attn_sync_status reports the timeout."""
    _check(lib().attn_selftest_bounded_wait(int(limit_us), _stream(stream)),
           "attn_selftest_bounded_wait")


# ------------------------------------------- allocating conveniences (torch)

def forward(q, k, v, causal: bool = False, scale: float | None = None, with_lse: bool = True,
            stream=None, mask: AttnMask | None = None):
    """O, LSE = attention(q, k, v); outputs allocated by torch on q's device.
    ``mask`` (``make_mask``) replaces ``causal`` when given."""
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if with_lse else None
    if mask is not None:
        attn_fwd_masked(q, k, v, o, lse, scale, mask, stream)
    else:
        attn_fwd(q, k, v, o, lse, scale, causal, stream)
    return o, lse


def backward(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None,
             stream=None, mask: AttnMask | None = None):
    """dQ, dK, dV by recomputation from the forward's O and LSE (``mask``, the
    forward's mask, replaces ``causal`` when given)."""
    B, Hq, Nq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    ws = torch.empty(attn_bwd_workspace_size(B, Hq, k.shape[1], Nq, k.shape[2], d, q.dtype),
                     dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if mask is not None:
        attn_bwd_masked(q, k, v, o, do, lse, dq, dk, dv, scale, mask, ws, stream)
    else:
        attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws, stream)
    return dq, dk, dv


def decode(q, k_cache, v_cache, num_splits: int, scale: float | None = None, stream=None,
           workspace=None):
    """Split-KV decode: O [B,Hq,d] bf16 and LSE [B,Hq] float32."""
    B, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(attn_decode_workspace_size(B, Hq, d, num_splits),
                                dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    attn_decode_splitkv(q, k_cache, v_cache, o, lse, scale, num_splits, workspace, stream)
    return o, lse


def decode_paged(q, k_pages, v_pages, block_table, seq_lens, num_splits: int,
                 scale: float | None = None, stream=None, workspace=None):
    """Paged, variable-length split-KV decode: O [B,Hq,d] bf16, LSE [B,Hq] float32."""
    B, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(attn_decode_workspace_size(B, Hq, d, num_splits),
                                dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    attn_decode_paged(q, k_pages, v_pages, block_table, seq_lens, o, lse, scale, num_splits,
                      workspace, stream)
    return o, lse


def decode_sparse(q, k_cache, v_cache, indices, counts, num_splits: int,
                  scale: float | None = None, stream=None, workspace=None):
    """Sparse-index decode of T tokens per request: O [B,Hq,T,d] bf16, LSE [B,Hq,T]."""
    B, Hq, T, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(attn_decode_workspace_size(B, Hq * T, d, num_splits),
                                dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    attn_decode_sparse(q, k_cache, v_cache, indices, counts, o, lse, scale, num_splits, workspace,
                       stream)
    return o, lse


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_length: int = 0, low: float = 1.0,
                     high: float = 32.0, device=None):
    """Rotary frequencies (radians per position) of the rot_dim / 2 pairs,
    float64, for ``rope``: base^(-2i / rot_dim), scaled for a context
    ``factor`` times as long as the trained one by

    "linear"  every frequency divided by ``factor``;
    "base"    the base raised to base * factor^(rot_dim / (rot_dim - 2)), which
              divides the lowest frequency by ``factor`` and keeps the highest;
    "ramp"    pairs that make more than ``high`` turns over ``original_length``
              positions kept, those with fewer than ``low`` divided by
              ``factor``, linearly in between.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not (factor > 0 and base > 0):
        raise ValueError("base and factor must be positive")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError('"base" needs at least two pairs')
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-i / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if original_length <= 0 or not high > low:
            raise ValueError('"ramp" needs original_length > 0 and low < high')
        keep = ((original_length * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}: none, linear, base or ramp")
    return f.to(device) if device is not None else f


def rope(q, k, positions, inv_freq, interleaved: bool = False, magnitude: float = 1.0,
         inverse: bool = False, stream=None, out=None):
    """Rotated q and k (k may be None), contiguous, or written to
    ``out`` = (q_out, k_out), which may be (q, k) themselves. ``inverse``
    turns back: the gradient of the call when given dy and the same
    magnitude. See attn_rope for shapes, rope_frequencies for inv_freq."""
    if out is not None:
        _calls().rope(q, k, positions, inv_freq, interleaved, magnitude, inverse, *out,
                      _handle(stream))
        return out
    if stream is not None:
        with _allocating_on(stream, q):
            return rope(q, k, positions, inv_freq, interleaved, magnitude, inverse)
    return _calls().rope(q, k, positions, inv_freq, interleaved, magnitude, inverse, None, None,
                         None)


def evict(k, v, scores, n_keep: int, n_sink: int = 0, n_recent: int = 0, seq_lens=None,
          block_table=None, stream=None, out=None):
    """Keep n_keep keys per request and KV head by score: k_out, v_out
    [B,Hkv,n_keep,d], scores_out [B,Hkv,n_keep], kept indices [B,Hkv,n_keep]
    and new_lens [B] (or ``out``, those five tensors, of which k_out, v_out and
    scores_out may be longer than n_keep). Rows past a new length are left as
    they were; allocated here they are zero. With block_table =
    arange(B)[:, None] the outputs are a paged cache for decode_paged."""
    if out is None:
        if stream is not None:
            with _allocating_on(stream, k):
                return evict(k, v, scores, n_keep, n_sink, n_recent, seq_lens, block_table)
        B, Hkv = scores.shape[:2]
        out = (k.new_zeros((B, Hkv, n_keep, k.shape[3])), k.new_zeros((B, Hkv, n_keep, k.shape[3])),
               scores.new_zeros((B, Hkv, n_keep)),
               torch.empty((B, Hkv, n_keep), dtype=torch.int32, device=k.device),
               torch.empty((B,), dtype=torch.int32, device=k.device))
    k_out, v_out, scores_out, kept, new_lens = out
    if kept.shape[2] != n_keep:
        raise ValueError("the kept indices must be [B, Hkv, n_keep]")
    attn_cache_evict(k, v, scores, k_out, v_out, scores_out, kept, new_lens, n_sink, n_recent,
                     seq_lens, block_table, stream)
    return out


def decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start, k_pages, v_pages,
                  block_table, seq_lens, num_prefix_splits: int = 0, num_splits: int = 0,
                  scale: float | None = None, stream=None, workspace=None):
    """Decode of requests that share prefixes: O [B,Hq,d] bf16, LSE [B,Hq]
    float32 over each request's prefix keys and its own. Requests
    prefix_start[p] .. prefix_start[p+1]-1 share prefix p. Splits of 0 are
    chosen by the library."""
    if stream is not None:
        with _allocating_on(stream, q):
            return decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start,
                                 k_pages, v_pages, block_table, seq_lens, num_prefix_splits,
                                 num_splits, scale, None, workspace)
    return _calls().decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start,
                                  k_pages, v_pages, block_table, seq_lens, None, None,
                                  q.shape[-1] ** -0.5 if scale is None else scale,
                                  num_prefix_splits, num_splits, workspace, True, None)


def key_weights(q, k, lse, prev=None, decay: float = 1.0, causal: bool = True,
                scale: float | None = None, seq_lens=None, block_table=None, out=None,
                stream=None, workspace=None):
    """Attention weight each cached key received from the last T tokens, in
    float32 [B,Hkv,L] (paged: [B,Hkv,max_pages * page_size]), plus decay *
    prev. ``out`` may be ``prev``; keys past a request's length are left as
    they were (allocated here, they are zero)."""
    if stream is not None:
        with _allocating_on(stream, q):
            return key_weights(q, k, lse, prev, decay, causal, scale, seq_lens, block_table, out,
                               None, workspace)
    return _calls().key_weights(q, k, lse, prev, out,
                                q.shape[-1] ** -0.5 if scale is None else scale, decay, causal,
                                seq_lens, block_table, workspace, True, None)
