"""Thin ctypes binding of ``libhs2.so`` (include/hs2.h) over torch tensors.

Argument marshalling only: torch provides device memory and the current
stream; every step of the Hybrid-Block path runs in the library's CUDA
kernels.  If the library is missing or fails to load, every call raises --
there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhs2.so")

HS2_F32, HS2_BF16, HS2_E4M3 = 0, 1, 2
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(6)

_DTYPE = {torch.float32: HS2_F32, torch.bfloat16: HS2_BF16, torch.uint8: HS2_E4M3,
          torch.float8_e4m3fn: HS2_E4M3}


class Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_slots", ctypes.c_int64)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Tokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("token_stride", ctypes.c_int64)]


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_context", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("low_freq_factor", ctypes.c_double),
                ("high_freq_factor", ctypes.c_double)]


class HS2Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"hs2 error {code}: {msg}")
        self.code = code


_lib = None
EXPORTS = ["hs2_full_attn_select_workspace", "hs2_full_attn_select", "hs2_full_attn_select_marked",
           "hs2_full_attn_select_blocks", "hs2_full_attn_select_fused",
           "hs2_full_attn_select_static", "hs2_full_attn_select_static_status", "hs2_selftest_bounded_wait_static",
           "hs2_sparse_attn",
           "hs2_workspace_status", "hs2_selftest_bounded_wait", "hs2_selftest_grid_barrier",
           "hs2_kv_bridge_workspace", "hs2_kv_bridge_append",
           "hs2_rope_table", "hs2_rope_append", "hs2_tree_attn_workspace", "hs2_tree_attn", "hs2_tree_accept",
           "hs2_full_attn_accumulate", "hs2_full_attn_accumulate_each", "hs2_cache_evict",
           "hs2_copy_peak", "hs2_last_error", "hs2_version"]


def lib():
    """The loaded library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m long_context_decode_full_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.hs2_full_attn_select_workspace.argtypes = [I32, I32, I32, I32, I64]
        L.hs2_full_attn_select_workspace.restype = SZ
        L.hs2_full_attn_select.argtypes = [ctypes.POINTER(Heads), ctypes.POINTER(Cache), ctypes.POINTER(Cache),
                                           P, P, I32, I32, I32, ctypes.POINTER(Heads), P, P, SZ, P]
        L.hs2_full_attn_select.restype = ctypes.c_int
        L.hs2_full_attn_select_marked.argtypes = L.hs2_full_attn_select.argtypes + [P]
        L.hs2_full_attn_select_marked.restype = ctypes.c_int
        L.hs2_full_attn_select_fused.argtypes = L.hs2_full_attn_select.argtypes
        L.hs2_full_attn_select_fused.restype = ctypes.c_int
        L.hs2_full_attn_select_blocks.argtypes = [ctypes.POINTER(Heads), ctypes.POINTER(Cache), ctypes.POINTER(Cache),
                                                  P, P, I32, I32, I32, I32, ctypes.POINTER(Heads), P, P, SZ, P]
        L.hs2_full_attn_select_blocks.restype = ctypes.c_int
        L.hs2_full_attn_select_static.argtypes = [ctypes.POINTER(Heads), ctypes.POINTER(Cache),
                                                  ctypes.POINTER(Cache), P, P, I32, I32, I32,
                                                  ctypes.POINTER(Heads), P, P]
        L.hs2_full_attn_select_static.restype = ctypes.c_int
        L.hs2_full_attn_select_static_status.argtypes = [P]
        L.hs2_full_attn_select_static_status.restype = ctypes.c_int
        L.hs2_selftest_bounded_wait_static.argtypes = [P]
        L.hs2_selftest_bounded_wait_static.restype = ctypes.c_int
        L.hs2_sparse_attn.argtypes = [ctypes.POINTER(Heads), ctypes.POINTER(Cache), ctypes.POINTER(Cache), P, I32,
                                      ctypes.POINTER(Heads), P]
        L.hs2_sparse_attn.restype = ctypes.c_int
        L.hs2_workspace_status.argtypes = [P, SZ, P]
        L.hs2_workspace_status.restype = ctypes.c_int
        L.hs2_kv_bridge_workspace.argtypes = [I32, I32, I32, I32]
        L.hs2_kv_bridge_workspace.restype = SZ
        L.hs2_kv_bridge_append.argtypes = [P, I32, I32, P, P, P, P, I32, ctypes.POINTER(Cache),
                                           ctypes.POINTER(Cache), P, SZ, P]
        L.hs2_kv_bridge_append.restype = ctypes.c_int
        T, C, F = ctypes.POINTER(Tokens), ctypes.POINTER(Cache), ctypes.c_float
        L.hs2_rope_table.argtypes = [ctypes.POINTER(Rope), P, ctypes.POINTER(F)]
        L.hs2_rope_table.restype = ctypes.c_int
        L.hs2_rope_append.argtypes = [T, T, T, P, P, I32, I32, F, P, P, P, I32, C, C, P, P]
        L.hs2_rope_append.restype = ctypes.c_int
        L.hs2_tree_attn_workspace.argtypes = [I32, I32, I32, I32, I32, I32]
        L.hs2_tree_attn_workspace.restype = SZ
        L.hs2_tree_attn.argtypes = [T, C, C, P, P, P, P, I32, T, P, SZ, P]
        L.hs2_tree_attn.restype = ctypes.c_int
        L.hs2_tree_accept.argtypes = [C, C, P, P, P, P, I32, I32, P, I32, P, P]
        L.hs2_tree_accept.restype = ctypes.c_int
        L.hs2_full_attn_accumulate.argtypes = [ctypes.POINTER(Heads), C, C, P, P, I32, F, I32, P, I64,
                                               ctypes.POINTER(Heads), P, SZ, P]
        L.hs2_full_attn_accumulate.restype = ctypes.c_int
        L.hs2_full_attn_accumulate_each.argtypes = [ctypes.POINTER(Heads), C, C, P, P, I32, F, P, P, I64,
                                                    ctypes.POINTER(Heads), P, SZ, P]
        L.hs2_full_attn_accumulate_each.restype = ctypes.c_int
        L.hs2_cache_evict.argtypes = [C, C, P, I32, P, I32, P, I64, I32, I32, P, P, P]
        L.hs2_cache_evict.restype = ctypes.c_int
        L.hs2_selftest_bounded_wait.argtypes = [P, SZ, P]
        L.hs2_selftest_bounded_wait.restype = ctypes.c_int
        L.hs2_selftest_grid_barrier.argtypes = [P, SZ, P]
        L.hs2_selftest_grid_barrier.restype = ctypes.c_int
        L.hs2_copy_peak.argtypes = [P, P, SZ, P]
        L.hs2_copy_peak.restype = ctypes.c_int
        L.hs2_last_error.argtypes = []
        L.hs2_last_error.restype = ctypes.c_char_p
        L.hs2_version.argtypes = []
        L.hs2_version.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int):
    if rc != OK:
        raise HS2Error(rc, lib().hs2_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(name, t, dtypes, dim=None, shape=None):
    """The C ABI takes bare pointers: check what they cannot carry (element
    type, rank, shape, contiguity, a CUDA device) before the call."""
    if t is None:
        return
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t.dtype not in dtypes:
        raise HS2Error(ERR_INVALID_ARG, f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if dim is not None and t.dim() != dim:
        raise HS2Error(ERR_INVALID_ARG, f"{name}: {t.dim()} dimensions, expected {dim}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise HS2Error(ERR_INVALID_ARG, f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise HS2Error(ERR_INVALID_ARG, f"{name}: not contiguous")


def _need_cuda(**tensors):
    """Checked after every element type and shape, so a type error is
    reported as such whatever the device."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise HS2Error(ERR_INVALID_ARG, f"{name}: not on a CUDA device")


def _need_lens(seq_lens, page_table, B):
    _need("seq_lens", seq_lens, torch.int32, shape=(B,))
    if page_table is not None:
        _need("page_table", page_table, torch.int32, dim=2)
        if page_table.shape[0] != B:
            raise HS2Error(ERR_INVALID_ARG, f"page_table: {page_table.shape[0]} rows for batch {B}")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Where a call makes the results and workspaces that it is not given: on the stream that it runs on, so that their
    fills come before its kernels and their memory is used again only behind them.  As with tensors made under
    torch.cuda.stream(), a result used on another stream is ordered by the caller."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def cache_desc(kv: torch.Tensor, scale: Optional[torch.Tensor], page_size: int) -> Cache:
    assert kv.dim() == 3 and kv.is_contiguous(), "cache must be a contiguous [num_slots, Hkv, d] tensor"
    return Cache(kv.data_ptr(), None if scale is None else scale.data_ptr(), _DTYPE[kv.dtype], kv.shape[1],
                 kv.shape[2], page_size, kv.shape[0])


def heads_desc(x: torch.Tensor) -> Heads:
    assert x.dim() == 3 and x.is_contiguous(), "q/out must be a contiguous [B, H, d] tensor"
    return Heads(x.data_ptr(), _DTYPE[x.dtype], x.shape[0], x.shape[1], x.shape[2])


def full_workspace_bytes(batch: int, num_kv_heads: int, group: int, head_dim: int, t_cap: int) -> int:
    return int(lib().hs2_full_attn_select_workspace(batch, num_kv_heads, group, head_dim, t_cap))


def alloc_workspace(batch, num_kv_heads, group, head_dim, t_cap, device="cuda") -> torch.Tensor:
    n = full_workspace_bytes(batch, num_kv_heads, group, head_dim, t_cap)
    if n == 0:
        raise HS2Error(ERR_INVALID_ARG, "invalid workspace shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def full_attn_select(q, k, v, seq_lens, page_table=None, page_size=None, window=128, k_global=1024,
                     k_scale=None, v_scale=None, out=None, idx_out=None, workspace=None, stream=None,
                     mark_event=None, fused=False):
    """Full-attention layer + token selection.  Returns (out, idx) where idx
    holds selected slots [B, Hkv, window + k_global], ascending, -1 padded.
    ``mark_event`` (a recorded-once torch.cuda.Event) is recorded between the
    attention kernel and the selection kernels.  ``fused`` runs the attention
    and the selection's score pass in one cooperative persistent kernel
    (hs2_full_attn_select_fused; no mark event)."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    _need_lens(seq_lens, page_table, B)
    _need("idx_out", idx_out, torch.int32, shape=(B, Hkv, window + k_global))
    _need_cuda(q=q, k=k, v=v, seq_lens=seq_lens, page_table=page_table, idx_out=idx_out)
    if page_size is None:
        assert page_table is None, "page_size is required with a page table"
        page_size = k.shape[0] // B
    max_pages = 1 if page_table is None else page_table.shape[1]
    t_cap = page_size * max_pages
    with _on(stream):
        if out is None:
            out = torch.empty_like(q)
        if idx_out is None:
            idx_out = torch.empty(B, Hkv, window + k_global, dtype=torch.int32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(B, Hkv, Hq // Hkv, d, t_cap, q.device)
    kc, vc = cache_desc(k, k_scale, page_size), cache_desc(v, v_scale, page_size)
    qd, od = heads_desc(q), heads_desc(out)
    if fused:
        assert mark_event is None, "the fused call records no mark event"
        _check(lib().hs2_full_attn_select_fused(ctypes.byref(qd), ctypes.byref(kc), ctypes.byref(vc),
                                                _ptr(seq_lens), _ptr(page_table), max_pages, window, k_global,
                                                ctypes.byref(od), _ptr(idx_out), _ptr(workspace), workspace.numel(),
                                                _stream(stream)))
        return out, idx_out
    ev = None if mark_event is None else ctypes.c_void_p(mark_event.cuda_event)
    _check(lib().hs2_full_attn_select_marked(ctypes.byref(qd), ctypes.byref(kc), ctypes.byref(vc),
                                             _ptr(seq_lens), _ptr(page_table), max_pages, window, k_global,
                                             ctypes.byref(od), _ptr(idx_out), _ptr(workspace), workspace.numel(),
                                             _stream(stream), ev))
    return out, idx_out


def full_attn_select_blocks(q, k, v, seq_lens, page_table=None, page_size=None, window=128, k_global=1024,
                            block=16, k_scale=None, v_scale=None, out=None, idx_out=None, workspace=None,
                            stream=None):
    """Full-attention layer + BLOCK-level selection (the first-generation
    comparator): the same attention output, and idx [B, Hkv, window + k_global]
    with the slots of the k_global / block best blocks' positions and the
    window, ascending, -1 padded."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    _need_lens(seq_lens, page_table, B)
    _need("idx_out", idx_out, torch.int32, shape=(B, Hkv, window + k_global))
    _need_cuda(q=q, k=k, v=v, seq_lens=seq_lens, page_table=page_table, idx_out=idx_out)
    if page_size is None:
        assert page_table is None, "page_size is required with a page table"
        page_size = k.shape[0] // B
    max_pages = 1 if page_table is None else page_table.shape[1]
    with _on(stream):
        if out is None:
            out = torch.empty_like(q)
        if idx_out is None:
            idx_out = torch.empty(B, Hkv, window + k_global, dtype=torch.int32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(B, Hkv, Hq // Hkv, d, page_size * max_pages, q.device)
    kc, vc = cache_desc(k, k_scale, page_size), cache_desc(v, v_scale, page_size)
    qd, od = heads_desc(q), heads_desc(out)
    _check(lib().hs2_full_attn_select_blocks(ctypes.byref(qd), ctypes.byref(kc), ctypes.byref(vc), _ptr(seq_lens),
                                             _ptr(page_table), max_pages, window, k_global, block, ctypes.byref(od),
                                             _ptr(idx_out), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out, idx_out


def full_attn_select_static(q, k, v, seq_lens, page_table=None, page_size=None, window=128, k_global=1024,
                            k_scale=None, v_scale=None, out=None, idx_out=None, stream=None):
    """full_attn_select() without a workspace: the library's own fixed 32 MiB
    device scratch is used (for callers that may not allocate).  Calls that
    overlap on the GPU race on that scratch; static_status() reports an
    expired device wait of these calls."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    _need_lens(seq_lens, page_table, B)
    _need("idx_out", idx_out, torch.int32, shape=(B, Hkv, window + k_global))
    _need_cuda(q=q, k=k, v=v, seq_lens=seq_lens, page_table=page_table, idx_out=idx_out)
    if page_size is None:
        assert page_table is None, "page_size is required with a page table"
        page_size = k.shape[0] // B
    max_pages = 1 if page_table is None else page_table.shape[1]
    with _on(stream):
        if out is None:
            out = torch.empty_like(q)
        if idx_out is None:
            idx_out = torch.empty(B, Hkv, window + k_global, dtype=torch.int32, device=q.device)
    kc, vc = cache_desc(k, k_scale, page_size), cache_desc(v, v_scale, page_size)
    qd, od = heads_desc(q), heads_desc(out)
    _check(lib().hs2_full_attn_select_static(ctypes.byref(qd), ctypes.byref(kc), ctypes.byref(vc),
                                             _ptr(seq_lens), _ptr(page_table), max_pages, window, k_global,
                                             ctypes.byref(od), _ptr(idx_out), _stream(stream)))
    return out, idx_out


def static_status(stream=None) -> int:
    """Synchronises the stream, returns and clears the sticky device error flag
    of full_attn_select_static() calls in the current CUDA context."""
    return int(lib().hs2_full_attn_select_static_status(_stream(stream)))


def sparse_attn(q_l, k, v, idx, k_scale=None, v_scale=None, page_size=1, out=None, stream=None):
    """Sparse-attention layer over the rows listed in ``idx`` (slots)."""
    _need("idx", idx, torch.int32, dim=3)
    _need_cuda(q=q_l, k=k, v=v, idx=idx)
    if out is None:
        with _on(stream):
            out = torch.empty_like(q_l)
    kc, vc = cache_desc(k, k_scale, page_size), cache_desc(v, v_scale, page_size)
    qd, od = heads_desc(q_l), heads_desc(out)
    _check(lib().hs2_sparse_attn(ctypes.byref(qd), ctypes.byref(kc), ctypes.byref(vc), _ptr(idx), idx.shape[-1],
                                 ctypes.byref(od), _stream(stream)))
    return out


def hybrid_block_step(q_full, q_sparse: Sequence[torch.Tensor], k, v, seq_lens, page_table=None, page_size=None,
                      window=128, k_global=1024, k_scale=None, v_scale=None, outs=None, idx_out=None,
                      workspace=None, stream=None, fused=False):
    """One decode step of a Hybrid Block: the full layer (attention + token
    selection) then every sparse layer with its own query, all reusing the
    same cache and the same index list.  Returns (outs, idx).  ``fused``
    selects the fused full-layer call (see full_attn_select)."""
    outs = outs if outs is not None else [None] * (1 + len(q_sparse))
    o0, idx = full_attn_select(q_full, k, v, seq_lens, page_table, page_size, window, k_global, k_scale, v_scale,
                               outs[0], idx_out, workspace, stream, fused=fused)
    ps = page_size if page_size is not None else k.shape[0] // q_full.shape[0]
    res = [o0]
    for i, q in enumerate(q_sparse):
        res.append(sparse_attn(q, k, v, idx, k_scale, v_scale, ps, outs[1 + i], stream))
    return res, idx


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronises the stream, returns and clears the sticky device error flag."""
    return int(lib().hs2_workspace_status(_ptr(workspace), workspace.numel(), _stream(stream)))


def kv_bridge_workspace_bytes(batch: int, d_model: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().hs2_kv_bridge_workspace(batch, d_model, num_kv_heads, head_dim))


def kv_bridge_append(hidden, w_k, w_v, k, v, seq_lens, page_table=None, page_size=None, k_scale=None, v_scale=None,
                     workspace=None, stream=None):
    """KV Bridging append: writes the new token's K/V rows (hidden [B, d_model]
    bf16 times w_k / w_v [d_model, Hkv * d] bf16) at position seq_lens[b] - 1
    of the caches k / v (and the E4M3 scales).  A workspace passed in must
    have been zero-filled once (see kv_bridge_workspace_bytes)."""
    _need("hidden", hidden, torch.bfloat16, dim=2)
    B, dm = hidden.shape
    if k.dim() != 3:
        raise HS2Error(ERR_INVALID_ARG, "k: expected a [num_slots, Hkv, d] cache")
    N = k.shape[1] * k.shape[2]
    _need("w_k", w_k, torch.bfloat16, shape=(dm, N))
    _need("w_v", w_v, torch.bfloat16, shape=(dm, N))
    _need_lens(seq_lens, page_table, B)
    _need("k_scale", k_scale, torch.float32, shape=k.shape[:2])
    _need("v_scale", v_scale, torch.float32, shape=v.shape[:2])
    _need_cuda(hidden=hidden, w_k=w_k, w_v=w_v, k=k, v=v, seq_lens=seq_lens, page_table=page_table,
               k_scale=k_scale, v_scale=v_scale)
    if page_size is None:
        assert page_table is None, "page_size is required with a page table"
        page_size = k.shape[0] // B
    max_pages = 1 if page_table is None else page_table.shape[1]
    if workspace is None:
        n = kv_bridge_workspace_bytes(B, dm, k.shape[1], k.shape[2])
        if n == 0:
            raise HS2Error(ERR_INVALID_ARG, "invalid KV bridge shape")
        with _on(stream):
            workspace = torch.zeros(n, dtype=torch.uint8, device=hidden.device)
    kc, vc = cache_desc(k, k_scale, page_size), cache_desc(v, v_scale, page_size)
    _check(lib().hs2_kv_bridge_append(_ptr(hidden), B, dm, _ptr(w_k), _ptr(w_v), _ptr(seq_lens), _ptr(page_table),
                                      max_pages, ctypes.byref(kc), ctypes.byref(vc), _ptr(workspace),
                                      workspace.numel(), _stream(stream)))


# ---------------------------------------------------------------- drafted tokens, bounded caches
# These calls run on the device that holds the cache, whichever is current, on
# its current stream unless one is given.  A decode step makes several of them,
# so their checks are written to cost a microsecond or two.
_ROPE_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class RopeTable(NamedTuple):
    """Turns per position of each rotated pair (hs2_rope_table), on the device."""
    turns: torch.Tensor  # int64 [rot_dim / 2], the bits of the C table
    rot_dim: int
    interleaved: bool
    scale: float


def rope_table(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: Optional[str] = None,
               factor: float = 1.0, original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
               low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, device="cuda") -> RopeTable:
    """The frequencies of rope_append(): ``rot_dim`` first elements of a head turn, in pairs (e, e + rot_dim / 2) or,
    ``interleaved``, (2e, 2e + 1).  ``scaling``: None, "linear", "ntk", "yarn" or "bands" (see HS2_ROPE_* in hs2.h).
    Built on the host and copied once."""
    if scaling not in _ROPE_SCALING:
        raise HS2Error(ERR_INVALID_ARG, f"scaling {scaling!r}, expected one of {sorted(map(str, _ROPE_SCALING))}")
    r = Rope(rot_dim, _ROPE_SCALING[scaling], base, factor, original_context, beta_fast, beta_slow, low_freq_factor,
             high_freq_factor)
    turns = torch.empty(64, dtype=torch.int64)
    scale = ctypes.c_float()
    _check(lib().hs2_rope_table(ctypes.byref(r), _ptr(turns), ctypes.byref(scale)))
    return RopeTable(turns[:rot_dim // 2].to(device), rot_dim, bool(interleaved), scale.value)


def _arg(name, t, dtype, shape):
    """The pointer of an optional contiguous array, checked."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _need(name, t, dtype, shape=shape)
    return t.data_ptr()


def _paged(k, v, k_scale, v_scale, page_table, page_size, B):
    """Checked cache descriptors, the page table's pointer and max_pages."""
    kd, vd, shape, v_shape = _DTYPE.get(k.dtype), _DTYPE.get(v.dtype), k.shape, v.shape
    if kd is None or vd is None:
        raise HS2Error(ERR_INVALID_ARG, f"k, v: dtype {k.dtype}, {v.dtype} is no cache type")
    if len(shape) != 3 or len(v_shape) != 3 or not k.is_contiguous() or not v.is_contiguous():
        raise HS2Error(ERR_INVALID_ARG, "k, v: expected contiguous [num_slots, Hkv, d] caches")
    pages, max_pages = None, 1
    if page_table is not None:
        if page_size is None:
            raise HS2Error(ERR_INVALID_ARG, "page_size is required with a page table")
        max_pages = page_table.shape[1] if page_table.dim() == 2 else 0
        pages = _arg("page_table", page_table, torch.int32, (B, max_pages))
    elif page_size is None:
        page_size = shape[0] // max(B, 1)
    ks = None if k_scale is None else _arg("k_scale", k_scale, torch.float32, shape[:2])
    vs = None if v_scale is None else _arg("v_scale", v_scale, torch.float32, v_shape[:2])
    return (Cache(k.data_ptr(), ks, kd, shape[1], shape[2], page_size, shape[0]),
            Cache(v.data_ptr(), vs, vd, v_shape[1], v_shape[2], page_size, v_shape[0]), pages, max_pages)


def _tokens(name, x, dtype) -> Tokens:
    """[B, N, H, d], the heads of a token side by side and its tokens evenly spaced (a slice of a fused projection)."""
    if x.dtype is not dtype:
        raise HS2Error(ERR_INVALID_ARG, f"{name}: dtype {x.dtype}, expected {dtype}")
    if x.dim() != 4:
        raise HS2Error(ERR_INVALID_ARG, f"{name}: {x.dim()} dimensions, expected [B, N, H, d]")
    B, N, H, d = x.shape
    sb, sn, sh, sd = x.stride()
    stride = sn if N > 1 else (sb if B > 1 else H * d)
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (B > 1 and N > 1 and sb != N * sn):
        raise HS2Error(ERR_INVALID_ARG, f"{name}: strides {x.stride()}, expected heads and tokens in order")
    return Tokens(x.data_ptr(), _DTYPE[dtype], B, N, H, d, stride)


def _device(names, k, *tensors) -> int:
    """The CUDA device of the cache, on which every tensor has to be."""
    i = k.get_device()
    if i < 0:
        raise HS2Error(ERR_INVALID_ARG, "k: not on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != i:
            name = next(n for n, x in zip(names, tensors) if x is t)
            raise HS2Error(ERR_INVALID_ARG, f"{name}: on {t.device}, the cache on {k.device}")
    return i


def _run(call, device, stream, *args):
    """``call(*args, stream)`` on `device`, on its current stream unless one is given."""
    if device == _current_device():
        rc = call(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = call(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    if rc != OK:
        _check(rc)


_current_device, _raw_stream = torch.cuda.current_device, getattr(
    torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_ROPE_NAMES = ("v", "q", "k_new", "v_new", "positions", "table", "seq_lens", "num_new", "page_table", "k_scale", "v_scale", "q_out")
_TREE_NAMES = ("v", "q", "out", "tree_mask", "seq_lens", "num_draft", "page_table", "k_scale", "v_scale", "workspace")
_ACCEPT_NAMES = ("v", "seq_lens", "path", "path_len", "num_draft", "page_table", "k_scale", "v_scale", "lens_out")
_ACCUMULATE_NAMES = ("v", "q", "seq_lens", "acc", "fresh", "page_table", "k_scale", "v_scale", "out", "workspace")
_EVICT_NAMES = ("v", "seq_lens", "acc", "page_table", "k_scale", "v_scale", "kept", "lens_out")


def _q_dtype(k):
    return torch.float32 if k.dtype == torch.float32 else torch.bfloat16


def rope_append(q, k_new, v_new, positions, table: RopeTable, k, v, seq_lens, page_table=None, page_size=None,
                num_new=None, k_scale=None, v_scale=None, q_out=None, stream=None):
    """Rotary positions on new tokens and the append of their K/V rows: q [B, N, Hq, d] (or None), k_new and v_new
    [B, N, Hkv, d] -- contiguous, or parts of a fused projection -- at int32 ``positions`` [B, N]; the rows go to
    positions seq_lens[b] - num_new[b] + i of the caches k / v.  Returns the rotated queries (q_out; rows of tokens
    that a sequence does not have are left as they are)."""
    kt, vt = _tokens("k_new", k_new, _q_dtype(k)), _tokens("v_new", v_new, _q_dtype(k))
    B, N = kt.batch, kt.tokens
    qt = None
    if q is not None:
        qt = _tokens("q", q, _q_dtype(k))
        if q_out is None:
            with _on(stream):
                q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        _arg("q_out", q_out, q.dtype, q.shape)
    pp, lp = _arg("positions", positions, torch.int32, (B, N)), _arg("seq_lens", seq_lens, torch.int32, (B,))
    np_ = _arg("num_new", num_new, torch.int32, (B,))
    kc, vc, pages, max_pages = _paged(k, v, k_scale, v_scale, page_table, page_size, B)
    device = _device(_ROPE_NAMES, k, v, q, k_new, v_new, positions, table.turns, seq_lens, num_new, page_table, k_scale, v_scale,
                     q_out)
    _run((_lib or lib()).hs2_rope_append, device, stream, qt, kt, vt, pp, table.turns.data_ptr(), table.rot_dim, table.interleaved,
         table.scale, lp, np_, pages, max_pages, kc, vc, None if q_out is None else q_out.data_ptr())
    return q_out


def tree_mask(parents) -> torch.Tensor:
    """int64 [B, N] masks for tree_attn() from parents [B, N] (CPU), N <= 64: parents[b, i] < i is the draft that token i
    continues, -1 for the context; each token sees its ancestors and itself."""
    parents = torch.as_tensor(parents)
    if parents.dim() != 2 or parents.shape[1] > 64:
        raise HS2Error(ERR_UNSUPPORTED, f"parents: shape {tuple(parents.shape)}, expected [B, N] with N of at most 64")
    rows = []
    for row in parents.tolist():
        m = []
        for i, p in enumerate(row):
            if not -1 <= p < i:
                raise HS2Error(ERR_INVALID_ARG, f"parents: draft {i} continues {p}")
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        rows.append([x - (1 << 64) if x >> 63 else x for x in m])
    return torch.tensor(rows, dtype=torch.int64)


def tree_workspace_bytes(batch: int, tokens: int, num_kv_heads: int, group: int, head_dim: int, kv_dtype: int) -> int:
    return int(lib().hs2_tree_attn_workspace(batch, tokens, num_kv_heads, group, head_dim, kv_dtype))


def alloc_tree_workspace(q, k) -> torch.Tensor:
    """A workspace for tree_attn() of queries like q [B, N, Hq, d] over caches like k, or of fewer sequences or tokens."""
    B, N, Hq, d = q.shape
    with torch.cuda.device(k.device):
        n = tree_workspace_bytes(B, N, k.shape[1], Hq // k.shape[1], d, _DTYPE[k.dtype])
    if n == 0:
        raise HS2Error(ERR_INVALID_ARG, "invalid workspace shape")
    workspace = torch.empty(n, dtype=torch.uint8, device=k.device)
    workspace[:256].zero_()  # the sticky error flag
    return workspace


def tree_attn(q, k, v, seq_lens, page_table=None, page_size=None, tree_mask=None, num_draft=None, k_scale=None,
              v_scale=None, out=None, workspace=None, stream=None):
    """Attention of drafted tokens q [B, N, Hq, d] (N <= 64), whose K/V rows are the last num_draft[b] of the
    seq_lens[b] rows: each sees the context and the drafts j with bit j of its int64 ``tree_mask`` [B, N] (None: a
    chain).  Rows of tokens that a sequence does not have are left as they are in ``out``."""
    qt = _tokens("q", q, _q_dtype(k))
    B, N = qt.batch, qt.tokens
    if out is None:
        with _on(stream):
            out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    ot = _tokens("out", out, q.dtype)
    mp, lp = _arg("tree_mask", tree_mask, torch.int64, (B, N)), _arg("seq_lens", seq_lens, torch.int32, (B,))
    np_ = _arg("num_draft", num_draft, torch.int32, (B,))
    kc, vc, pages, max_pages = _paged(k, v, k_scale, v_scale, page_table, page_size, B)
    device = _device(_TREE_NAMES, k, v, q, out, tree_mask, seq_lens, num_draft, page_table, k_scale, v_scale, workspace)
    if workspace is None:
        with _on(stream):
            workspace = alloc_tree_workspace(q, k)
    _need("workspace", workspace, torch.uint8)
    _run(lib().hs2_tree_attn, device, stream, qt, kc, vc, lp, np_, mp, pages, max_pages, ot, workspace.data_ptr(),
         workspace.numel())
    return out


def tree_accept(k, v, seq_lens, path, path_len, page_table=None, page_size=None, num_draft=None, k_scale=None,
                v_scale=None, lens_out=None, stream=None):
    """After a verification: the rows of the accepted drafts path[b, :path_len[b]] move to the front of the draft, whose
    size is num_draft[b] (None: the width of ``path``, so a path narrower than the draft needs it).  Returns the new
    lengths."""
    if path.dim() != 2:
        _need("path", path, torch.int32, dim=2)
    B, M = path.shape
    pp, one = _arg("path", path, torch.int32, (B, M)), (B,)
    lp, ap = _arg("seq_lens", seq_lens, torch.int32, one), _arg("path_len", path_len, torch.int32, one)
    np_ = _arg("num_draft", num_draft, torch.int32, one)
    kc, vc, pages, max_pages = _paged(k, v, k_scale, v_scale, page_table, page_size, B)
    if lens_out is None:
        with _on(stream):
            lens_out = torch.empty_like(seq_lens)
    op = _arg("lens_out", lens_out, torch.int32, one)
    device = _device(_ACCEPT_NAMES, k, v, seq_lens, path, path_len, num_draft, page_table, k_scale, v_scale, lens_out)
    _run((_lib or lib()).hs2_tree_accept, device, stream, kc, vc, lp, np_, pp, ap, B, M, pages, max_pages, op)
    return lens_out


def _sums(acc, B, Hkv):
    """Row length and pointer of running sums [B, Hkv, capacity]."""
    _need("acc", acc, torch.float32, dim=3)
    if acc.shape[:2] != (B, Hkv):
        raise HS2Error(ERR_INVALID_ARG, f"acc: shape {tuple(acc.shape)}, expected ({B}, {Hkv}, capacity)")
    return acc.shape[2], acc.data_ptr()


def full_attn_accumulate(q, k, v, seq_lens, acc, page_table=None, page_size=None, decay=1.0, fresh=1, k_scale=None,
                         v_scale=None, out=None, workspace=None, stream=None):
    """The full layer's attention, its weights added to the running sums acc [B, Hkv, >= capacity] (fp32):
    acc = decay * acc + weights, the newest ``fresh`` positions starting anew: as many as each sequence gained since the
    last call, a number for all or int32 [B] (after tree_accept(), its path_len).  Returns (out, acc)."""
    _need("q", q, _q_dtype(k), dim=3)
    B, Hq, d = q.shape
    lp = _arg("seq_lens", seq_lens, torch.int32, (B,))
    kc, vc, pages, max_pages = _paged(k, v, k_scale, v_scale, page_table, page_size, B)
    cap, sums = _sums(acc, B, k.shape[1])
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    _arg("out", out, q.dtype, q.shape)
    each = fresh if torch.is_tensor(fresh) else None
    call, new = lib().hs2_full_attn_accumulate, fresh
    if each is not None:
        call, new = lib().hs2_full_attn_accumulate_each, _arg("fresh", each, torch.int32, (B,))
    device = _device(_ACCUMULATE_NAMES, k, v, q, seq_lens, acc, each, page_table, k_scale, v_scale, out, workspace)
    if workspace is None:
        with torch.cuda.device(device), _on(stream):
            workspace = alloc_workspace(B, k.shape[1], Hq // k.shape[1], d, kc.page_size * max_pages, k.device)
    _need("workspace", workspace, torch.uint8)
    _run(call, device, stream, heads_desc(q), kc, vc, lp, pages, max_pages, decay, new, sums, cap,
         heads_desc(out), workspace.data_ptr(), workspace.numel())
    return out, acc


def cache_evict(k, v, seq_lens, acc, budget, window=None, page_table=None, page_size=None, k_scale=None, v_scale=None,
                kept=None, lens_out=None, stream=None):
    """Where a sequence is longer than ``budget``, every kv head keeps its newest ``window`` tokens (None: 128, or the
    whole of a smaller budget) and the budget - window others with the largest sums in acc [B, Hkv, >= capacity]; their
    rows, scales and sums move to the front, in order and in place.  Returns (lens_out [B], kept [B, Hkv, budget]: the
    kept positions, -1 padded)."""
    _need("seq_lens", seq_lens, torch.int32, dim=1)
    B, lp = seq_lens.shape[0], seq_lens.data_ptr()
    kc, vc, pages, max_pages = _paged(k, v, k_scale, v_scale, page_table, page_size, B)
    Hkv = k.shape[1]
    cap, sums = _sums(acc, B, Hkv)
    if window is None:
        window = min(128, budget)
    with _on(stream):
        if kept is None:
            kept = torch.empty(B, Hkv, max(budget, 0), dtype=torch.int32, device=k.device)
        if lens_out is None:
            lens_out = torch.empty_like(seq_lens)
    kp, op = _arg("kept", kept, torch.int32, (B, Hkv, budget)), _arg("lens_out", lens_out, torch.int32, (B,))
    device = _device(_EVICT_NAMES, k, v, seq_lens, acc, page_table, k_scale, v_scale, kept, lens_out)
    _run(lib().hs2_cache_evict, device, stream, kc, vc, lp, B, pages, max_pages, sums, cap, budget, window, kp, op)
    return lens_out, kept


def selftest_bounded_wait(workspace: torch.Tensor, stream=None):
    """Makes one bounded device wait expire on purpose (it sets the sticky flag)."""
    _check(lib().hs2_selftest_bounded_wait(_ptr(workspace), workspace.numel(), _stream(stream)))


def selftest_grid_barrier(workspace: torch.Tensor, stream=None):
    """Makes the fused call's grid barrier expire on purpose (two CTAs wait for
    a third that never comes; it sets the sticky flag)."""
    _check(lib().hs2_selftest_grid_barrier(_ptr(workspace), workspace.numel(), _stream(stream)))


def copy_peak(dst: torch.Tensor, src: torch.Tensor, stream=None):
    _check(lib().hs2_copy_peak(_ptr(dst), _ptr(src), src.numel() * src.element_size(), _stream(stream)))


def version() -> int:
    return int(lib().hs2_version())


def last_error() -> str:
    return lib().hs2_last_error().decode()
