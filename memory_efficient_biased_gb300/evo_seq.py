"""ctypes binding of the causal-sequence operators (include/evo_seq.h): argument
marshalling only, like ``evo_attn``.

``evo_prompt_fwd`` / ``evo_prompt_bwd``: attention over packed prompts and its
gradients (differentiable as ``autograd.prompt_attention``);
``evo_cache_append`` / ``evo_paged_fwd`` / ``evo_cache_evict``: a paged cache, the
attention of new tokens over it, and its eviction by accumulated attention weight.
The header states what each computes, its layouts and its limits.

Tensors live on the current CUDA device.  With ``stream`` the call, and what it
allocates, belong to that stream; a tensor made on another stream has to be
synchronised with it by the caller, and kept alive, as for any other use.
Token rows ([tokens, heads, head_dim] tensors) may be strided views whose heads
are packed, such as the parts of one fused projection; anything else is refused
with ValueError.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import evo_attn as E
from .evo_attn import EVO_OK, EvoAttnError, _DTYPE_CODE, _check, _on_current_device, _ptr, _stream_ptr

STRIDE_FIELDS = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


class SeqShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "seqs", "q_heads", "kv_heads", "head_dim")]


class SeqStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in STRIDE_FIELDS]


class CacheShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "pages_per_seq", "k_page_stride",
                                               "v_page_stride")]


class SeqOptions(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_uint32), ("wait_limit_ns", ctypes.c_uint64), ("status", ctypes.c_void_p)]


_bound = None


def load():
    """The library of ``evo_attn``, with this module's entry points declared."""
    global _bound
    if _bound is not None:
        return _bound
    lib = E.load()
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    strides, opts = ctypes.POINTER(SeqStrides), ctypes.POINTER(SeqOptions)
    tail = [i32, strides, opts, vp]
    for name, res, args in (
            ("evo_prompt_fwd_workspace_bytes", sz, [SeqShape]),
            ("evo_prompt_bwd_workspace_bytes", sz, [SeqShape]),
            ("evo_paged_fwd_workspace_bytes", sz, [SeqShape, CacheShape, i64]),
            ("evo_prompt_fwd", i32, [vp] * 7 + [sz, SeqShape] + tail),
            ("evo_prompt_bwd", i32, [vp] * 11 + [sz, SeqShape] + tail),
            ("evo_cache_append", i32, [vp] * 7 + [SeqShape, CacheShape] + tail),
            ("evo_paged_fwd", i32, [vp] * 9 + [i64, vp, sz, SeqShape, CacheShape] + tail),
            ("evo_cache_evict", i32, [vp] * 5 + [i64, vp, i64, i64, SeqShape, CacheShape, i32, opts, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _bound = lib
    return lib


def _options(scale, wait_limit_ns, status):
    if scale is None and not wait_limit_ns and status is None:
        return None
    if status is not None:
        _check(status, "status", dtype=torch.int32)
        if status.numel() < 1:
            raise ValueError("status must have an element")
    if scale is not None and not (0.0 < scale < float("inf")):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    o = SeqOptions(ctypes.sizeof(SeqOptions), 0, scale or 0.0, 0, int(wait_limit_ns),
                   None if status is None else status.data_ptr())
    return ctypes.byref(o)


def _rows(t: torch.Tensor, name: str, shape, dtype) -> int:
    """Checks a [tokens, heads, head_dim] tensor; its token stride (0 = packed)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    _on_current_device(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    tokens, heads, d = shape
    if (d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name} must have packed (heads, head_dim) dimensions")
    stride = t.stride(0)
    if tokens <= 1 or stride == heads * d:
        return 0
    if stride < heads * d or stride % 8:
        raise ValueError(f"{name} has token stride {stride}: at least {heads * d} and a multiple of 8 is needed")
    return stride


def _ints(t: torch.Tensor, name: str, shape):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    _check(t, name, shape, torch.int32)


def _heads(q: torch.Tensor, k_heads: int, d: int, name: str = "q"):
    if q.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("inputs must be float16 or bfloat16")
    if q.shape[2] != d or k_heads < 1 or q.shape[1] % k_heads:
        raise ValueError(f"{name} has {q.shape[1]} heads of {q.shape[2]}, the keys {k_heads} of {d}")


def _offsets(cu: torch.Tensor) -> int:
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor [seqs + 1]")
    _ints(cu, "cu_seqlens", cu.shape)
    return cu.shape[0] - 1


def _cache(k_pages, v_pages, block_table, dtype) -> CacheShape:
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{n} must be [num_pages, page_size, kv_heads, head_dim]")
        _on_current_device(t, n)
        if t.dtype != dtype:
            raise ValueError(f"{n} has dtype {t.dtype}, expected {dtype}")
        if t.shape != k_pages.shape:
            raise ValueError(f"{n} has shape {tuple(t.shape)}, expected {tuple(k_pages.shape)}")
        if t.numel() and not t[0].is_contiguous():
            raise ValueError(f"{n} must have contiguous pages")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [seqs, pages_per_seq]")
    _ints(block_table, "block_table", block_table.shape)
    pages, page = k_pages.shape[:2]
    strides = [t.stride(0) if pages > 1 else 0 for t in (k_pages, v_pages)]
    return CacheShape(pages, page, block_table.shape[1], *strides)


class _On:
    """Allocations of a call go to the stream it runs on."""

    def __init__(self, stream):
        self.ctx = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *a):
        if self.ctx is not None:
            self.ctx.__exit__(*a)


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _check(workspace, "workspace")
    return workspace


def _done(st: int, where: str):
    if st != EVO_OK:
        raise EvoAttnError(st, where)


def _nbytes(t):
    return t.numel() * t.element_size()


def evo_prompt_fwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim) -> int:
    return int(load().evo_prompt_fwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim)))


def evo_prompt_bwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim) -> int:
    return int(load().evo_prompt_bwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim)))


def evo_prompt_fwd(q, k, v, cu_seqlens, out=None, lse=None, workspace=None, stream=None, *,
                   scale: Optional[float] = None, wait_limit_ns: int = 0, status: Optional[torch.Tensor] = None):
    """Causal attention within each of the packed sequences; (out [T,Hq,D], lse [Hq,T] fp32).
    Rows in no sequence keep what out and lse held (new ones are uninitialised there)."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, head_dim]")
    _heads(q, k.shape[1], k.shape[2])
    T, Hq, D = q.shape
    Hk, dt = k.shape[1], q.dtype
    B = _offsets(cu_seqlens)
    sq, sk, sv = _rows(q, "q", q.shape, dt), _rows(k, "k", (T, Hk, D), dt), _rows(v, "v", (T, Hk, D), dt)
    shape, lib = SeqShape(T, B, Hq, Hk, D), load()
    sp = _stream_ptr(stream)
    opts = _options(scale, wait_limit_ns, status)
    with _On(stream):
        if out is None:
            out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        ws = _workspace(workspace, lib.evo_prompt_fwd_workspace_bytes(shape), q.device)
    strides = SeqStrides(q=sq, k=sk, v=sv, out=_rows(out, "out", q.shape, dt))
    _check(lse, "lse", (Hq, T), torch.float32)
    _done(lib.evo_prompt_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(out), _ptr(lse), _ptr(ws), _nbytes(ws),
                             shape, _DTYPE_CODE[dt], ctypes.byref(strides), opts, sp), "evo_prompt_fwd")
    return out, lse


def evo_prompt_bwd(q, k, v, cu_seqlens, out, lse, dout, dq=None, dk=None, dv=None, workspace=None, stream=None, *,
                   scale: Optional[float] = None, wait_limit_ns: int = 0, status: Optional[torch.Tensor] = None):
    """Gradients of evo_prompt_fwd from its inputs and outputs; (dq, dk, dv).  Rows in no
    sequence keep what dq, dk and dv held (new ones are uninitialised there)."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, head_dim]")
    _heads(q, k.shape[1], k.shape[2])
    T, Hq, D = q.shape
    Hk, dt = k.shape[1], q.dtype
    B = _offsets(cu_seqlens)
    keys = torch.Size((T, Hk, D))
    strides = SeqStrides(q=_rows(q, "q", q.shape, dt), k=_rows(k, "k", keys, dt), v=_rows(v, "v", keys, dt),
                         out=_rows(out, "out", q.shape, dt), dout=_rows(dout, "dout", q.shape, dt))
    _check(lse, "lse", (Hq, T), torch.float32)
    shape, lib = SeqShape(T, B, Hq, Hk, D), load()
    sp = _stream_ptr(stream)
    opts = _options(scale, wait_limit_ns, status)
    with _On(stream):
        if dq is None:
            dq = torch.empty((T, Hq, D), dtype=dt, device=q.device)
        if dk is None:
            dk = torch.empty(keys, dtype=dt, device=q.device)
        if dv is None:
            dv = torch.empty(keys, dtype=dt, device=q.device)
        ws = _workspace(workspace, lib.evo_prompt_bwd_workspace_bytes(shape), q.device)
    strides.dq, strides.dk, strides.dv = (_rows(dq, "dq", q.shape, dt), _rows(dk, "dk", keys, dt),
                                          _rows(dv, "dv", keys, dt))
    _done(lib.evo_prompt_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                             _ptr(dk), _ptr(dv), _ptr(ws), _nbytes(ws), shape, _DTYPE_CODE[dt], ctypes.byref(strides),
                             opts, sp), "evo_prompt_bwd")
    return dq, dk, dv


def evo_cache_append(k, v, cu_seqlens, seq_lens, k_pages, v_pages, block_table, stream=None, *,
                     status: Optional[torch.Tensor] = None):
    """Writes the new tokens' rows k, v [T,Hkv,D] into the cache: sequence b's are the last
    of its seq_lens[b] (which counts them already)."""
    if k.dim() != 3 or k.dtype not in _DTYPE_CODE:
        raise ValueError("k must be a float16 or bfloat16 tensor [tokens, heads, head_dim]")
    T, Hk, D = k.shape
    dt, B = k.dtype, _offsets(cu_seqlens)
    cache = _cache(k_pages, v_pages, block_table, dt)
    if tuple(k_pages.shape[2:]) != (Hk, D):
        raise ValueError(f"k has {Hk} heads of {D}, the cache {tuple(k_pages.shape[2:])}")
    if block_table.shape[0] != B:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, expected {B}")
    _ints(seq_lens, "seq_lens", (B,))
    strides = SeqStrides(k=_rows(k, "k", k.shape, dt), v=_rows(v, "v", k.shape, dt))
    sp = _stream_ptr(stream)
    _done(load().evo_cache_append(_ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(seq_lens), _ptr(block_table), _ptr(k_pages),
                                  _ptr(v_pages), SeqShape(T, B, Hk, Hk, D), cache, _DTYPE_CODE[dt],
                                  ctypes.byref(strides), _options(None, 0, status), sp), "evo_cache_append")


def evo_paged_fwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim, num_pages, page_size,
                                  pages_per_seq, weights_len=0) -> int:
    return int(load().evo_paged_fwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim),
                                                    CacheShape(num_pages, page_size, pages_per_seq, 0, 0),
                                                    weights_len))


def evo_paged_fwd(q, k_pages, v_pages, cu_seqlens, seq_lens, block_table, out=None, lse=None, weights=None,
                  workspace=None, stream=None, *, scale: Optional[float] = None, wait_limit_ns: int = 0,
                  status: Optional[torch.Tensor] = None):
    """Attention of the new tokens q [T,Hq,D] over the cache that already holds them;
    (out, lse [Hq,T] fp32).  ``weights`` [B,Hkv,n] fp32, where given, gains for every key the
    attention weight that this call's rows gave it."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, page_size, kv_heads, head_dim]")
    Hk = k_pages.shape[2]
    _heads(q, Hk, k_pages.shape[3])
    T, Hq, D = q.shape
    dt, B = q.dtype, _offsets(cu_seqlens)
    cache = _cache(k_pages, v_pages, block_table, dt)
    if block_table.shape[0] != B:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, expected {B}")
    _ints(seq_lens, "seq_lens", (B,))
    sq = _rows(q, "q", q.shape, dt)
    wlen = 0
    if weights is not None:
        if weights.dim() != 3:
            raise ValueError("weights must be [seqs, kv_heads, n]")
        wlen = weights.shape[2]
        _check(weights, "weights", (B, Hk, wlen), torch.float32)
    shape, lib = SeqShape(T, B, Hq, Hk, D), load()
    sp = _stream_ptr(stream)
    opts = _options(scale, wait_limit_ns, status)
    with _On(stream):
        if out is None:
            out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        ws = _workspace(workspace, lib.evo_paged_fwd_workspace_bytes(shape, cache, wlen), q.device)
    strides = SeqStrides(q=sq, out=_rows(out, "out", q.shape, dt))
    _check(lse, "lse", (Hq, T), torch.float32)
    _done(lib.evo_paged_fwd(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(cu_seqlens), _ptr(seq_lens),
                            _ptr(block_table), _ptr(out), _ptr(lse), _ptr(weights), wlen, _ptr(ws), _nbytes(ws), shape,
                            cache, _DTYPE_CODE[dt], ctypes.byref(strides), opts, sp), "evo_paged_fwd")
    return out, lse


def evo_cache_evict(k_pages, v_pages, block_table, seq_lens, weights, budget: int, recent: int = 0, kept=None,
                    stream=None, *, status: Optional[torch.Tensor] = None):
    """Cuts every sequence longer than ``budget`` down to it, in place and per key/value head:
    its ``recent`` newest tokens and the others of the largest ``weights`` [B,Hkv,n]; returns
    kept [B,Hkv,budget] int32, the place every row came from (-1 behind the last)."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4 or k_pages.dtype not in _DTYPE_CODE:
        raise ValueError("k_pages must be a float16 or bfloat16 tensor [num_pages, page_size, kv_heads, head_dim]")
    dt, (Hk, D) = k_pages.dtype, k_pages.shape[2:]
    cache = _cache(k_pages, v_pages, block_table, dt)
    B = block_table.shape[0]
    _ints(seq_lens, "seq_lens", (B,))
    if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
        raise ValueError("weights must be a tensor [seqs, kv_heads, n]")
    _check(weights, "weights", (B, Hk, weights.shape[2]), torch.float32)
    budget, recent = int(budget), int(recent)
    if budget < 1 or not 0 <= recent <= budget:
        raise ValueError(f"1 <= budget and 0 <= recent <= budget are needed, got budget {budget}, recent {recent}")
    sp = _stream_ptr(stream)
    with _On(stream):
        if kept is None:
            kept = torch.empty((B, Hk, budget), dtype=torch.int32, device=k_pages.device)
    _ints(kept, "kept", (B, Hk, budget))
    _done(load().evo_cache_evict(_ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens), _ptr(weights),
                                 weights.shape[2], _ptr(kept), budget, recent, SeqShape(0, B, Hk, Hk, D), cache,
                                 _DTYPE_CODE[dt], _options(None, 0, status), sp), "evo_cache_evict")
    return kept
