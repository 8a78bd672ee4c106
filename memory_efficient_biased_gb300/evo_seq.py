"""ctypes binding of the causal-sequence operators (include/evo_seq.h): argument
marshalling only, like ``evo_attn``.

``evo_prompt_fwd`` / ``evo_prompt_bwd``: attention over packed prompts and its
gradients (differentiable as ``autograd.prompt_attention``);
``evo_cache_append`` / ``evo_paged_fwd`` / ``evo_cache_evict``: a paged cache, the
attention of new tokens over it, and its eviction by accumulated attention weight;
``evo_rotary``: rotary positions of queries and keys, and of their gradients
(differentiable as ``autograd.rotary``), with ``rotary_frequencies`` for long contexts;
``evo_cache8_append`` / ``evo_cache8_read`` / ``evo_paged8_fwd``: a cache in 8 bits with a
scale for each block of tokens and head.
The header states what each computes, its layouts and its limits.

Tensors live on the current CUDA device.  With ``stream`` the call, and what it
allocates, belong to that stream; a tensor made on another stream has to be
synchronised with it by the caller, and kept alive, as for any other use.
Token rows ([tokens, heads, head_dim] tensors) may be strided views whose heads
are packed, such as the parts of one fused projection; anything else is refused
with ValueError.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import evo_attn as E
from .evo_attn import EVO_OK, EvoAttnError, _DTYPE_CODE, _stream_ptr

STRIDE_FIELDS = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


class SeqShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "seqs", "q_heads", "kv_heads", "head_dim")]


class SeqStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in STRIDE_FIELDS]


class CacheShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "pages_per_seq", "k_page_stride",
                                               "v_page_stride")]


class Rotary(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int64), ("flags", ctypes.c_uint32), ("factor", ctypes.c_float),
                ("q_out", ctypes.c_int64), ("k_out", ctypes.c_int64)]


ROTARY_INTERLEAVED, ROTARY_INVERSE = 1, 2  # evo_rotary_t flags


class Cache8Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "pages_per_seq", "scale_block",
                                               "k_page_stride", "v_page_stride")]


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
            ("evo_cache_evict", i32, [vp] * 5 + [i64, vp, i64, i64, SeqShape, CacheShape, i32, opts, vp]),
            ("evo_rotary", i32, [vp] * 6 + [SeqShape, ctypes.POINTER(Rotary), i32, strides, vp]),
            ("evo_cache8_append", i32, [vp] * 9 + [SeqShape, Cache8Shape] + tail),
            ("evo_cache8_read", i32, [vp] * 9 + [SeqShape, Cache8Shape] + tail),
            ("evo_paged8_fwd_workspace_bytes", sz, [SeqShape, Cache8Shape]),
            ("evo_paged8_fwd", i32, [vp] * 11 + [sz, SeqShape, Cache8Shape] + tail)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _bound = lib
    return lib


# The checks of a call run on every one of its tensors, in front of kernels of a few microseconds:
# the current device is asked for once, tensors are looked at through their own methods, and what
# is as it should be passes in one line (append and attention of one token, on an Arm host: 37 us with a function for
# each question, 34 so).
_Tensor = torch.Tensor
_MOST_SCALE = 2.358e38  # times log2 e it is still a float32


def _options(scale, wait_limit_ns, status, dev):
    if scale is None and not wait_limit_ns and status is None:
        return None
    if status is not None:
        _flat(status, "status", None, torch.int32, dev)
        if status.numel() < 1:
            raise ValueError("status must have an element")
    # as the float32 it becomes: a 0 would mean the default, and the kernels multiply it by log2 e
    if scale is not None and not (0.0 < ctypes.c_float(scale).value <= _MOST_SCALE):
        raise ValueError(f"scale must be positive and at most {_MOST_SCALE}, got {scale}")
    if not 0 <= wait_limit_ns < 1 << 64:
        raise ValueError(f"wait_limit_ns must be an unsigned 64-bit number, got {wait_limit_ns}")
    o = SeqOptions(ctypes.sizeof(SeqOptions), 0, scale or 0.0, 0, int(wait_limit_ns),
                   None if status is None else status.data_ptr())
    return ctypes.byref(o)


def _placed(t, name: str, dtype, dev: int):
    if not isinstance(t, _Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.get_device() != dev:
        E._on_current_device(t, name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _flat(t, name: str, shape, dtype, dev: int):
    """Checks a contiguous tensor."""
    if (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype == dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    _placed(t, name, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t, name: str, shape, dtype, dev: int) -> int:
    """Checks a [tokens, heads, head_dim] tensor; its token stride (0 = packed)."""
    if isinstance(t, _Tensor) and t.get_device() == dev and t.dtype == dtype and t.shape == shape:
        if t.is_contiguous():
            return 0
        stride, head, one = t.stride()
        if one == 1 and head == shape[2] and shape[0] > 1 and stride > head * shape[1] and stride % 8 == 0:
            return stride
    _placed(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return 0
    tokens, heads, d = shape
    stride, head, one = t.stride()
    if (d > 1 and one != 1) or (heads > 1 and head != d):
        raise ValueError(f"{name} must have packed (heads, head_dim) dimensions")
    if tokens <= 1 or stride == heads * d:
        return 0
    if stride < heads * d or stride % 8:
        raise ValueError(f"{name} has token stride {stride}: at least {heads * d} and a multiple of 8 is needed")
    return stride


def _like(t, stride: int):
    """A packed tensor of t's shape, from what _rows said of t (torch.empty_like is quicker: 1.4 us on an Arm host, not 1.8)."""
    return torch.empty(t.shape, dtype=t.dtype, device=t.device) if stride else torch.empty_like(t)


def _queries(q, k_heads: int, d: int, keys: str):
    """Shape of q [T, Hq, D] beside keys with k_heads heads of d."""
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [tokens, heads, head_dim]")
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("inputs must be float16 or bfloat16")
    T, Hq, D = q.shape
    if D != d or k_heads < 1 or Hq % k_heads:
        raise ValueError(f"q has {Hq} heads of {D}, {keys} {k_heads} of {d}")
    return T, Hq, D


def _offsets(cu, dev: int) -> int:
    if not isinstance(cu, _Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor [seqs + 1]")
    _flat(cu, "cu_seqlens", None, torch.int32, dev)
    return cu.shape[0] - 1


def _pages(k_pages):
    if not isinstance(k_pages, _Tensor) or k_pages.dim() != 4 or k_pages.dtype not in _DTYPE_CODE:
        raise ValueError("k_pages must be a float16 or bfloat16 tensor [num_pages, page_size, kv_heads, head_dim]")
    return k_pages.shape


def _page_stride(t, name: str, shape, dtype, dev: int, step: int = 8) -> int:
    """Checks the pages of one cache; their stride (0 = packed), a multiple of ``step``."""
    if (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype == dtype and t.is_contiguous()
            and t.shape == shape):
        return 0
    _placed(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.numel() and not t[0].is_contiguous():
        raise ValueError(f"{name} must have contiguous pages")
    if t.shape[0] <= 1 or t.is_contiguous():
        return 0
    stride, packed = t.stride(0), t.shape[1] * t.shape[2] * t.shape[3]
    if stride < packed or stride % step:  # (0, an expanded page, would read as packed)
        raise ValueError(f"{name} has page stride {stride}: at least {packed} and a multiple of {step} is needed")
    return stride


def _cache(k_pages, v_pages, block_table, seqs, dtype, dev: int) -> CacheShape:
    shape = k_pages.shape
    sk, sv = _page_stride(k_pages, "k_pages", shape, dtype, dev), _page_stride(v_pages, "v_pages", shape, dtype, dev)
    return CacheShape(shape[0], shape[1], _columns(block_table, seqs, dev), sk, sv)


def _columns(block_table, seqs, dev: int) -> int:
    """Checks the table; pages a sequence."""
    if not isinstance(block_table, _Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [seqs, pages_per_seq]")
    _flat(block_table, "block_table", None, torch.int32, dev)
    rows, columns = block_table.shape
    if seqs is not None and rows != seqs:
        raise ValueError(f"block_table has {rows} rows, expected {seqs}")
    return columns


def _device_and_stream(t, stream):
    """The current device, which t must be on, and the handle of the stream to launch on."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    dev = torch._C._cuda_getDevice()  # (t is on a GPU: CUDA is up)
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, _stream_ptr(stream).value or 0


_HERE = contextlib.nullcontext()


def _on(stream):
    """Allocations of a call go to the stream it runs on."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _workspace(workspace, need, like, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device), need
    _flat(workspace, "workspace", None, None, dev)
    return workspace, workspace.numel() * workspace.element_size()


def _done(st: int, where: str):
    if st != EVO_OK:
        raise EvoAttnError(st, where)


def _p(t):
    return None if t is None else t.data_ptr()


def evo_prompt_fwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim) -> int:
    return int(load().evo_prompt_fwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim)))


def evo_prompt_bwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim) -> int:
    return int(load().evo_prompt_bwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim)))


def evo_prompt_fwd(q, k, v, cu_seqlens, out=None, lse=None, workspace=None, stream=None, *,
                   scale: Optional[float] = None, wait_limit_ns: int = 0, status: Optional[torch.Tensor] = None):
    """Causal attention within each of the packed sequences; (out [T,Hq,D], lse [Hq,T] fp32).
    Rows in no sequence keep what out and lse held (new ones are uninitialised there)."""
    if not isinstance(k, _Tensor) or k.dim() != 3:
        raise ValueError("k must be a tensor [tokens, heads, head_dim]")
    Hk = k.shape[1]
    T, Hq, D = _queries(q, Hk, k.shape[2], "k")
    dev, sp = _device_and_stream(q, stream)
    dt, rows, keys = q.dtype, q.shape, (T, Hk, D)
    B = _offsets(cu_seqlens, dev)
    sq, sk, sv = _rows(q, "q", rows, dt, dev), _rows(k, "k", keys, dt, dev), _rows(v, "v", keys, dt, dev)
    opts = None if scale is status is None and not wait_limit_ns else _options(scale, wait_limit_ns, status, dev)
    shape, lib, so = SeqShape(T, B, Hq, Hk, D), _bound or load(), 0
    with _on(stream):
        if out is None:
            out = torch.empty(rows, dtype=dt, device=q.device)
        else:
            so = _rows(out, "out", rows, dt, dev)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        else:
            _flat(lse, "lse", (Hq, T), torch.float32, dev)
        ws, size = _workspace(workspace, lib.evo_prompt_fwd_workspace_bytes(shape), q, dev)
    strides = SeqStrides(sq, sk, sv, so) if sq or sk or sv or so else None
    _done(lib.evo_prompt_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), out.data_ptr(),
                             lse.data_ptr(), ws.data_ptr(), size, shape, _DTYPE_CODE[dt], strides, opts, sp),
          "evo_prompt_fwd")
    return out, lse


def evo_prompt_bwd(q, k, v, cu_seqlens, out, lse, dout, dq=None, dk=None, dv=None, workspace=None, stream=None, *,
                   scale: Optional[float] = None, wait_limit_ns: int = 0, status: Optional[torch.Tensor] = None):
    """Gradients of evo_prompt_fwd from its inputs and outputs; (dq, dk, dv).  Rows in no
    sequence keep what dq, dk and dv held (new ones are uninitialised there)."""
    if not isinstance(k, _Tensor) or k.dim() != 3:
        raise ValueError("k must be a tensor [tokens, heads, head_dim]")
    Hk = k.shape[1]
    T, Hq, D = _queries(q, Hk, k.shape[2], "k")
    dev, sp = _device_and_stream(q, stream)
    dt, rows, keys = q.dtype, q.shape, (T, Hk, D)
    B = _offsets(cu_seqlens, dev)
    given = [_rows(q, "q", rows, dt, dev), _rows(k, "k", keys, dt, dev), _rows(v, "v", keys, dt, dev),
             _rows(out, "out", rows, dt, dev), _rows(dout, "dout", rows, dt, dev), 0, 0, 0]
    _flat(lse, "lse", (Hq, T), torch.float32, dev)
    opts = None if scale is status is None and not wait_limit_ns else _options(scale, wait_limit_ns, status, dev)
    shape, lib = SeqShape(T, B, Hq, Hk, D), _bound or load()
    with _on(stream):
        if dq is None:
            dq = torch.empty(rows, dtype=dt, device=q.device)
        else:
            given[5] = _rows(dq, "dq", rows, dt, dev)
        if dk is None:
            dk = torch.empty(keys, dtype=dt, device=q.device)
        else:
            given[6] = _rows(dk, "dk", keys, dt, dev)
        if dv is None:
            dv = torch.empty(keys, dtype=dt, device=q.device)
        else:
            given[7] = _rows(dv, "dv", keys, dt, dev)
        ws, size = _workspace(workspace, lib.evo_prompt_bwd_workspace_bytes(shape), q, dev)
    strides = SeqStrides(*given) if any(given) else None
    _done(lib.evo_prompt_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), out.data_ptr(),
                             lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                             ws.data_ptr(), size, shape, _DTYPE_CODE[dt], strides, opts, sp), "evo_prompt_bwd")
    return dq, dk, dv


def evo_cache_append(k, v, cu_seqlens, seq_lens, k_pages, v_pages, block_table, stream=None, *,
                     status: Optional[torch.Tensor] = None):
    """Writes the new tokens' rows k, v [T,Hkv,D] into the cache: sequence b's are the last
    of its seq_lens[b] (which counts them already)."""
    if not isinstance(k, _Tensor) or k.dim() != 3 or k.dtype not in _DTYPE_CODE:
        raise ValueError("k must be a float16 or bfloat16 tensor [tokens, heads, head_dim]")
    dev, sp = _device_and_stream(k, stream)
    T, Hk, D = keys = k.shape
    dt, B = k.dtype, _offsets(cu_seqlens, dev)
    if tuple(_pages(k_pages)[2:]) != (Hk, D):
        raise ValueError(f"k has {Hk} heads of {D}, the cache {tuple(k_pages.shape[2:])}")
    cache = _cache(k_pages, v_pages, block_table, B, dt, dev)
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    sk, sv = _rows(k, "k", keys, dt, dev), _rows(v, "v", keys, dt, dev)
    strides = SeqStrides(0, sk, sv) if sk or sv else None
    _done(load().evo_cache_append(k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(),
                                  block_table.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                  SeqShape(T, B, Hk, Hk, D), cache, _DTYPE_CODE[dt], strides,
                                  _options(None, 0, status, dev), sp), "evo_cache_append")


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
    _, _, Hk, d = _pages(k_pages)
    T, Hq, D = _queries(q, Hk, d, "the cache")
    dev, sp = _device_and_stream(q, stream)
    dt, rows = q.dtype, q.shape
    B = _offsets(cu_seqlens, dev)
    cache = _cache(k_pages, v_pages, block_table, B, dt, dev)
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    sq, so, wlen = _rows(q, "q", rows, dt, dev), 0, 0
    if weights is not None:
        if not isinstance(weights, _Tensor) or weights.dim() != 3:
            raise ValueError("weights must be a tensor [seqs, kv_heads, n]")
        wlen = weights.shape[2]
        _flat(weights, "weights", (B, Hk, wlen), torch.float32, dev)
    opts = None if scale is status is None and not wait_limit_ns else _options(scale, wait_limit_ns, status, dev)
    shape, lib = SeqShape(T, B, Hq, Hk, D), _bound or load()
    with _on(stream):
        if out is None:
            out = torch.empty(rows, dtype=dt, device=q.device)
        else:
            so = _rows(out, "out", rows, dt, dev)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        else:
            _flat(lse, "lse", (Hq, T), torch.float32, dev)
        ws, size = _workspace(workspace, lib.evo_paged_fwd_workspace_bytes(shape, cache, wlen), q, dev)
    strides = SeqStrides(sq, 0, 0, so) if sq or so else None
    _done(lib.evo_paged_fwd(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), cu_seqlens.data_ptr(),
                            seq_lens.data_ptr(), block_table.data_ptr(), out.data_ptr(), lse.data_ptr(), _p(weights),
                            wlen, ws.data_ptr(), size, shape, cache, _DTYPE_CODE[dt], strides, opts, sp),
          "evo_paged_fwd")
    return out, lse


def evo_cache_evict(k_pages, v_pages, block_table, seq_lens, weights, budget: int, recent: int = 0, kept=None,
                    stream=None, *, status: Optional[torch.Tensor] = None):
    """Cuts every sequence longer than ``budget`` down to it, in place and per key/value head:
    its ``recent`` newest tokens and the others of the largest ``weights`` [B,Hkv,n]; returns
    kept [B,Hkv,budget] int32, the place every row came from (-1 behind the last)."""
    _, _, Hk, D = _pages(k_pages)
    dev, sp = _device_and_stream(k_pages, stream)
    dt = k_pages.dtype
    cache = _cache(k_pages, v_pages, block_table, None, dt, dev)
    B = block_table.shape[0]
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    if not isinstance(weights, _Tensor) or weights.dim() != 3:
        raise ValueError("weights must be a tensor [seqs, kv_heads, n]")
    n = weights.shape[2]
    _flat(weights, "weights", (B, Hk, n), torch.float32, dev)
    budget, recent = int(budget), int(recent)
    if budget < 1 or not 0 <= recent <= budget:
        raise ValueError(f"1 <= budget and 0 <= recent <= budget are needed, got budget {budget}, recent {recent}")
    if kept is None:
        with _on(stream):
            kept = torch.empty((B, Hk, budget), dtype=torch.int32, device=seq_lens.device)
    else:
        _flat(kept, "kept", (B, Hk, budget), torch.int32, dev)
    _done(load().evo_cache_evict(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                 weights.data_ptr(), n, kept.data_ptr(), budget, recent, SeqShape(0, B, Hk, Hk, D),
                                 cache, _DTYPE_CODE[dt], _options(None, 0, status, dev), sp), "evo_cache_evict")
    return kept


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none", stretch: float = 1.0,
                       trained: Optional[int] = None, fast: float = 32.0, slow: float = 1.0, device=None):
    """(inv_freq [rotary_dim / 2] float64, factor) for ``evo_rotary``: pair i turns by
    base^(-2i / rotary_dim) a position.  For contexts ``stretch`` times as long as trained on, ``scaling``
        "linear"  divides every frequency by stretch (positions interpolated);
        "base"    raises the base to base · stretch^(R / (R - 2)): the slowest pair turns
                  stretch times more slowly, the fastest as before;
        "parts"   divides by stretch the pairs that turn fewer than ``slow`` times within the ``trained`` tokens,
                  leaves those that turn more than ``fast`` times, goes over linearly in between,
                  and returns the factor 0.1 ln(stretch) + 1 (otherwise 1)."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not (base > 0 and stretch > 0 and math.isfinite(base) and math.isfinite(stretch)):
        raise ValueError(f"base and stretch must be positive and finite, got {base} and {stretch}")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError(f"scaling must be none, linear, base or parts, got {scaling!r}")
    if scaling == "base" and rotary_dim > 2:
        base = base * stretch ** (rotary_dim / (rotary_dim - 2))
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        return f / stretch, 1.0
    if scaling != "parts":
        return f, 1.0
    if trained is None or trained < 1 or not fast > slow:
        raise ValueError(f"scaling by parts needs trained >= 1 and fast > slow, got {trained}, {fast} and {slow}")
    keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
    return f * keep + f / stretch * (1.0 - keep), 0.1 * math.log(stretch) + 1.0


def evo_rotary(q, k, positions, inv_freq, q_out=None, k_out=None, stream=None, *, interleaved: bool = False,
               inverse: bool = False, factor: float = 1.0):
    """q [T,Hq,D] and k [T,Hk,D] (or None) turned by positions [T] int32 times inv_freq
    [rotary_dim / 2] float64; (q_out, k_out).  An output may be its own input.  ``inverse`` turns back: the
    gradients of the outputs become those of the inputs."""
    if not isinstance(q, _Tensor) or q.dim() != 3 or q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be a float16 or bfloat16 tensor [tokens, heads, head_dim]")
    T, Hq, D = rows = q.shape
    dev, sp = _device_and_stream(q, stream)
    dt, sq, Hk, sk, keys = q.dtype, _rows(q, "q", rows, q.dtype, dev), 0, 0, None
    if k is not None:
        if not isinstance(k, _Tensor) or k.dim() != 3 or k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k must be a tensor [{T}, heads, {D}]")
        keys, Hk = k.shape, k.shape[1]
        sk = _rows(k, "k", keys, dt, dev)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    _flat(positions, "positions", (T,), torch.int32, dev)
    if not isinstance(inv_freq, _Tensor) or inv_freq.dim() != 1 or not 1 <= inv_freq.shape[0] <= D // 2:
        raise ValueError(f"inv_freq must be a tensor of 1 to {D // 2} frequencies")
    _flat(inv_freq, "inv_freq", None, torch.float64, dev)
    if factor != 1.0 and not (0.0 < abs(ctypes.c_float(factor).value) < math.inf):  # (as the float32 it becomes)
        raise ValueError(f"factor must be finite and not 0, got {factor}")
    so, to = 0, 0
    with _on(stream):
        if q_out is None:
            q_out = _like(q, sq)
        else:
            so = _rows(q_out, "q_out", rows, dt, dev)
        if k is not None:
            if k_out is None:
                k_out = _like(k, sk)
            else:
                to = _rows(k_out, "k_out", keys, dt, dev)
    flags = (ROTARY_INTERLEAVED if interleaved else 0) | (ROTARY_INVERSE if inverse else 0)
    strides = SeqStrides(sq, sk) if sq or sk else None
    _done((_bound or load()).evo_rotary(q.data_ptr(), _p(k), positions.data_ptr(), inv_freq.data_ptr(), q_out.data_ptr(),
                                        _p(k_out), SeqShape(T, 0, Hq, Hk, D),
                                        Rotary(2 * inv_freq.shape[0], flags, factor, so, to), _DTYPE_CODE[dt], strides, sp),
          "evo_rotary")
    return q_out, k_out


def _pages8(k_pages):
    if not isinstance(k_pages, _Tensor) or k_pages.dim() != 4 or k_pages.dtype != torch.float8_e4m3fn:
        raise ValueError("k_pages must be a float8_e4m3fn tensor [num_pages, page_size, kv_heads, head_dim]")
    return k_pages.shape


def _cache8(k_pages, v_pages, k_scales, v_scales, block_table, seqs, dev: int) -> Cache8Shape:
    shape, dt = k_pages.shape, k_pages.dtype
    P, page, Hk, _ = shape
    sk = _page_stride(k_pages, "k_pages", shape, dt, dev, 16)
    sv = _page_stride(v_pages, "v_pages", shape, dt, dev, 16)
    n = k_scales.shape[2] if isinstance(k_scales, _Tensor) and k_scales.dim() == 3 else 0
    if n < 1 or page % n:
        raise ValueError("k_scales must be a tensor [num_pages, kv_heads, page_size / scale_block]")
    _flat(k_scales, "k_scales", (P, Hk, n), torch.float32, dev)
    _flat(v_scales, "v_scales", (P, Hk, n), torch.float32, dev)
    return Cache8Shape(P, page, _columns(block_table, seqs, dev), page // n, sk, sv)


def evo_cache8_append(k, v, cu_seqlens, seq_lens, k_pages, v_pages, k_scales, v_scales, block_table, stream=None, *,
                      status: Optional[torch.Tensor] = None):
    """``evo_cache_append`` into a cache in 8 bits: pages float8_e4m3fn
    [num_pages, page_size, Hkv, D], scales float32 [num_pages, Hkv, page_size / scale_block]."""
    if not isinstance(k, _Tensor) or k.dim() != 3 or k.dtype not in _DTYPE_CODE:
        raise ValueError("k must be a float16 or bfloat16 tensor [tokens, heads, head_dim]")
    dev, sp = _device_and_stream(k, stream)
    T, Hk, D = keys = k.shape
    dt, B = k.dtype, _offsets(cu_seqlens, dev)
    if tuple(_pages8(k_pages)[2:]) != (Hk, D):
        raise ValueError(f"k has {Hk} heads of {D}, the cache {tuple(k_pages.shape[2:])}")
    cache = _cache8(k_pages, v_pages, k_scales, v_scales, block_table, B, dev)
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    sk, sv = _rows(k, "k", keys, dt, dev), _rows(v, "v", keys, dt, dev)
    strides = SeqStrides(0, sk, sv) if sk or sv else None
    _done((_bound or load()).evo_cache8_append(
        k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), SeqShape(T, B, Hk, Hk, D),
        cache, _DTYPE_CODE[dt], strides, _options(None, 0, status, dev), sp), "evo_cache8_append")


def evo_cache8_read(k_pages, v_pages, k_scales, v_scales, cu_seqlens, seq_lens, block_table, tokens: int,
                    dtype: torch.dtype = torch.bfloat16, k=None, v=None, stream=None, *,
                    status: Optional[torch.Tensor] = None):
    """The last tokens of every sequence out of a cache in 8 bits, as rows (k, v) [tokens,Hkv,D] of
    ``dtype``: rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 are the last of sequence b's seq_lens[b].
    Rows in no sequence keep what k and v held (new ones are uninitialised there)."""
    _, _, Hk, D = _pages8(k_pages)
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype must be float16 or bfloat16, got {dtype}")
    dev, sp = _device_and_stream(k_pages, stream)
    B, T = _offsets(cu_seqlens, dev), int(tokens)
    if T < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    cache = _cache8(k_pages, v_pages, k_scales, v_scales, block_table, B, dev)
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    sk, sv, keys = 0, 0, (T, Hk, D)
    with _on(stream):
        if k is None:
            k = torch.empty(keys, dtype=dtype, device=k_pages.device)
        else:
            sk = _rows(k, "k", keys, dtype, dev)
        if v is None:
            v = _like(k, sk)
        else:
            sv = _rows(v, "v", keys, dtype, dev)
    strides = SeqStrides(0, sk, sv) if sk or sv else None
    _done((_bound or load()).evo_cache8_read(
        k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), cu_seqlens.data_ptr(),
        seq_lens.data_ptr(), block_table.data_ptr(), k.data_ptr(), v.data_ptr(), SeqShape(T, B, Hk, Hk, D), cache,
        _DTYPE_CODE[dtype], strides, _options(None, 0, status, dev), sp), "evo_cache8_read")
    return k, v


def evo_paged8_fwd_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim, num_pages, page_size, pages_per_seq,
                                   scale_block) -> int:
    return int(load().evo_paged8_fwd_workspace_bytes(SeqShape(tokens, seqs, q_heads, kv_heads, head_dim),
                                                     Cache8Shape(num_pages, page_size, pages_per_seq, scale_block, 0, 0)))


def evo_paged8_fwd(q, k_pages, v_pages, k_scales, v_scales, cu_seqlens, seq_lens, block_table, out=None, lse=None,
                   workspace=None, stream=None, *, scale: Optional[float] = None, wait_limit_ns: int = 0,
                   status: Optional[torch.Tensor] = None):
    """Attention of the new tokens q [T,Hq,D] over a cache in 8 bits that already holds them;
    (out, lse [Hq,T] fp32)."""
    _, _, Hk, d = _pages8(k_pages)
    T, Hq, D = _queries(q, Hk, d, "the cache")
    dev, sp = _device_and_stream(q, stream)
    dt, rows = q.dtype, q.shape
    B = _offsets(cu_seqlens, dev)
    cache = _cache8(k_pages, v_pages, k_scales, v_scales, block_table, B, dev)
    _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    sq, so = _rows(q, "q", rows, dt, dev), 0
    opts = None if scale is status is None and not wait_limit_ns else _options(scale, wait_limit_ns, status, dev)
    shape, lib = SeqShape(T, B, Hq, Hk, D), _bound or load()
    with _on(stream):
        if out is None:
            out = _like(q, sq)
        else:
            so = _rows(out, "out", rows, dt, dev)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        else:
            _flat(lse, "lse", (Hq, T), torch.float32, dev)
        need = lib.evo_paged8_fwd_workspace_bytes(shape, cache)
        ws, size = _workspace(workspace, need, q, dev) if need or workspace is not None else (None, 0)
    strides = SeqStrides(sq, 0, 0, so) if sq or so else None
    _done(lib.evo_paged8_fwd(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                             v_scales.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                             out.data_ptr(), lse.data_ptr(), _p(ws), size, shape, cache, _DTYPE_CODE[dt],
                             strides, opts, sp), "evo_paged8_fwd")
    return out, lse
