"""PyTorch autograd over the C ABI: ``evoformer_attention(q, k, v, biases)``.

The call form of the pages' ``DS4Sci_EvoformerAttention(Q, K, V, biases)``
(web page "DeepSpeed4Science 技术指南…" §3.6–§3.7): q, k, v are [B, N, L, H, D]
fp16/bf16 CUDA tensors, ``biases`` a list of at most two tensors — the key mask
[B, N, 1, 1, L] and the pair bias [B, 1, H, L, L], either may be None or left out.
The forward saves O and the fp32 log-sum-exp; the backward returns the gradients
of q, k, v and of whichever biases require them (§3.7: both bias gradients).
Every step runs in the library's sm_103a kernels; there is no fallback.

q, k, v and the incoming gradient are read in place when only their B, N, L
strides differ from a packed tensor's (for instance the transposed view that
column-wise MSA attention or triangle attention around the ending node works
on, §3.6); other layouts are made contiguous first.  O and the gradients are
returned packed in the shape of q.
"""
from typing import List, Optional

import torch
from torch.autograd.function import once_differentiable

from . import evo_attn as E
from . import evo_seq as Q


def readable_in_place(t: torch.Tensor) -> bool:
    """True if the library can read ``t`` through its strides: packed (H, D), a
    16-byte aligned start, B/N/L strides that are positive multiples of 8 below 2^36 and
    rows that do not overlap (the rules of the C ABI's evo_layout_t)."""
    if t.dim() != 5 or not E.row_strided(t) or t.data_ptr() % 16:
        return False
    dims = sorted((t.stride(i), t.shape[i]) for i in range(3) if t.shape[i] > 1)
    need = t.shape[3] * t.shape[4]
    for stride, ext in dims:
        if stride % 8 or stride < need or stride >= 1 << 36:
            return False
        need = stride * ext
    return True


def _in_place_or_packed(t: torch.Tensor) -> torch.Tensor:
    return t if readable_in_place(t) else t.contiguous()


class EvoformerAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, bias1, bias2):
        q, k, v = _in_place_or_packed(q), _in_place_or_packed(k), _in_place_or_packed(v)
        bias1 = None if bias1 is None else bias1.contiguous()
        bias2 = None if bias2 is None else bias2.contiguous()
        out, lse = E.evo_attn_fwd_strided(q, k, v, bias1, bias2)
        ctx.save_for_backward(q, k, v, bias1, bias2, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, bias1, bias2, out, lse = ctx.saved_tensors
        dout = _in_place_or_packed(dout)
        want_db1 = bias1 is not None and ctx.needs_input_grad[3]
        want_db2 = bias2 is not None and ctx.needs_input_grad[4]
        # the pair-bias gradient is computed only when the pair bias needs one
        dq, dk, dv, db1, db2 = E.evo_attn_bwd_opts(q, k, v, bias1, bias2, out, lse, dout, want_dbias1=want_db1,
                                                   want_dbias2=want_db2)
        return dq, dk, dv, db1, db2


def evoformer_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        biases: Optional[List[Optional[torch.Tensor]]] = None) -> torch.Tensor:
    """softmax(q kᵀ D^-1/2 + bias1 + bias2) v over [B, N, L, H, D], differentiable."""
    biases = list(biases or [])
    if len(biases) > 2:
        raise ValueError("at most two biases: the key mask [B,N,1,1,L] and the pair bias [B,1,H,L,L]")
    biases += [None] * (2 - len(biases))
    return EvoformerAttentionFunction.apply(q, k, v, biases[0], biases[1])


# The pages' name for the same call.
DS4Sci_EvoformerAttention = evoformer_attention


def _packed_rows(t: torch.Tensor) -> torch.Tensor:
    """``t`` itself where the library reads its token rows in place, else a packed copy."""
    T, H, D = t.shape
    ok = (D == 1 or t.stride(2) == 1) and (H == 1 or t.stride(1) == D) and t.data_ptr() % 16 == 0
    ok = ok and (T <= 1 or (t.stride(0) >= H * D and t.stride(0) % 8 == 0 and t.stride(0) < 1 << 36))
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class PromptAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale):
        q, k, v = _packed_rows(q), _packed_rows(k), _packed_rows(v)
        # rows in no sequence: zero, so that whatever reads them next is defined
        out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        out, lse = Q.evo_prompt_fwd(q, k, v, cu_seqlens, out=out, scale=scale)
        ctx.save_for_backward(q, k, v, cu_seqlens, out, lse)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, cu_seqlens, out, lse = ctx.saved_tensors
        dq, dk, dv = (torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        Q.evo_prompt_bwd(q, k, v, cu_seqlens, out, lse, _packed_rows(dout), dq, dk, dv, scale=ctx.scale)
        return dq, dk, dv, None, None


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     scale: Optional[float] = None) -> torch.Tensor:
    """Causal attention within each of the packed sequences, differentiable: q [T, Hq, D],
    k, v [T, Hkv, D] with Hq a multiple of Hkv, cu_seqlens int32 [B + 1] on the device; ``scale``
    defaults to D^-1/2.  Rows in no sequence get zeros, and zero gradients.

    Strided token rows (the parts of one fused projection) are read in place.  The gradients are
    not differentiable themselves (an error says so).  To capture the
    backward into a CUDA graph, run the forward inside the same capture, on the stream that is
    being captured: PyTorch ties the accumulation of a leaf's gradient to the stream on which
    the leaf was first used, and a capture that meets another stream's work ends with an error."""
    return PromptAttentionFunction.apply(q, k, v, cu_seqlens, scale)


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, factor):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = {"interleaved": interleaved, "factor": factor}
        q, k = Q.evo_rotary(_packed_rows(q), None if k is None else _packed_rows(k), positions, inv_freq, **ctx.how)
        return q, k

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        positions, inv_freq = ctx.saved_tensors
        # (autograd gives zeros for an output that nothing used)
        dq, dk = Q.evo_rotary(_packed_rows(dq), None if dk is None else _packed_rows(dk), positions, inv_freq,
                              inverse=True, **ctx.how)
        return dq, dk, None, None, None, None


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, *,
           interleaved: bool = False, factor: float = 1.0):
    """Rotary positions, differentiable: q [T, Hq, D] and k [T, Hk, D] (or None) turned by positions [T] int32
    times inv_freq [rotary_dim / 2] float64 (``evo_seq.rotary_frequencies``); (q, k), as
    ``prompt_attention`` takes them.  Strided token rows are read in place.  The gradients are not differentiable
    themselves, and a captured backward needs its forward inside the same capture, as there.  Frequencies get no
    gradient: some that require one are refused."""
    if isinstance(inv_freq, torch.Tensor) and inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq gets no gradient here: give it detached")
    return RotaryFunction.apply(q, k, positions, inv_freq, interleaved, factor)
