"""The training step as autograd functions: ``rotary`` on Q and K, then
``attention``, dense or skipping. Each is one forward and one backward call of
the library; nothing here computes.

    q, k = training.rotary(q, k, positions, inv_freq, sections, interleaved=True)
    out = training.attention(q, k, v, cu_seqlens, max_seqlen, threshold_scale_factor)
    out.backward(dout)

Rows outside every sequence of ``cu_seqlens`` are zero in the output and in the
gradients. Skip decisions count as constants in the backward pass.

Autograd graphs are not captured into CUDA graphs (the engine's accumulation
nodes may belong to a graph of another stream, which ends the process): under
capture these functions raise. ``fwd_lse``, ``bwd`` and ``rotary`` of the
package can be captured.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import bitmap_words as _bitmap_words
from . import bwd as _bwd
from . import bwd_fp8 as _bwd_fp8
from . import fwd_lse as _fwd_lse
from . import num_qblocks as _num_qblocks
from . import rotary as _rotary
from . import save_fp8 as _save_fp8


def _no_capture(what: str):
    if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what}: autograd functions cannot be captured into a CUDA graph; "
                           "capture fwd_lse, bwd and rotary instead")


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, sections, interleaved, scale):
        _no_capture("rotary")
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = dict(sections=sections, interleaved=interleaved, scale=scale)
        ctx.set_materialize_grads(False)
        return _rotary(q, k, positions, inv_freq, **ctx.how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        _no_capture("rotary")
        positions, inv_freq = ctx.saved_tensors
        grads = [None if g is None else g.contiguous() for g in (dq, dk)]
        turn = lambda a, b: _rotary(a, b, positions, inv_freq, transpose=True, **ctx.how)
        if grads[0] is not None:
            grads = list(turn(grads[0], grads[1]))
        elif grads[1] is not None:
            grads[1] = turn(grads[1], None)[0]
        return grads[0], grads[1], None, None, None, None, None


def rotary(q, k, positions, inv_freq, sections: Optional[Sequence[int]] = None, interleaved: bool = False,
           scale: float = 1.0):
    """Differentiable ``rotary`` (see the package's); k may be None. Gradients
    flow to q and k."""
    return _Rotary.apply(q, k, positions, inv_freq, None if sections is None else tuple(sections), bool(interleaved),
                         float(scale))


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_seqlen, threshold_scale_factor, softmax_scale, num_qblocks, save_8bit):
        _no_capture("attention")
        bitmap = None
        if threshold_scale_factor > 0.0:
            n = _num_qblocks(cu_seqlens) if num_qblocks is None else int(num_qblocks)
            bitmap = torch.empty((q.shape[1], n, _bitmap_words(max_seqlen)), dtype=torch.int32, device=q.device)
        out, lse = _fwd_lse(q, k, v, cu_seqlens, max_seqlen, threshold_scale_factor, softmax_scale,
                            out=torch.zeros_like(q), decision_bitmap=bitmap)
        saved = [t for x in (q, k, v) for t in _save_fp8(x)] if save_8bit else [q, k, v]
        ctx.save_for_backward(out, lse, cu_seqlens, bitmap, *saved)
        ctx.how = (max_seqlen, softmax_scale, save_8bit)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        _no_capture("attention")
        out, lse, cu_seqlens, bitmap, *saved = ctx.saved_tensors
        max_seqlen, softmax_scale, save_8bit = ctx.how
        if save_8bit:
            (q, qs, k, ks, v, vs), call = saved, _bwd_fp8
            inputs = ((q, qs), (k, ks), (v, vs))
        else:
            inputs, call = saved, _bwd
            q, k, v = saved
        grads = [torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device) for x in (q, k, v)]
        call(dout.contiguous(), *inputs, out, lse, cu_seqlens, max_seqlen, softmax_scale, bitmap, *grads)
        return (*grads, None, None, None, None, None, None)


def attention(q, k, v, cu_seqlens, max_seqlen: int, threshold_scale_factor: float = 0.0, softmax_scale: float = 0.0,
              num_qblocks: Optional[int] = None, save_8bit: bool = False):
    """Differentiable skip-softmax attention: q bf16 [total_tokens, H, D], k and
    v [total_tokens, Hkv, D]. With a threshold the forward's decisions are kept
    for the backward pass; ``num_qblocks`` (the package's num_qblocks() of the
    batch) then saves reading cu_seqlens on the host. ``save_8bit`` keeps Q, K
    and V between the passes as save_fp8() codes, in about half the memory, and
    differentiates at the restored values."""
    return _Attention.apply(q, k, v, cu_seqlens, int(max_seqlen), float(threshold_scale_factor), float(softmax_scale),
                            num_qblocks, bool(save_8bit))
