"""torch.autograd functions whose reverse pass is deterministic.

Warp user guide "Deterministic Execution", "Tape and Backward Passes": a
forward gather has no atomic, but its adjoint accumulates the output gradient
into the gradient of the gathered array -- a scatter-add, and with repeated
indices a nondeterministic one.  Here the forward runs ``det_gather_rows`` and
the adjoint runs ``det_scatter_add`` (1-D values) or ``det_scatter_add_rows``
(row tables) of the library, so the gradient bits are the same on every run
and at every launch shape.  Indices outside the source get zero outputs and
send no gradient.  Two operators of language models follow the same rule: the log
probabilities of given tokens, and the learned relative position bias, whose
adjoint is a scatter-add on a few buckets.  Argument marshalling only: every step runs in the
library's CUDA kernels (the gradient buffer is zero-filled by torch).
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import det


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, src: torch.Tensor, idx: torch.Tensor, row_offset: int):
        ctx.save_for_backward(idx)
        ctx.src_shape = src.shape
        ctx.row_offset = row_offset
        return det.det_gather_rows(src.contiguous(), idx, row_offset=row_offset)

    @staticmethod
    def backward(ctx, grad_out: torch.Tensor):
        (idx,) = ctx.saved_tensors
        grad_src = None
        if ctx.needs_input_grad[0]:
            g = grad_out.contiguous()
            grad_src = torch.zeros(ctx.src_shape, dtype=g.dtype, device=g.device)
            if len(ctx.src_shape) == 1 and ctx.row_offset == 0:
                det.det_scatter_add(grad_src, idx, g)
            elif len(ctx.src_shape) == 1:   # same bits as det_scatter_add: rows of one element
                det.det_scatter_add_rows(grad_src.view(-1, 1), idx, g.view(-1, 1), row_offset=ctx.row_offset)
            else:
                det.det_scatter_add_rows(grad_src, idx, g, row_offset=ctx.row_offset)
        return grad_src, None, None


def gather(src: torch.Tensor, idx: torch.Tensor, row_offset: int = 0) -> torch.Tensor:
    """``src[idx + row_offset]`` (rows for a 2-D ``src``) with a deterministic backward.

    ``src`` is float32 or float64 on CUDA, ``idx`` int32 on the same device."""
    return _Gather.apply(src, idx, int(row_offset))


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits: torch.Tensor, tokens: torch.Tensor):
        r = det.det_token_logprobs(logits, tokens)
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        ctx.set_materialize_grads(False)
        return r.logprob, r.entropy

    @staticmethod
    def backward(ctx, grad_logprob, grad_entropy):
        if not ctx.needs_input_grad[0] or (grad_logprob is None and grad_entropy is None):
            return None, None
        return _TokenLogprobsGrad.apply(*ctx.saved_tensors, grad_logprob, grad_entropy), None


class _TokenLogprobsGrad(torch.autograd.Function):
    """The gradient as a function of the logits, so that under create_graph its own derivative is asked for here and refused
    (once_differentiable would notice only incoming gradients that need one)."""

    @staticmethod
    def forward(ctx, logits, tokens, lse, entropy, grad_logprob, grad_entropy):
        return det.det_token_logprobs_backward(
            logits, tokens, lse, entropy,
            grad_logprob=None if grad_logprob is None else grad_logprob.contiguous(),
            grad_entropy=None if grad_entropy is None else grad_entropy.contiguous())

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("token_logprobs has no second derivative")


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(log probability of each token, entropy of each row) under softmax(logits), float32.

    logits is [..., vocab] (float32, bfloat16 or float16), tokens int32 of the leading shape; tokens outside the
    vocabulary (padding) have log probability 0 and send no gradient.  Any strides will do; logits whose rows do not lie at
    one stride (logits[:, :-1] against tokens[:, 1:]) are copied, which whole logits with a token of -1 at each
    sequence's end are not.  There is no second derivative."""
    if not tokens.is_contiguous():
        tokens = tokens.contiguous()
    if logits.dim() and not logits.is_contiguous() and (
            (logits.shape[-1] > 1 and logits.stride(-1) != 1) or det._row_stride(logits) is None):
        logits = logits.contiguous()
    return _TokenLogprobs.apply(logits, tokens)


class _RelativeBias(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, bounds, q_len, k_len, q_offset, bidirectional, batch, dtype):
        ctx.save_for_backward(bounds)
        ctx.how = dict(q_offset=q_offset, bidirectional=bidirectional, dtype=table.dtype)
        out = det.det_relative_bias(table, bounds, q_len, k_len, q_offset=q_offset, bidirectional=bidirectional,
                                    dtype=dtype)
        return out if batch is None else out.expand(batch, *out.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (bounds,) = ctx.saved_tensors
        table_grad = None
        if ctx.needs_input_grad[0]:
            if grad.shape[-1] > 1 and grad.stride(-1) != 1:
                grad = grad.contiguous()
            table_grad = det.det_relative_bias_backward(grad, bounds, **ctx.how)
        return (table_grad,) + (None,) * 7


def relative_bias(table: torch.Tensor, bounds: torch.Tensor, q_len: int, k_len: int, *, q_offset: int = 0,
                  bidirectional: bool = False, batch: Optional[int] = None,
                  dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """det.det_relative_bias with a deterministic gradient for the table.

    With ``batch`` the result is expanded (not copied) to [batch, heads, q_len, k_len], and the gradient's sum over
    the batch is taken with the buckets' sums, in one pass over the gradient.  There is no second derivative."""
    return _RelativeBias.apply(table, bounds, int(q_len), int(k_len), int(q_offset), bool(bidirectional), batch, dtype)
