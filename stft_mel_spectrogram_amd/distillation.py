"""Distillation from a teacher's top log probabilities.

Per row of logits [..., vocab] (float32, float16 or bfloat16, rows at one or two
strides) and a teacher's best tokens with their log probabilities, as
token_logprobs(..., top_k) of a larger model gives them:

    loss = T^2 sum_k q_k (log q_k - log_softmax(logits / T)[ids_k]),  q = softmax(lps / T)

over the given tokens, T the temperature.  With rest=True (T = 1) q = exp(lps),
and the mass that the teacher leaves for all others stands against the
student's: one more term, r log(r / R).  A negative id is no entry; a row without
entries has loss 0 and no gradient.  A student that leaves no other token any
probability (all of them -inf, or none there) has no such term, since r may be
rounding alone; a named token of -inf gives an infinite loss.
"""
from __future__ import annotations

import torch

from . import _native as N
from . import _tensors as T


def _detached(lps):
    if T.wants_grad(lps):
        raise ValueError("teacher_logprobs has no gradient here: detach it")


def _check(logits, ids, lps):
    code = T.dtype_code(logits, "logits")
    rows, vocab, *at = T.grouped_rows_of(logits, "logits")
    T.same_device(logits, teacher_ids=ids, teacher_logprobs=lps)
    if ids.dtype != torch.int64:
        raise TypeError(f"teacher_ids must be int64, got {ids.dtype}")
    if ids.shape[:-1] != logits.shape[:-1] or ids.dim() != logits.dim() or not 1 <= ids.shape[-1] <= 64:
        raise ValueError(f"teacher_ids must be a tensor of shape {tuple(logits.shape[:-1])} and 1 .. 64 entries, "
                         f"got {tuple(ids.shape)}")
    if lps.dtype != torch.float32:
        raise TypeError(f"teacher_logprobs must be float32, got {lps.dtype}")
    if lps.shape != ids.shape:
        raise ValueError(f"teacher_logprobs must have teacher_ids' shape {tuple(ids.shape)}, got {tuple(lps.shape)}")
    _detached(lps)
    at = (*at, 0, 0) if len(at) == 1 else at
    if not ids.is_contiguous():
        ids = ids.contiguous()
    if not lps.is_contiguous():
        lps = lps.contiguous()
    return code, rows, vocab, at, ids, lps


def _forward(logits, ids, lps, temperature, rest, stats: bool):
    code, rows, vocab, at, ids, lps = _check(logits, ids, lps)
    loss = logits.new_empty(logits.shape[:-1], dtype=torch.float32)
    st = logits.new_empty((*logits.shape[:-1], 4), dtype=torch.float32) if stats else None
    ws = T.workspace(logits, N.lib.fm_distill_workspace(rows, vocab, code))
    T.call(logits, N.lib.fm_distill, logits.data_ptr(), *at, ids.data_ptr(), lps.data_ptr(), loss.data_ptr(),
           T.ptr(st), T.ptr(ws), rows, vocab, ids.shape[-1], float(temperature), 1 if rest else 0, code)
    return loss, st


def topk_distillation(logits, teacher_ids, teacher_logprobs, *, temperature: float = 1.0, rest: bool = False):
    """The loss of every row, float32 [...]; differentiable in the logits.

    teacher_ids int64 and teacher_logprobs float32 [..., k], 1 <= k <= 64;
    temperature in 2^-10 .. 2^10; rest=True counts the mass outside the named
    tokens too (temperature 1 only, teacher_logprobs as they are).
    """
    _detached(teacher_logprobs)  # (within the recorded function nothing wants a gradient)
    if T.wants_grad(logits):
        return _TopkDistillation.apply(logits, teacher_ids, teacher_logprobs, temperature, rest)
    return _forward(logits, teacher_ids, teacher_logprobs, temperature, rest, False)[0]


def topk_distillation_forward(logits, teacher_ids, teacher_logprobs, *, temperature: float = 1.0,
                              rest: bool = False):
    """(loss, stats): the losses and the float32 [..., 4] row statistics that
    topk_distillation_backward takes."""
    return _forward(logits, teacher_ids, teacher_logprobs, temperature, rest, True)


def topk_distillation_backward(grad_loss, logits, teacher_ids, teacher_logprobs, stats, *, temperature: float = 1.0,
                               rest: bool = False):
    """The logits' gradient of sum(grad_loss * loss); grad_loss float32 [...]."""
    code, rows, vocab, at, ids, lps = _check(logits, teacher_ids, teacher_logprobs)
    T.same_device(logits, grad_loss=grad_loss, stats=stats)
    T.contiguous_f32(grad_loss, logits.shape[:-1], "grad_loss")
    T.contiguous_f32(stats, (*logits.shape[:-1], 4), "stats")
    dx = T.like(logits)
    T.call(logits, N.lib.fm_distill_backward, logits.data_ptr(), *at, ids.data_ptr(), lps.data_ptr(),
           stats.data_ptr(), grad_loss.data_ptr(), dx.data_ptr(), rows, vocab, ids.shape[-1], float(temperature),
           1 if rest else 0, code)
    return dx


class _TopkDistillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, lps, temperature, rest):
        loss, stats = topk_distillation_forward(logits, ids, lps, temperature=temperature, rest=rest)
        ctx.how = dict(temperature=temperature, rest=rest)
        ctx.save_for_backward(logits, ids, lps, stats)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, ids, lps, stats = ctx.saved_tensors
        return (topk_distillation_backward(grad.float().contiguous(), logits, ids, lps, stats, **ctx.how),
                None, None, None, None)
