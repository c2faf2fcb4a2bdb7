"""Log probabilities of given tokens, with entropy and top alternatives.

One pass over the logits [..., vocab] (float32, float16 or bfloat16, rows at
one or two strides: logits[:, :-1] beside tokens[:, 1:] is read as it lies)
gives, per row, the token's log probability, the entropy of the softmax and the
best entries in descending order, ties to the lower index; all in float32.  A
negative token asks for nothing (log probability 0, no gradient), one past the
vocabulary gives NaN.  Entries of -inf have probability 0; a row of only -inf
has log probability -inf, entropy 0 and a zero gradient.
"""
from __future__ import annotations

import collections

import torch

from . import _native as N
from . import _tensors as T

TokenLogprobs = collections.namedtuple("TokenLogprobs",
                                       ["logprobs", "entropy", "top_ids", "top_logprobs"])


def _check(logits, tokens, top_k):
    code = T.dtype_code(logits, "logits")
    rows, vocab, *at = T.rows_of(logits, "logits") if logits.is_contiguous() else T.grouped_rows_of(logits, "logits")
    T.same_device(logits, tokens=tokens)
    if tokens.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"tokens must be int64 or int32, got {tokens.dtype}")
    if tokens.shape != logits.shape[:-1]:
        raise ValueError(f"tokens must be a tensor of shape {tuple(logits.shape[:-1])}")
    top_k = int(top_k)
    if not 0 <= top_k <= min(64, vocab):
        raise ValueError(f"top_k must be in 0 .. {min(64, vocab)}, got {top_k}")
    if not tokens.is_contiguous():
        tokens = tokens.contiguous()
    return code, rows, vocab, at, tokens, 64 if tokens.dtype == torch.int64 else 32, top_k


def _forward(logits, tokens, top_k, need_lse):
    code, rows, vocab, at, tokens, bits, top_k = _check(logits, tokens, top_k)
    lead = logits.shape[:-1]
    lp = logits.new_empty(lead, dtype=torch.float32)
    ent = torch.empty_like(lp)
    lse = torch.empty_like(lp) if need_lse else None
    ids = tops = None
    if top_k:
        tops = logits.new_empty((*lead, top_k), dtype=torch.float32)
        ids = logits.new_empty((*lead, top_k), dtype=torch.int64)
    ws = T.workspace(logits, N.lib.fm_token_logprobs_workspace(rows, vocab, top_k, code))
    fn = N.lib.fm_token_logprobs if len(at) == 1 else N.lib.fm_token_logprobs_strided
    T.call(logits, fn, logits.data_ptr(), *at, tokens.data_ptr(), bits, lp.data_ptr(), ent.data_ptr(),
           T.ptr(lse), T.ptr(ids), T.ptr(tops), T.ptr(ws), rows, vocab, top_k, code)
    return TokenLogprobs(lp, ent, ids, tops), lse


def token_logprobs_forward(logits, tokens, top_k: int = 0):
    """(TokenLogprobs, lse): the results and the float32 log sum exp of every
    row, which token_logprobs_backward takes."""
    return _forward(logits, tokens, top_k, True)


def token_logprobs(logits, tokens, top_k: int = 0) -> TokenLogprobs:
    """TokenLogprobs(logprobs, entropy, top_ids, top_logprobs) of logits
    [..., vocab] and tokens [...]; the last two are None for top_k = 0.
    Differentiable with respect to the logits."""
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top_k))
    return _forward(logits, tokens, top_k, False)[0]


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logprobs=None, grad_entropy=None,
                            top_ids=None, grad_top_logprobs=None) -> torch.Tensor:
    """The logits' gradient of sum(grad_logprobs * logprobs) + sum(grad_entropy
    * entropy) + sum(grad_top_logprobs * top_logprobs); float32 gradients, None
    where there is none."""
    top_k = top_ids.shape[-1] if isinstance(top_ids, torch.Tensor) and top_ids.dim() else 0
    code, rows, vocab, at, tokens, bits, top_k = _check(logits, tokens, top_k)
    lead = logits.shape[:-1]
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    T.same_device(logits, ("entropy", "grad_logprobs", "grad_entropy", "top_ids", "grad_top_logprobs"),
                  lse=lse, entropy=entropy, grad_logprobs=grad_logprobs,
                  grad_entropy=grad_entropy, top_ids=top_ids, grad_top_logprobs=grad_top_logprobs)
    for name, t in (("lse", lse), ("entropy", entropy), ("grad_logprobs", grad_logprobs),
                    ("grad_entropy", grad_entropy)):
        T.contiguous_f32(t, lead, name)
    if grad_top_logprobs is not None:
        if top_ids is None:
            raise ValueError("grad_top_logprobs needs top_ids")
        T.contiguous_f32(grad_top_logprobs, (*lead, top_k), "grad_top_logprobs")
    if top_ids is not None and (top_ids.dtype != torch.int64 or not top_ids.is_contiguous()
                                or tuple(top_ids.shape) != (*lead, top_k)):
        raise ValueError(f"top_ids must be a contiguous int64 tensor of shape {(*lead, top_k)}")
    dx = logits.new_empty(logits.shape)
    fn = N.lib.fm_token_logprobs_backward if len(at) == 1 else N.lib.fm_token_logprobs_backward_strided
    T.call(logits, fn, logits.data_ptr(), *at, tokens.data_ptr(), bits, lse.data_ptr(), T.ptr(entropy),
           T.ptr(grad_logprobs), T.ptr(grad_entropy), T.ptr(top_ids), T.ptr(grad_top_logprobs), dx.data_ptr(),
           rows, vocab, top_k, code)
    return dx


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top_k):
        r, lse = token_logprobs_forward(logits, tokens, top_k)
        ctx.set_materialize_grads(False)
        if r.top_ids is not None:
            ctx.mark_non_differentiable(r.top_ids)
        ctx.save_for_backward(logits, tokens, lse, r.entropy, r.top_ids)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_lp, g_ent, _, g_top):
        logits, tokens, lse, ent, ids = ctx.saved_tensors
        g_lp, g_ent, g_top = (None if g is None else g.float().contiguous()
                              for g in (g_lp, g_ent, g_top))
        return token_logprobs_backward(logits, tokens, lse, ent, g_lp, g_ent,
                                       ids if g_top is not None else None, g_top), None, None
