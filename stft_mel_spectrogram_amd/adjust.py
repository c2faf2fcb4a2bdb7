"""Logits before a token is chosen from them: penalties for repeated tokens,
biases, and masks of allowed tokens, in one pass.

    x = x > 0 ? x (1 / repetition) : x repetition     for tokens of the history
    x = x - frequency * count - presence * (count > 0)
    x = x + the token's biases
    x = -inf                                          where a token is not allowed

in float32, rounded once to the logits' type.  token_logprobs takes the result.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as N
from . import _tensors as T


def _per_row(x, lead, value, name):
    """(tensor or None, number) of a penalty."""
    if not isinstance(value, torch.Tensor):
        return None, float(value)
    T.same_device(x, **{name: value})
    T.contiguous_f32(value, lead, name)
    return value, 0.0


def _lengths(lead, t, name):
    if t is not None and (t.dtype != torch.int32 or t.shape != lead or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(lead)}")


def adjust_logits(logits, history=None, history_lengths=None, *, prompt_lengths=None, repetition=1.0, frequency=0.0,
                  presence=0.0, bias_ids=None, bias=None, allowed=None, out=None) -> torch.Tensor:
    """The adjusted logits, contiguous, of logits [..., vocab] (float32, float16
    or bfloat16, rows at one stride).

    history: the tokens so far, int64 or int32 [..., length], of which
    history_lengths (int32 [...], None: all) count, tokens outside the vocabulary
    never; the first prompt_lengths of them (int32 [...], None: 0) are penalised
    by repetition alone.  repetition (> 0), frequency and presence: numbers or
    float32 [...].  bias_ids int64 and bias float32 [..., n], n <= 1024: ids
    outside the vocabulary are none, the same id twice counts twice.  allowed:
    int32 words of 32 tokens' bits, the lowest bit first, [(vocab + 31) // 32]
    for all rows or [..., (vocab + 31) // 32].  out takes the result and may be
    the logits themselves.  Up to 2^22 rows times segments of 2048 tokens.  Not
    differentiable: tensors that require grad are refused.
    """
    code = T.dtype_code(logits, "logits")
    if T.wants_grad(logits, repetition, frequency, presence, bias, out):
        raise ValueError("adjust_logits has no gradient: call it on detached tensors or under no_grad")
    rows, vocab, stride = T.rows_of(logits, "logits")
    lead = logits.shape[:-1]
    T.same_device(logits, ("history", "history_lengths", "prompt_lengths", "bias_ids", "bias", "allowed", "out"),
                  history=history, history_lengths=history_lengths, prompt_lengths=prompt_lengths,
                  bias_ids=bias_ids, bias=bias, allowed=allowed, out=out)
    length, bits, h_stride = 0, 64, 0
    if history is not None:
        if history.dtype not in (torch.int64, torch.int32):
            raise TypeError(f"history must be int64 or int32, got {history.dtype}")
        if history.dim() != logits.dim() or history.shape[:-1] != lead:
            raise ValueError(f"history must be a tensor of shape {tuple(lead)} and a length, got "
                             f"{tuple(history.shape)}")
        length, bits = history.shape[-1], 64 if history.dtype == torch.int64 else 32
        if length:
            h_stride = T.rows_of(history, "history")[2]
    elif history_lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths need a history")
    _lengths(lead, history_lengths, "history_lengths")
    _lengths(lead, prompt_lengths, "prompt_lengths")
    rep, rep_value = _per_row(logits, lead, repetition, "repetition")
    freq, freq_value = _per_row(logits, lead, frequency, "frequency")
    pres, pres_value = _per_row(logits, lead, presence, "presence")
    biases = 0
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        if bias_ids.dtype != torch.int64:
            raise TypeError(f"bias_ids must be int64, got {bias_ids.dtype}")
        if bias_ids.dim() != logits.dim() or bias_ids.shape[:-1] != lead or not bias_ids.is_contiguous():
            raise ValueError(f"bias_ids must be a contiguous tensor of shape {tuple(lead)} and a number of biases")
        biases = bias_ids.shape[-1]
        T.contiguous_f32(bias, bias_ids.shape, "bias")
    given = out is not None
    a_stride = 0
    if allowed is not None:
        words = (vocab + 31) // 32
        if allowed.dtype != torch.int32:
            raise TypeError(f"allowed must be int32, got {allowed.dtype}")
        if allowed.shape != (words,) and allowed.shape != (*lead, words):
            raise ValueError(f"allowed must be a tensor of shape ({words},) or {(*lead, words)}, got "
                             f"{tuple(allowed.shape)}")
        _, _, a_stride = T.rows_of(allowed, "allowed")
        if allowed.dim() == 1:
            a_stride = 0
    if out is None:
        out = T.like(logits)
    elif out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {logits.dtype} tensor of shape {tuple(logits.shape)}")
    a = N.AdjustArgs(code, bits, rows, vocab, length, biases, stride, h_stride, a_stride, rep_value, freq_value,
                     pres_value, logits.data_ptr(), out.data_ptr(), T.ptr(history), T.ptr(history_lengths),
                     T.ptr(prompt_lengths), T.ptr(rep), T.ptr(freq), T.ptr(pres), T.ptr(bias_ids), T.ptr(bias),
                     T.ptr(allowed))
    T.call(logits, N.lib.fm_adjust_logits, ctypes.byref(a))
    if given:
        T.written(out)
    return out
