"""Gated linear recurrence over time, forward and backward.

    a = sigmoid(forget[t]),  h[t] = a h[t - 1] + (1 - a) x[t],  y[t] = h[t] silu(gate[t])

per channel, from h[-1] = state.  x, forget and gate are [batch, time,
channels] in float32, float16 or bfloat16 on the GPU, with any stride of batch and
strides of time below 8 MiB (slices of one projection are read as they lie; a
single frame's does not matter); states are float32 [batch, channels].  forget of
+inf keeps the state, -inf replaces it; without a gate y = h.  Frames at or past
an entry's length are not part of the sequence: what lies there (NaN) does no
harm, and y and the gradients are 0 there.  The last state carries a sequence on:
a whole recording in pieces, or frame by frame.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as N
from . import _tensors as T

SAVED_FRAMES = 64  # frames between the states that the forward keeps for the backward


class _Call:
    """Checked arguments of a call."""

    __slots__ = ("x", "gate", "state", "shape", "head", "strides")

    def __init__(self, x, forget, gate, state, lengths):
        code = T.dtype_code(x, "x")
        T.same_device(x, ("gate", "state", "lengths"), forget=forget, gate=gate, state=state, lengths=lengths)
        shape = x.shape
        if len(shape) != 3:
            raise ValueError("x must be [batch, time, channels]")
        b, t, c = shape
        if c == 0:
            raise ValueError("x must have at least one channel")
        strides = ()
        for name, v in (("x", x), ("forget", forget), ("gate", gate)):
            if v is None:
                strides += (0, 0)
                continue
            if v.dtype != x.dtype:
                raise TypeError(f"{name} must be {x.dtype} like x, got {v.dtype}")
            if v.shape != shape:
                raise ValueError(f"{name} must have x's shape {tuple(shape)}, got {tuple(v.shape)}")
            st = v.stride()
            if c > 1 and st[2] != 1:
                raise ValueError(f"{name}'s last axis must be contiguous")
            strides += st[:2]
        T.contiguous_f32(state, (b, c), "state")
        if lengths is not None and (lengths.dtype != torch.int32 or lengths.shape != (b,)
                                    or not lengths.is_contiguous()):
            raise ValueError(f"lengths must be a contiguous int32 tensor of shape ({b},)")
        self.x, self.gate, self.state, self.shape, self.strides = x, gate, state, shape, strides
        self.head = (code, 0, b, t, c, x.data_ptr(), forget.data_ptr(), T.ptr(gate), T.ptr(state), T.ptr(lengths))

    def saved_shape(self):
        b, t, c = self.shape
        return b, (t + SAVED_FRAMES - 1) // SAVED_FRAMES, c

    def forward(self, save: bool, out=None, out_state=None):
        x, (b, t, c) = self.x, self.shape
        given = out is not None or out_state is not None
        if out is None:
            out = x.new_empty(self.shape)
        elif (not isinstance(out, torch.Tensor) or out.shape != self.shape or out.dtype != x.dtype
              or out.device != x.device or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous {x.dtype} tensor of shape {tuple(self.shape)} on {x.device}")
        if out_state is None:
            out_state = x.new_empty((b, c), dtype=torch.float32) if self.state is None else torch.empty_like(self.state)
        else:
            T.same_device(x, out_state=out_state)
            T.contiguous_f32(out_state, (b, c), "out_state")
        saved = x.new_empty(self.saved_shape(), dtype=torch.float32) if save else None
        a = N.RecurrenceArgs(*self.head, out.data_ptr(), out_state.data_ptr(), T.ptr(saved), None, None, None, None,
                             None, None, *self.strides, 0, 0)
        ref = ctypes.byref(a)
        # (one tile takes none)
        ws = T.workspace(x, N.lib.fm_gated_recurrence_workspace(ref, 0)) if t > SAVED_FRAMES else None
        T.call(x, N.lib.fm_gated_recurrence_forward, ref, T.ptr(ws))
        if given:
            T.written(out, out_state)
        return out, out_state, saved

    def backward(self, grad_y, saved, grad_state, with_state: bool):
        x, (b, t, c) = self.x, self.shape
        T.same_device(x, ("grad_state",), grad_y=grad_y, saved=saved, grad_state=grad_state)
        if grad_y.shape != self.shape or grad_y.dtype != x.dtype or (c > 1 and grad_y.stride(2) != 1):
            raise ValueError(f"grad_y must be a {x.dtype} tensor of shape {tuple(self.shape)} with a contiguous "
                             "last axis")
        T.contiguous_f32(saved, self.saved_shape(), "saved")
        T.contiguous_f32(grad_state, (b, c), "grad_state")
        dx, df = T.like(grad_y), T.like(grad_y)
        dg = None if self.gate is None else T.like(grad_y)
        ds = x.new_empty((b, c), dtype=torch.float32) if with_state else None
        a = N.RecurrenceArgs(*self.head, None, None, saved.data_ptr(), grad_y.data_ptr(), T.ptr(grad_state),
                             dx.data_ptr(), df.data_ptr(), T.ptr(dg), T.ptr(ds), *self.strides,
                             *grad_y.stride()[:2])
        ref = ctypes.byref(a)
        ws = T.workspace(x, N.lib.fm_gated_recurrence_workspace(ref, 1))
        T.call(x, N.lib.fm_gated_recurrence_backward, ref, T.ptr(ws))
        return dx, df, dg, ds


def gated_recurrence(x, forget, gate=None, state=None, *, lengths=None, out=None, out_state=None):
    """(y, last state) of x, forget, gate [batch, time, channels]; differentiable
    in x, forget, gate and state.

    state: float32 [batch, channels] or None (zeros); lengths: int32 [batch] or
    None; out and out_state take the results (out_state may be state itself, for
    a program that goes on frame by frame).
    """
    if T.wants_grad(x, forget, gate, state, out, out_state):
        if out is not None or out_state is not None:
            raise ValueError("out= and out_state= are not supported for tensors that require grad")
        return _GatedRecurrence.apply(x, forget, gate, state, lengths)
    return _Call(x, forget, gate, state, lengths).forward(False, out, out_state)[:2]


def gated_recurrence_forward(x, forget, gate=None, state=None, *, lengths=None):
    """(y, last state, saved): the results and the states that
    gated_recurrence_backward takes."""
    return _Call(x, forget, gate, state, lengths).forward(True)


def gated_recurrence_backward(grad_y, x, forget, gate, state, saved, *, lengths=None, grad_state=None):
    """(grad_x, grad_forget, grad_gate, grad_state) of sum(grad_y * y) +
    sum(grad_state * last state); the latter two are None without a gate or a
    state.  grad_state: float32 [batch, channels] or None."""
    return _Call(x, forget, gate, state, lengths).backward(grad_y, saved, grad_state, state is not None)


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, forget, gate, state, lengths):
        y, last, saved = gated_recurrence_forward(x, forget, gate, state, lengths=lengths)
        ctx.set_materialize_grads(False)
        # not the state: `saved` has it, and a program may go on in its memory meanwhile
        ctx.save_for_backward(x, forget, gate, lengths, saved)
        ctx.with_state = state is not None
        return y, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_state):
        x, forget, gate, lengths, saved = ctx.saved_tensors
        if grad_y is None and grad_state is None:
            return None, None, None, None, None
        if grad_y is None:
            grad_y = torch.zeros_like(x, memory_format=torch.contiguous_format)
        elif grad_y.stride(-1) != 1:
            grad_y = grad_y.contiguous()
        if grad_state is not None:
            grad_state = grad_state.contiguous()
        grads = _Call(x, forget, gate, None, lengths).backward(grad_y, saved, grad_state, ctx.with_state)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None)
