"""Layer norm over the last axis, forward and backward.

y = (x - mean) / sqrt(var + eps) * weight + bias with float32 statistics, the
variance from the centred row.  x is float32, float16 or bfloat16 on the GPU,
its rows at one stride (a slice of a wider tensor is fine); weight and bias
have x's type or float32.  The backward also reduces the weight's and bias's
gradients over the rows, in a fixed order.
"""
from __future__ import annotations

import torch

from . import _native as N
from . import _tensors as T


def _check(x, weight, bias):
    code = T.dtype_code(x, "x")
    rows, width, stride = T.rows_of(x, "x")
    pcode = code
    if weight is not None:
        T.same_device(x, ("bias",), weight=weight, bias=bias)
        pcode = T.dtype_code(weight, "weight")
        if pcode not in (code, N.FM_F32):
            raise TypeError(f"weight must be {x.dtype} or float32, got {weight.dtype}")
        if tuple(weight.shape) != (width,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous tensor of shape ({width},)")
        if bias is not None:
            if bias.dtype != weight.dtype:
                raise TypeError(f"bias must be {weight.dtype} like the weight, got {bias.dtype}")
            if tuple(bias.shape) != (width,) or not bias.is_contiguous():
                raise ValueError(f"bias must be a contiguous tensor of shape ({width},)")
    elif bias is not None:
        raise ValueError("a bias needs a weight")
    return code, pcode, rows, width, stride


def _forward(x, weight, bias, eps, stats: bool, out=None):
    code, pcode, rows, width, stride = _check(x, weight, bias)
    if out is None:
        out = x.new_empty(x.shape)
    elif (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device
          or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {x.dtype} tensor of shape {tuple(x.shape)} "
                         f"on {x.device}")
    mean = rstd = None
    if stats:
        mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    T.call(x, N.lib.fm_layer_norm_forward, x.data_ptr(), stride, T.ptr(weight), T.ptr(bias),
           out.data_ptr(), T.ptr(mean), T.ptr(rstd), rows, width, float(eps), code, pcode)
    return out, mean, rstd


def layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """Layer norm over x's last axis; differentiable."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (x, weight, bias)):
        if out is not None:
            raise ValueError("out= is not supported for inputs that require grad")
        return _LayerNorm.apply(x, weight, bias, eps)
    return _forward(x, weight, bias, eps, False, out)[0]


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5):
    """(y, mean, rstd): the result and the float32 row statistics that
    layer_norm_backward takes."""
    return _forward(x, weight, bias, eps, True)


def layer_norm_backward(grad_out, x, weight, mean, rstd, params: bool = True):
    """(grad_x, grad_weight, grad_bias) of sum(grad_out * y).  The latter two
    have the weight's type, and are None without a weight or with
    params=False."""
    code, pcode, rows, width, stride = _check(x, weight, None)
    T.same_device(x, grad_out=grad_out, mean=mean, rstd=rstd)
    if grad_out.dtype != x.dtype or grad_out.shape != x.shape:
        raise ValueError(f"grad_out must be a {x.dtype} tensor of shape {tuple(x.shape)}")
    _, _, g_stride = T.rows_of(grad_out, "grad_out")
    T.contiguous_f32(mean, x.shape[:-1], "mean")
    T.contiguous_f32(rstd, x.shape[:-1], "rstd")
    dx = x.new_empty(x.shape)
    dw = db = ws = None
    if weight is not None and params:
        dw, db = torch.empty_like(weight), torch.empty_like(weight)
        ws = T.workspace(x, N.lib.fm_layer_norm_backward_workspace(rows, width, code))
    T.call(x, N.lib.fm_layer_norm_backward, grad_out.data_ptr(), g_stride, x.data_ptr(), stride,
           T.ptr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), T.ptr(dw), T.ptr(db),
           T.ptr(ws), rows, width, code, pcode)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(grad.contiguous(), x, weight, mean, rstd,
                                         params=need[1] or need[2])
        return dx if need[0] else None, dw if need[1] else None, db if need[2] else None, None
