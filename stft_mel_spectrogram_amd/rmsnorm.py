"""Root-mean-square norm over the last axis, with the residual's addition.

y = s / sqrt(mean(s^2) + eps) * weight with s = x, or s = x + residual rounded to
x's type, which is returned as the next residual.  x and residual are float32,
float16 or bfloat16 on the GPU, their rows at one stride each; the weight has x's
type or float32.  Sums are float32.  rms_norm_quantized gives y in 8 bits with a
float32 scale per row, for products in 8 bits.
"""
from __future__ import annotations

import torch

from . import _native as N
from . import _tensors as T

_OUT8 = {torch.float8_e4m3fn: N.FM_E4M3, torch.int8: N.FM_I8}


def _check(x, weight, residual):
    code = T.dtype_code(x, "x")
    T.same_device(x, ("weight", "residual"), weight=weight, residual=residual)
    rows, width, stride = T.rows_of(x, "x")
    pcode, r_stride = code, 0
    if weight is not None:
        pcode = T.dtype_code(weight, "weight")
        if pcode not in (code, N.FM_F32):
            raise TypeError(f"weight must be {x.dtype} or float32, got {weight.dtype}")
        if tuple(weight.shape) != (width,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous tensor of shape ({width},)")
    if residual is not None:
        if residual.dtype != x.dtype:
            raise TypeError(f"residual must be {x.dtype} like x, got {residual.dtype}")
        if residual.shape != x.shape:
            raise ValueError(f"residual must have x's shape {tuple(x.shape)}, got {tuple(residual.shape)}")
        _, _, r_stride = T.rows_of(residual, "residual")
    return code, pcode, rows, width, stride, r_stride


def _result(x, out, name):
    if out is None:
        return T.like(x)
    if (not isinstance(out, torch.Tensor) or out.shape != x.shape or out.dtype != x.dtype or out.device != x.device
            or not out.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {x.dtype} tensor of shape {tuple(x.shape)} on {x.device}")
    return out


def _sum(x, residual, out_sum):
    if residual is not None:
        return _result(x, out_sum, "out_sum")
    if out_sum is not None:
        raise ValueError("out_sum needs a residual")
    return None


def _forward(x, weight, residual, eps, stats: bool, out=None, out_sum=None):
    code, pcode, rows, width, stride, r_stride = _check(x, weight, residual)
    given = out is not None or out_sum is not None
    out = _result(x, out, "out")
    total = _sum(x, residual, out_sum)
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32) if stats else None
    T.call(x, N.lib.fm_rms_norm_forward, x.data_ptr(), stride, T.ptr(residual), r_stride, T.ptr(weight),
           out.data_ptr(), T.ptr(total), T.ptr(rstd), rows, width, float(eps), code, pcode)
    if given:
        T.written(out, total)
    return out, total, rstd


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, *, out=None, out_sum=None):
    """y, or (y, x + residual) with a residual; differentiable in all of them.
    out and out_sum take the results (out_sum may be the residual itself)."""
    if T.wants_grad(x, weight, residual, out, out_sum):
        if out is not None or out_sum is not None:
            raise ValueError("out= and out_sum= are not supported for tensors that require grad")
        y, total = _RmsNorm.apply(x, weight, residual, eps)
    else:
        y, total, _ = _forward(x, weight, residual, eps, False, out, out_sum)
    return y if residual is None else (y, total)


def rms_norm_forward(x, weight=None, residual=None, eps: float = 1e-6):
    """(y, what was normed, rstd): the result, x + residual (x itself without
    one) and the float32 row statistic, which rms_norm_backward takes."""
    y, total, rstd = _forward(x, weight, residual, eps, True)
    return y, x if total is None else total, rstd


def rms_norm_backward(grad_out, normed, weight, rstd, grad_sum=None, params: bool = True):
    """(grad_x, grad_weight) of sum(grad_out * y) + sum(grad_sum * (x +
    residual)); grad_x is the residual's gradient too.  grad_weight has the
    weight's type, and is None without a weight or with params=False."""
    code, pcode, rows, width, stride, _ = _check(normed, weight, None)
    T.same_device(normed, ("grad_sum",), grad_out=grad_out, rstd=rstd, grad_sum=grad_sum)
    strides = []
    for name, t in (("grad_out", grad_out), ("grad_sum", grad_sum)):
        if t is None:
            strides.append(0)
            continue
        if t.dtype != normed.dtype or t.shape != normed.shape:
            raise ValueError(f"{name} must be a {normed.dtype} tensor of shape {tuple(normed.shape)}")
        strides.append(T.rows_of(t, name)[2])
    T.contiguous_f32(rstd, normed.shape[:-1], "rstd")
    dx = T.like(normed)
    dw = ws = None
    if weight is not None and params:
        dw = torch.empty_like(weight)
        ws = T.workspace(normed, N.lib.fm_rms_norm_backward_workspace(rows, width, code))
    T.call(normed, N.lib.fm_rms_norm_backward, grad_out.data_ptr(), strides[0], normed.data_ptr(), stride,
           T.ptr(grad_sum), strides[1], T.ptr(weight), rstd.data_ptr(), dx.data_ptr(), T.ptr(dw), T.ptr(ws), rows,
           width, code, pcode)
    return dx, dw


def rms_norm_quantized(x, weight=None, residual=None, eps: float = 1e-6, dtype=torch.float8_e4m3fn, *, out_sum=None):
    """(q, scale), or (q, scale, x + residual) with a residual: y = q * scale in
    8 bits (float8_e4m3fn or int8) with a float32 scale per row, the row's
    largest |y| over 448 or 127.  Not differentiable."""
    if dtype not in _OUT8:
        raise TypeError(f"dtype must be torch.float8_e4m3fn or torch.int8, got {dtype}")
    if T.wants_grad(x, weight, residual, out_sum):
        raise ValueError("rms_norm_quantized has no gradient: call it on detached tensors or under no_grad")
    code, pcode, rows, width, stride, r_stride = _check(x, weight, residual)
    total = _sum(x, residual, out_sum)
    q = x.new_empty(x.shape, dtype=dtype)
    scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    T.call(x, N.lib.fm_rms_norm_quantized, x.data_ptr(), stride, T.ptr(residual), r_stride, T.ptr(weight),
           q.data_ptr(), scale.data_ptr(), T.ptr(total), rows, width, float(eps), code, pcode, _OUT8[dtype])
    if out_sum is not None:
        T.written(out_sum)
    return (q, scale) if residual is None else (q, scale, total)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, normed, rstd = rms_norm_forward(x, weight, residual, eps)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(normed, weight, rstd)
        return y, None if residual is None else normed

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_sum):
        normed, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if grad is None:  # only the sum was used
            return grad_sum if need[0] else None, None, grad_sum if need[2] else None, None
        if grad_sum is not None:
            grad_sum = grad_sum.contiguous()
        dx, dw = rms_norm_backward(grad.contiguous(), normed, weight, rstd, grad_sum, params=need[1])
        return dx if need[0] else None, dw, dx if need[2] else None, None
