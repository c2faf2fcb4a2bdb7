"""What the operators' torch-facing callers share: element types, the rows of
a strided tensor, the launch on a tensor's device and torch's current stream."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import _native as N

DTYPES = {torch.float32: N.FM_F32, torch.float16: N.FM_F16, torch.bfloat16: N.FM_BF16}


def _no_tangent(x: torch.Tensor, name: str) -> None:
    """The operators have no forward-mode derivative: a dual number's tangent
    would be lost without a word."""
    if forward_ad.unpack_dual(x).tangent is not None:
        raise NotImplementedError(f"{name} carries a forward-mode tangent, which the operators do not "
                                  "propagate")


def dtype_code(x: torch.Tensor, name: str) -> int:
    """The library's code of x's element type; x must be a GPU tensor."""
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(x).__name__}")
    if forward_ad._current_level >= 0:
        _no_tangent(x, name)
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {x.device}")
    code = DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    return code


def rows_of(x: torch.Tensor, name: str):
    """(rows, width, elements between rows) of x's last axis."""
    if x.dim() < 1:
        raise ValueError(f"{name} must have at least one axis")
    width = x.shape[-1]
    if width == 0:
        raise ValueError(f"{name} must have a last axis of at least one element")
    n = x.numel()
    if x.is_contiguous():
        return n // width, width, width
    if n == 0:
        return 0, width, width
    if width > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    stride, rows = None, 1
    for size, st in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * rows:
            raise ValueError(f"{name}'s leading axes must lie at one stride (make it contiguous)")
        rows *= size
    return rows, width, width if stride is None else stride


def grouped_rows_of(x: torch.Tensor, name: str):
    """(rows, width, elements between rows) of x's last axis, and (rows of a
    group, elements between groups) besides where its rows lie at two strides."""
    if x.is_contiguous() or x.dim() < 3 or x.numel() == 0:
        return rows_of(x, name)
    width = x.shape[-1]
    if width > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    groups = []  # (rows, stride), the last axis's first
    for size, st in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if size == 1:
            continue
        if groups and st == groups[-1][1] * groups[-1][0]:
            groups[-1] = (groups[-1][0] * size, groups[-1][1])
        else:
            groups.append((size, st))
    if len(groups) > 2:
        raise ValueError(f"{name}'s leading axes must lie at one or two strides (make it contiguous)")
    rows = x.numel() // width
    if len(groups) < 2:
        return rows, width, groups[0][1] if groups else width
    return rows, width, groups[0][1], groups[0][0], groups[1][1]


def same_device(x: torch.Tensor, optional: tuple = (), **others) -> None:
    """Checks that the others are tensors on x's device; those named in
    `optional` may be None."""
    dev = x.get_device()
    duals = forward_ad._current_level >= 0
    for name, t in others.items():
        if t is None and name in optional:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
        if duals:
            _no_tangent(t, name)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on {x.device}, got {t.device}")


def contiguous_f32(t, shape, name: str) -> None:
    """Checks a float32 statistics or gradient tensor (None passes)."""
    if t is None:
        return
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")


_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() builds a Stream object first


def call(x: torch.Tensor, fn, *args) -> None:
    """fn(*args, stream) on x's device, on torch's current stream there."""
    dev = x.get_device()
    if torch.cuda.current_device() == dev:
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st < 0:
        N.check(st)


def workspace(x: torch.Tensor, nbytes: int):
    """Scratch memory from torch's allocator (None for 0 bytes); it may be
    freed as soon as the call is enqueued, since the allocator hands it out
    again in stream order."""
    if nbytes < 0:
        N.check(nbytes)
    return x.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None


def ptr(t):
    return None if t is None else t.data_ptr()
