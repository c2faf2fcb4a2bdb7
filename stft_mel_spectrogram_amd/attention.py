"""Attention with a learned relative position bias by buckets.

    s[i, j] = scale * q[i].k[j] + table[buckets[far + clamp(j - pos(i), -far, far)]][head]
    o[i] = sum_j softmax_j(s[i, j]) v[j],   pos(i) = query_offset + i

over the keys j < key_lengths of the batch entry, and j <= pos(i) if causal.
q, k, v are [batch, heads, time, head_dim] (fewer key heads than query heads
are shared evenly) with any strides whose last axis is contiguous, so a slice
of a fused projection or a cache can be passed as it lies.  Scores, softmax
statistics and sums are float32; probabilities and score gradients are
rounded to the element type for their matrix products.  A query without any
key gives zeros and zero gradients.  Keys at or past key_lengths are not read;
those that causal hides have to be finite (their probability is 0, which times
an infinity or NaN is NaN).  Finite table values beyond +-65536 count as
+-65536, so a bucket of the type's lowest value hides its keys from queries that
see others, and leaves queries without others an ordinary softmax; one of -inf
hides them always.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from . import _tensors as T

@functools.lru_cache(maxsize=64)
def _bucket_list(num_buckets: int, max_distance: int, bidirectional: bool) -> tuple:
    side = num_buckets // 2 if bidirectional else num_buckets
    near = side // 2
    grow = side - near

    def bucket(n):
        if n < near:
            return n
        # floor(grow * log(n / near) / log(max_distance / near)), decided in whole numbers
        k = 0
        while k + 1 < grow and n ** grow * near ** (k + 1) >= max_distance ** (k + 1) * near ** grow:
            k += 1
        return near + k

    one = [bucket(n) for n in range(max_distance + 1)]
    left = one[:0:-1]
    right = [side + b for b in one[1:]] if bidirectional else [0] * max_distance
    return tuple(left + [0] + right)


def relative_buckets(num_buckets: int = 32, max_distance: int = 128, bidirectional: bool = True,
                     device=None) -> torch.Tensor:
    """The bucket of every distance key - query in -max_distance .. max_distance
    (int32, on `device`): on each side, half of the buckets hold one distance
    each and the rest grow by a constant ratio up to max_distance, where the
    last one starts.  bidirectional=False puts keys after the query into
    bucket 0.  Any other int32 map of odd length serves relative_attention as
    well; an entry outside the table gives its distance no bias."""
    side = num_buckets // 2 if bidirectional else num_buckets
    if num_buckets < 2 or side < 2 or num_buckets > 1024:
        raise ValueError(f"num_buckets must be in {4 if bidirectional else 2} .. 1024, "
                         f"got {num_buckets}")
    if not side // 2 < max_distance <= 1024:
        raise ValueError(f"max_distance must be in {side // 2 + 1} .. 1024, got {max_distance}")
    dev = torch.device("cuda") if device is None else torch.device(device)
    return torch.tensor(_bucket_list(int(num_buckets), int(max_distance), bool(bidirectional)),
                        dtype=torch.int32, device=dev)


class _Call:
    """Checked arguments of a call."""

    __slots__ = ("q", "k", "v", "table", "code", "head", "inputs", "shape")

    def __init__(self, q, k, v, table, buckets, scale, causal, key_lengths, query_offset):
        code = T.dtype_code(q, "q")
        offset, offset_value = None, 0
        if isinstance(query_offset, torch.Tensor):
            offset = query_offset
        else:
            offset_value = int(query_offset)
        T.same_device(q, ("key_lengths", "query_offset"), k=k, v=v, table=table, buckets=buckets,
                      key_lengths=key_lengths, query_offset=offset)
        shape, kshape = q.shape, k.shape
        if len(shape) != 4 or len(kshape) != 4 or v.dim() != 4:
            raise ValueError("q, k and v must be [batch, heads, time, head_dim]")
        dtype = q.dtype
        if k.dtype != dtype or v.dtype != dtype:
            raise TypeError(f"k and v must be {dtype} like q, got {k.dtype} and {v.dtype}")
        b, h, tq, d = shape
        kb, hk, tk, kd = kshape
        if kshape != v.shape or kb != b or kd != d:
            raise ValueError(f"k and v must be [{b}, key heads, key time, {d}], got "
                             f"{tuple(kshape)} and {tuple(v.shape)}")
        if hk == 0 or h % hk:
            raise ValueError(f"{h} query heads do not divide among {hk} key heads")
        if d < 1 or d > 128:
            raise ValueError(f"head_dim must be in 1 .. 128, got {d}")
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        if d > 1 and not qs[3] == ks[3] == vs[3] == 1:
            raise ValueError("the last axis of q, k and v must be contiguous")
        table_code = T.dtype_code(table, "table")
        if table_code != code and table_code != N.FM_F32:
            raise TypeError(f"table must be {dtype} or float32, got {table.dtype}")
        tshape = table.shape
        if len(tshape) != 2 or tshape[1] != h or not table.is_contiguous():
            raise ValueError(f"table must be a contiguous tensor of shape [buckets, {h}], "
                             f"got {tuple(tshape)}")
        if not 1 <= tshape[0] <= 1024:
            raise ValueError(f"table must have 1 .. 1024 buckets, got {tshape[0]}")
        if buckets.dtype != torch.int32 or buckets.dim() != 1 or not buckets.is_contiguous():
            raise TypeError("buckets must be a contiguous one-dimensional int32 tensor")
        size = buckets.shape[0]
        if size % 2 == 0 or size > 2049:
            raise ValueError(f"buckets must have an odd length of at most 2049, got {size}")
        if key_lengths is not None and (key_lengths.dtype != torch.int32
                                        or key_lengths.shape != (b,)
                                        or not key_lengths.is_contiguous()):
            raise ValueError(f"key_lengths must be a contiguous int32 tensor of shape ({b},)")
        if offset is not None and (offset.dtype != torch.int32 or offset.shape != (b,)
                                   or not offset.is_contiguous()):
            raise ValueError("query_offset must be an int or a contiguous int32 tensor of "
                             f"shape ({b},)")
        self.q, self.k, self.v, self.table, self.code, self.shape = q, k, v, table, code, shape
        self.head = (code, table_code, 1 if causal else 0, size // 2, tshape[0], 0,
                     b, h, hk, tq, tk, d, offset_value,
                     d ** -0.5 if scale is None else float(scale),
                     q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                     buckets.data_ptr(), T.ptr(key_lengths), T.ptr(offset))
        self.inputs = qs[:3] + ks[:3] + vs[:3]

    def forward(self, stats: bool, out=None):
        q = self.q
        if out is None:
            out = _like(q)
        elif (out.shape != q.shape or out.dtype != q.dtype or out.device != q.device
              or (q.shape[3] > 1 and out.stride(3) != 1)):
            raise ValueError(f"out must be a {q.dtype} tensor of shape {tuple(q.shape)} on "
                             f"{q.device} with a contiguous last axis")
        lse = q.new_empty(self.shape[:3], dtype=torch.float32) if stats else None
        a = N.AttentionArgs(*self.head, out.data_ptr(), T.ptr(lse), None, None, None, None, None,
                            *self.inputs, *out.stride()[:3])
        ref = ctypes.byref(a)
        ws = T.workspace(q, N.lib.fm_attention_workspace(ref, 0))
        T.call(q, N.lib.fm_attention_forward, ref, T.ptr(ws))
        return out, lse

    def backward(self, grad_out, out, lse, need_table=True):
        q, k, v = self.q, self.k, self.v
        T.same_device(q, grad_out=grad_out, out=out, lse=lse)
        for name, t in (("grad_out", grad_out), ("out", out)):
            if t.shape != q.shape or t.dtype != q.dtype or (q.shape[3] > 1 and t.stride(3) != 1):
                raise ValueError(f"{name} must be a {q.dtype} tensor of shape {tuple(q.shape)} "
                                 "with a contiguous last axis")
        T.contiguous_f32(lse, q.shape[:3], "lse")
        dq, dk, dv = _like(q), _like(k), _like(v)
        dt = torch.empty_like(self.table) if need_table else None
        a = N.AttentionArgs(*self.head, out.data_ptr(), lse.data_ptr(),
                            grad_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                            T.ptr(dt), *self.inputs, *out.stride()[:3], *grad_out.stride()[:3],
                            *dq.stride()[:3], *dk.stride()[:3], *dv.stride()[:3])
        ref = ctypes.byref(a)
        ws = T.workspace(q, N.lib.fm_attention_workspace(ref, 1))
        T.call(q, N.lib.fm_attention_backward, ref, T.ptr(ws))
        return dq, dk, dv, dt


def _like(x):
    """A dense tensor of x's shape with time outside the heads where x has it
    so (the layout of a projection's output)."""
    b, h, t, d = x.shape
    s = x.stride()
    if h > 1 and s[2] > s[1]:
        return x.new_empty((b, t, h, d)).transpose(1, 2)
    return x.new_empty((b, h, t, d))


def relative_attention(q, k, v, table, buckets, *, scale=None, causal: bool = False,
                       key_lengths=None, query_offset=0, out=None) -> torch.Tensor:
    """o [batch, heads, time, head_dim]; differentiable in q, k, v and table.

    table [num_buckets, heads] (q's type or float32); buckets: an int32 map of
    distances as relative_buckets makes it; scale defaults to head_dim ** -0.5;
    key_lengths: int32 [batch] or None; query_offset: the position of each
    entry's first query, an int or int32 [batch] (for new tokens against a
    cache: the cache length before them).  Few queries against a longer cache
    take a kernel that divides the keys, so one token against a long cache runs
    on the whole GPU.
    """
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (q, k, v, table)):
        if out is not None:
            raise ValueError("out= is not supported for inputs that require grad")
        return _RelativeAttention.apply(q, k, v, table, buckets, scale, causal, key_lengths,
                                        query_offset)
    return _Call(q, k, v, table, buckets, scale, causal, key_lengths,
                 query_offset).forward(False, out)[0]


def relative_attention_forward(q, k, v, table, buckets, *, scale=None, causal: bool = False,
                               key_lengths=None, query_offset=0):
    """(o, lse): the result and the float32 log sum exp of every query's scores
    [batch, heads, time], which relative_attention_backward takes."""
    return _Call(q, k, v, table, buckets, scale, causal, key_lengths, query_offset).forward(True)


def relative_attention_backward(grad_out, q, k, v, table, buckets, out, lse, *, scale=None,
                                causal: bool = False, key_lengths=None, query_offset=0):
    """(grad_q, grad_k, grad_v, grad_table) of sum(grad_out * o), from the
    forward's inputs and both its results."""
    return _Call(q, k, v, table, buckets, scale, causal, key_lengths,
                 query_offset).backward(grad_out, out, lse)


class _RelativeAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, table, buckets, scale, causal, key_lengths, query_offset):
        o, lse = relative_attention_forward(q, k, v, table, buckets, scale=scale, causal=causal,
                                              key_lengths=key_lengths, query_offset=query_offset)
        offset = query_offset if isinstance(query_offset, torch.Tensor) else None
        ctx.how = (scale, causal, query_offset if offset is None else None)
        ctx.save_for_backward(q, k, v, table, buckets, key_lengths, offset, o, lse)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        q, k, v, table, buckets, lengths, offset, o, lse = ctx.saved_tensors
        scale, causal, value = ctx.how
        if grad.stride(-1) != 1:
            grad = grad.contiguous()
        call = _Call(q, k, v, table, buckets, scale, causal, lengths,
                     value if offset is None else offset)
        grads = call.backward(grad, o, lse, ctx.needs_input_grad[3])
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)),
                None, None, None, None, None)
