"""Refusals of the recurrence, the RMS norm, the distillation and the adjusted
logits, on the CPU: the C ABI checks every argument before any HIP call, so made-up
device addresses are never used."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")  # before the library, which then takes torch's HIP runtime
from stft_mel_spectrogram_amd import _native as N  # noqa: E402

P = 1 << 20  # an address that must not be touched


def fill(a, base, kw):
    base.update(kw)
    for name, value in base.items():
        assert hasattr(a, name), name
        setattr(a, name, value)
    return ctypes.byref(a)


def recurrence(backward=False, ws=P, **kw):
    names = ("x", "forget", "gate", "state", "lengths", "y", "last_state", "saved", "grad_y", "grad_last", "grad_x",
             "grad_forget", "grad_gate", "grad_state")
    base = dict(dtype=N.FM_BF16, batch=2, time=9000, channels=40, **{n: P for n in names})
    base.update({f"{t}_stride_{x}": 40 for t in ("x", "forget", "gate", "grad_y") for x in ("entry", "time")})
    fn = N.lib.fm_gated_recurrence_backward if backward else N.lib.fm_gated_recurrence_forward
    return fn(fill(N.RecurrenceArgs(), base, kw), ws, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [
    dict(dtype=N.FM_I16), dict(dtype=9), dict(batch=-1), dict(batch=1 << 30), dict(time=-1), dict(time=1 << 30),
    dict(channels=0), dict(channels=-4), dict(batch=1 << 20, channels=1 << 20), dict(x=None), dict(forget=None),
    dict(x=P + 1), dict(gate=P + 1), dict(state=P + 2), dict(lengths=P + 1), dict(saved=P + 2), dict(ws=None),
    dict(ws=P + 8), dict(x_stride_time=-1), dict(forget_stride_entry=-40), dict(gate_stride_time=-1)])
def test_recurrence_refuses(kw, backward):
    assert recurrence(backward, **kw) == N.FM_E_INVAL
    assert b"gated recurrence" in N.lib.fm_last_error()


def test_recurrence_ends():
    for kw in (dict(y=None), dict(last_state=None), dict(last_state=P + 2), dict(y=P + 1)):
        assert recurrence(False, **kw) == N.FM_E_INVAL
    for kw in (dict(grad_y=None), dict(grad_x=None), dict(grad_forget=None), dict(grad_gate=None), dict(saved=None),
               dict(grad_y_stride_time=-1), dict(grad_x=P + 1), dict(grad_last=P + 1), dict(grad_state=P + 3)):
        assert recurrence(True, **kw) == N.FM_E_INVAL
    for kw in (dict(channels=(1 << 20) + 1), dict(x_stride_time=1 << 22), dict(forget_stride_time=1 << 40)):
        assert recurrence(False, **kw) == recurrence(True, **kw) == N.FM_E_UNSUPPORTED
    assert recurrence(True, grad_y_stride_time=1 << 22) == N.FM_E_UNSUPPORTED
    assert recurrence(batch=0, ws=None, x=None, y=None) == N.FM_OK  # nothing to do, nothing launched
    assert N.lib.fm_gated_recurrence_forward(None, None, None) == N.FM_E_INVAL
    assert N.lib.fm_gated_recurrence_workspace(None, 0) == N.FM_E_INVAL


@pytest.mark.parametrize("backward", [0, 1])
def test_recurrence_workspace_does_not_look_at_pointers_and_strides(backward):
    def size(**kw):
        return N.lib.fm_gated_recurrence_workspace(
            fill(N.RecurrenceArgs(), dict(dtype=N.FM_F32, batch=1, time=20000, channels=24), kw), backward)

    want = size()
    assert want > 0
    assert size(x=1, y=3, state=2, x_stride_time=-5, grad_y_stride_entry=-(1 << 40)) == want
    assert size(batch=-1) == N.FM_E_INVAL
    assert size(time=60) == 0


def rms(rows=4, width=8, x=P, stride=8, res=P, rstride=8, w=P, y=P, total=P, rstd=P, eps=1e-6, dtype=N.FM_F32,
        pdtype=N.FM_F32):
    return N.lib.fm_rms_norm_forward(x, stride, res, rstride, w, y, total, rstd, rows, width, eps, dtype, pdtype, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(dtype=N.FM_I16), dict(dtype=N.FM_BF16, pdtype=N.FM_F16),
    dict(x=None), dict(y=None), dict(res=None), dict(total=None), dict(eps=-1.0), dict(eps=math.nan),
    dict(eps=math.inf), dict(stride=-8), dict(rstride=-8), dict(x=P + 2), dict(y=P + 1), dict(res=P + 1),
    dict(total=P + 2), dict(rstd=P + 1), dict(w=P + 2)])
def test_rms_norm_refuses(kw):
    assert rms(**kw) == N.FM_E_INVAL
    assert b"rms norm" in N.lib.fm_last_error()


def test_rms_norm_limits():
    assert rms(width=(1 << 20) + 1) == N.FM_E_UNSUPPORTED
    assert rms(rows=0, x=None, y=None) == N.FM_OK

    def quantized(scale=P, out=N.FM_E4M3, q=P):
        return N.lib.fm_rms_norm_quantized(P, 8, None, 0, None, q, scale, None, 4, 8, 1e-6, N.FM_F16, N.FM_F32, out,
                                           None)

    for kw in (dict(scale=None), dict(out=N.FM_F16), dict(out=N.FM_I16), dict(q=None), dict(scale=P + 1)):
        assert quantized(**kw) == N.FM_E_INVAL
    assert N.lib.fm_rms_norm_backward_workspace(4, 0, N.FM_F32) == N.FM_E_INVAL
    assert N.lib.fm_rms_norm_backward_workspace(4, 8, N.FM_F32) == 0


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(dtype=7), dict(dtype=N.FM_F16, pdtype=N.FM_BF16), dict(dy=None), dict(s=None),
    dict(rstd=None), dict(dx=None), dict(ws=None, rows=5000), dict(ws=P + 4, rows=5000), dict(w=None),
    dict(stride=-1), dict(ds_stride=-1), dict(dx=P + 2), dict(ds=P + 1), dict(dw=P + 2)])
def test_rms_norm_backward_refuses(kw):
    a = dict(rows=4, width=8, dy=P, stride=8, s=P, ds=P, ds_stride=8, w=P, rstd=P, dx=P, dw=P, ws=P, dtype=N.FM_F32,
             pdtype=N.FM_F32)
    a.update(kw)
    assert N.lib.fm_rms_norm_backward(a["dy"], a["stride"], a["s"], a["stride"], a["ds"], a["ds_stride"], a["w"],
                                      a["rstd"], a["dx"], a["dw"], a["ws"], a["rows"], a["width"], a["dtype"],
                                      a["pdtype"], None) == N.FM_E_INVAL


def distill(backward=False, **kw):
    a = dict(x=P, stride=50000, inner=0, outer=0, ids=P, lps=P, loss=P, stats=P, grad=P, dx=P, ws=P, rows=4,
             vocab=50000, top=5, tau=1.0, rest=0, dtype=N.FM_F32)
    a.update(kw)
    head = (a["x"], a["stride"], a["inner"], a["outer"], a["ids"], a["lps"])
    tail = (a["rows"], a["vocab"], a["top"], a["tau"], a["rest"], a["dtype"], None)
    if backward:
        return N.lib.fm_distill_backward(*head, a["stats"], a["grad"], a["dx"], *tail)
    return N.lib.fm_distill(*head, a["loss"], a["stats"], a["ws"], *tail)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 31) - 65536), dict(top=0), dict(top=65),
    dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan), dict(tau=math.inf), dict(tau=1e4), dict(rest=1, tau=2.0),
    dict(dtype=N.FM_I16), dict(x=None), dict(ids=None), dict(lps=None), dict(stride=-1), dict(inner=-1),
    dict(inner=1 << 31), dict(inner=2, outer=-8), dict(x=P + 2), dict(ids=P + 4), dict(lps=P + 2)])
def test_distillation_refuses(kw, backward):
    assert distill(backward, **kw) == N.FM_E_INVAL
    assert b"distillation" in N.lib.fm_last_error()


def test_distillation_ends():
    for kw in (dict(loss=None), dict(loss=P + 2), dict(ws=None), dict(ws=P + 8)):
        assert distill(**kw) == N.FM_E_INVAL
    for kw in (dict(stats=None), dict(grad=None), dict(dx=None), dict(dx=P + 1), dict(grad=P + 2)):
        assert distill(True, **kw) == N.FM_E_INVAL
    assert distill(rows=0, x=None, ids=None, ws=None) == N.FM_OK
    assert distill(True, rows=0, x=None) == N.FM_OK
    assert N.lib.fm_distill_workspace(-1, 10, N.FM_F32) == N.FM_E_INVAL


@pytest.mark.parametrize("kw", [
    dict(dtype=N.FM_I16), dict(rows=-1), dict(rows=1 << 31), dict(rows=1 << 22, vocab=1 << 20), dict(vocab=0),
    dict(vocab=(1 << 31) - 65536), dict(history_len=-1), dict(history_bits=16),
    dict(biases=-1), dict(x=None), dict(out=None), dict(history=None), dict(bias=None), dict(bias_ids=None),
    dict(repetition=None, repetition_value=0.0), dict(repetition=None, repetition_value=-2.0),
    dict(repetition=None, repetition_value=math.nan), dict(frequency=None, frequency_value=math.inf),
    dict(presence=None, presence_value=math.nan), dict(x_stride=-1), dict(history_stride=-1),
    dict(allowed_stride=-1), dict(x=P + 1), dict(history=P + 4), dict(bias=P + 2), dict(allowed=P + 2),
    dict(history_lengths=P + 1), dict(bias_ids=P + 4)])
def test_adjusted_logits_refuse(kw):
    names = ("x", "out", "history", "history_lengths", "prompt_lengths", "repetition", "frequency", "presence",
             "bias_ids", "bias", "allowed")
    base = dict(dtype=N.FM_F16, history_bits=64, rows=3, vocab=100, history_len=7, biases=2, x_stride=100,
                history_stride=7, allowed_stride=4, repetition_value=1.0, **{n: P for n in names})
    assert N.lib.fm_adjust_logits(fill(N.AdjustArgs(), base, kw), None) == N.FM_E_INVAL
    assert b"adjusted logits" in N.lib.fm_last_error()


def test_adjusted_logits_limits():
    base = dict(dtype=N.FM_F16, history_bits=64, rows=3, vocab=100, biases=1025, repetition_value=1.0, x=P, out=P,
                bias=P, bias_ids=P)
    assert N.lib.fm_adjust_logits(fill(N.AdjustArgs(), base, {}), None) == N.FM_E_UNSUPPORTED
    assert N.lib.fm_adjust_logits(fill(N.AdjustArgs(), base, dict(biases=0, history_len=1 << 20, history=P)),
                                  None) == N.FM_E_UNSUPPORTED
    assert N.lib.fm_adjust_logits(fill(N.AdjustArgs(), base, dict(history_len=0, rows=0, x=None)), None) == N.FM_OK
    assert N.lib.fm_adjust_logits(None, None) == N.FM_E_INVAL


def test_python_callers_refuse_tensors_off_the_gpu():
    from stft_mel_spectrogram_amd import (adjust_logits, gated_recurrence, rms_norm, rms_norm_quantized,
                                          topk_distillation)
    x = torch.zeros(2, 4, 8)
    for call in (lambda: gated_recurrence(x, x), lambda: rms_norm(x), lambda: rms_norm_quantized(x),
                 lambda: topk_distillation(x, x.long(), x), lambda: adjust_logits(x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (gated_recurrence, rms_norm, topk_distillation, adjust_logits):
        with pytest.raises(ValueError, match="tensor"):
            call(*[[1.0]] * (3 if call is topk_distillation else 2 if call is gated_recurrence else 1))


def test_tangents_are_refused_before_any_launch():
    from torch.autograd import forward_ad
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence, rms_norm, topk_distillation
    x = torch.zeros(2, 4, 8)
    for call in (lambda v: gated_recurrence(v, x), rms_norm, lambda v: topk_distillation(v, x.long(), x),
                 adjust_logits):
        with forward_ad.dual_level():
            with pytest.raises(NotImplementedError, match="tangent"):
                call(forward_ad.make_dual(x, torch.ones_like(x)))
