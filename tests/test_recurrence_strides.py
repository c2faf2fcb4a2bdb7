"""Strides in time that no address is made of are not looked at (on the CPU: calls
of no entries, which are checked and launch nothing)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")  # before the library, which then takes torch's HIP runtime
from stft_mel_spectrogram_amd import _native as N  # noqa: E402

P = 1 << 20  # an address that must not be touched
FAR = 1 << 40


def call(time, backward=False, saved=P, **strides):
    a = N.RecurrenceArgs()
    for name in ("x", "forget", "gate", "state", "y", "last_state", "grad_y", "grad_last", "grad_x", "grad_forget",
                 "grad_gate", "grad_state"):
        setattr(a, name, P)
    a.dtype, a.batch, a.time, a.channels, a.saved = N.FM_BF16, 0, time, 40, saved
    for name, v in strides.items():
        setattr(a, name, v)
    fn = N.lib.fm_gated_recurrence_backward if backward else N.lib.fm_gated_recurrence_forward
    return fn(ctypes.byref(a), P, None)


@pytest.mark.parametrize("name", ["x_stride_time", "forget_stride_time", "gate_stride_time", "grad_y_stride_time"])
def test_strides_of_few_frames(name):
    for time in (0, 1):
        assert call(time, **{name: FAR}) == call(time, True, **{name: FAR}) == N.FM_OK
        assert call(time, saved=None, **{name: FAR}) == N.FM_OK
    assert call(2, saved=None, **{name: FAR}) == N.FM_OK  # single steps
    assert call(2, True, **{name: FAR}) == N.FM_E_UNSUPPORTED
    assert call(3, True, **{name: FAR}) == N.FM_E_UNSUPPORTED
    if name != "grad_y_stride_time":
        assert call(2, **{name: FAR}) == call(3, saved=None, **{name: FAR}) == N.FM_E_UNSUPPORTED
