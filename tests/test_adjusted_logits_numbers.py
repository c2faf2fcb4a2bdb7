"""Penalties given as numbers have to be float32 numbers: a double beyond would reach
the kernel as 0 or infinity.  On the CPU, by calls of no rows."""
import ctypes

import pytest

torch = pytest.importorskip("torch")  # before the library, which then takes torch's HIP runtime
from stft_mel_spectrogram_amd import _native as N  # noqa: E402


def call(**kw):
    a = N.AdjustArgs()
    base = dict(dtype=N.FM_F32, history_bits=64, rows=0, vocab=100, repetition_value=1.0)
    for name, v in (base | kw).items():
        setattr(a, name, v)
    return N.lib.fm_adjust_logits(ctypes.byref(a), None)


@pytest.mark.parametrize("kw", [
    dict(repetition_value=1e-46), dict(repetition_value=1e-40), dict(repetition_value=1e39),
    dict(frequency_value=1e39), dict(frequency_value=-1e300), dict(presence_value=4e38)])
def test_numbers_past_float32_are_refused(kw):
    assert call(**kw) == N.FM_E_INVAL
    assert b"float32" in N.lib.fm_last_error()


@pytest.mark.parametrize("kw", [
    dict(repetition_value=1e-38), dict(repetition_value=3e38), dict(frequency_value=-3e38), dict(presence_value=1e-60)])
def test_numbers_within_are_not(kw):
    assert call(**kw) == N.FM_OK
