"""eps of the RMS norm is a float32 number: a double beyond is refused (on the CPU, by
calls of no rows)."""
import pytest

torch = pytest.importorskip("torch")  # before the library, which then takes torch's HIP runtime
from stft_mel_spectrogram_amd import _native as N  # noqa: E402


def call(eps):
    return (N.lib.fm_rms_norm_forward(None, 8, None, 0, None, None, None, None, 0, 8, eps, N.FM_F32, N.FM_F32, None),
            N.lib.fm_rms_norm_quantized(None, 8, None, 0, None, None, None, None, 0, 8, eps, N.FM_F32, N.FM_F32,
                                        N.FM_I8, None))


@pytest.mark.parametrize("eps", [1e39, 1e300])
def test_past_float32(eps):
    assert call(eps) == (N.FM_E_INVAL, N.FM_E_INVAL)
    assert b"float32" in N.lib.fm_last_error()


@pytest.mark.parametrize("eps", [0.0, 1e-300, 1e-46, 1e-6, 3e38])
def test_within(eps):
    assert call(eps) == (N.FM_OK, N.FM_OK)


@pytest.mark.gpu
def test_a_small_one_is_not_none():
    """Rows of zeros stay zeros with any eps above 0."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_quantized
    for width in (64, 20000):
        x = torch.zeros(2, width, device="cuda")
        x[1] = 3.0
        for eps in (1e-6, 1e-46, 1e-300):
            y = rms_norm(x, eps=eps)
            assert (y[0] == 0).all() and (y[1] - 1).abs().max() <= 2.0 ** -18
            q, scale = rms_norm_quantized(x, eps=eps)
            assert scale[0] == 1 and (q[0].float() == 0).all() and torch.isfinite(q.float()).all()
