"""The 8-bit RMS norm bit for bit: in single float32 steps y = s / sqrt(mean(s^2) +
eps) * weight, scale = max |y| / 448 (127) and y / scale, rounded to nearest with ties
to even.  Rows of small whole numbers: their sums of squares stay below 2^24 and are
exact in any order, and every other step is one correctly rounded operation.  Short
numbers often have quotients halfway between two 8-bit values, which one rounding
more (y times 1 / scale, s times 1 / sqrt) puts on the wrong side.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("width,most", [(40, 60), (129, 60), (1000, 60), (4096, 60), (8192, 40), (16390, 30)])
def test_every_rounding(width, most, dtype, out):
    from stft_mel_spectrogram_amd import rms_norm_quantized
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    rows = 400000 // width + 3
    s = torch.randint(-most, most + 1, (rows, width), generator=g, device="cuda").to(dtype)
    w = (torch.randn(width, generator=g, device="cuda") * 0.2 + 1).to(dtype)
    q, scale = rms_norm_quantized(s, w, None, 1e-6, out)
    f = np.float32  # numpy's float32 quotients and roots are rounded correctly (torch's roots are not)
    z = s.cpu().float().numpy()
    total = np.square(z, dtype=np.float64).sum(-1, keepdims=True)
    assert total.max() < 2 ** 24
    y = z / np.sqrt(total.astype(f) / f(width) + f(1e-6)) * w.cpu().float().numpy()
    want = np.abs(y).max(-1, keepdims=True) / f(448 if out == torch.float8_e4m3fn else 127)
    assert y.dtype == want.dtype == f
    assert np.array_equal(scale.cpu().numpy(), want[:, 0])
    v = torch.from_numpy(y / want)
    v = v.to(out).float() if out == torch.float8_e4m3fn else v.round().clamp(-127, 127)
    assert torch.equal(q.cpu().float(), v)


def test_rows_without_a_finite_root():
    """A sum of squares past float32 gives zeros, as s / inf does; a weight of inf a
    scale that is not finite, and nothing for the other columns' values."""
    from stft_mel_spectrogram_amd import rms_norm_quantized
    for width in (64, 9000):
        x = torch.full((2, width), 1e30, device="cuda")
        x[1] = 2.0
        w = torch.ones(width, device="cuda")
        for out in (torch.float8_e4m3fn, torch.int8):
            q, scale = rms_norm_quantized(x, w, None, 1e-6, out)
            assert scale[0] == 1 and (q[0].float() == 0).all() and torch.isfinite(q.float()).all()
            hot = w.clone()
            hot[3] = float("inf")
            q, scale = rms_norm_quantized(x[1:], hot, None, 1e-6, out)
            assert scale[0] == float("inf")
            keep = torch.arange(width, device="cuda") != 3
            assert (q[0].float()[keep] == 0).all()
