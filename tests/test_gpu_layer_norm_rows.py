"""Layer norm of more wide rows than one launch takes: 2^22 rows of 1024 lanes are
2^32 threads, more than a grid may have.  All rows are one (stride 0), the results
69 GB."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free memory")
    yield
    torch.cuda.empty_cache()


def test_more_wide_rows_than_one_launch_takes():
    from stft_mel_spectrogram_amd import layer_norm_backward, layer_norm_forward
    rows, width = (1 << 22) + 3, 8193
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    one = torch.randn(1, width, generator=g, device="cuda").half()
    dy = torch.randn(1, width, generator=g, device="cuda").half()
    some = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, 1 << 22, rows - 1], device="cuda")
    want, mean, rstd = layer_norm_forward(one)
    y, means, rstds = layer_norm_forward(one.expand(rows, width))
    assert bool((means == mean).all()) and bool((rstds == rstd).all())
    assert bool((y[some] == want).all())
    del y
    want = layer_norm_backward(dy, one, None, mean, rstd)[0]
    dx = layer_norm_backward(dy.expand(rows, width), one.expand(rows, width), None, means, rstds)[0]
    assert bool((dx[some] == want).all())
