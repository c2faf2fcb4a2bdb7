"""A gradient that an operator does not have is refused, not lost without a word."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_a_teachers():
    """Also where the logits' gradient is wanted."""
    from stft_mel_spectrogram_amd import topk_distillation
    x = torch.randn(4, 50, device="cuda")
    ids, lps = x.topk(5)[1], torch.log_softmax(x, -1).topk(5)[0]
    for logits in (x, x.clone().requires_grad_(True)):
        with pytest.raises(ValueError, match="detach"):
            topk_distillation(logits, ids, lps.clone().requires_grad_(True))
        topk_distillation(logits, ids, lps)
    with torch.no_grad():
        topk_distillation(x, ids, lps.clone().requires_grad_(True))
