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


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence", "bias"])
def test_penalties_and_biases(name):
    from stft_mel_spectrogram_amd import adjust_logits
    x = torch.randn(4, 50, device="cuda")
    h = torch.zeros(4, 3, dtype=torch.int64, device="cuda")
    kw = dict(repetition=torch.ones(4, device="cuda"), frequency=torch.ones(4, device="cuda"),
              presence=torch.ones(4, device="cuda"), bias_ids=h, bias=torch.ones(4, 3, device="cuda"))
    want = adjust_logits(x, h, **kw)
    kw[name] = kw[name].clone().requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        adjust_logits(x, h, **kw)
    with torch.no_grad():
        assert torch.equal(adjust_logits(x, h, **kw), want)
