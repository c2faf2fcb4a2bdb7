"""Token log probabilities: the precision of the logits' gradient, vocabularies
and row counts near the documented ends."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_the_largest_vocabulary():
    """One row of 2^31 - 65537 entries: the last segment ends with the row."""
    from stft_mel_spectrogram_amd import token_logprobs_backward, token_logprobs_forward
    vocab = (1 << 31) - 65537
    x = torch.zeros(1, vocab, dtype=torch.float16, device="cuda")
    x[0, vocab - 1] = 5.0
    tok = torch.tensor([vocab - 1], device="cuda")
    r, lse = token_logprobs_forward(x, tok, 2)
    want = math.log((vocab - 1) + math.exp(5.0))
    tol = 2.0 ** -23 * (want + vocab / (1280 * 256) + 2000)
    assert r.top_ids.tolist() == [[vocab - 1, 0]]
    assert abs(lse.item() - want) <= tol
    assert abs(r.logprobs.item() - (5.0 - want)) <= tol
    p = math.exp(5.0 - want)
    assert abs(r.entropy.item() - (want - 5.0 * p)) <= 2 * tol
    g = 2.0 ** 14
    dx = token_logprobs_backward(x, tok, lse, r.entropy, torch.full((1,), g, device="cuda"))
    assert abs(dx[0, vocab - 1].item() - g * (1 - p)) <= 2.0 ** -10 * g
    # the other gradients are subnormal in float16
    tail = dx[0, vocab - 20000:vocab - 1].double()
    assert ((tail + g * math.exp(-want)).abs() <= 2.0 ** -25 + 2 * tol * g * math.exp(-want)).all()
