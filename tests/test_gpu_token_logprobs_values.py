"""Token log probabilities: the precision of the logits' gradient, vocabularies
and row counts near the documented ends."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("rows,vocab", [(4000, 8), (500, 129), (40, 1025), (3, 50001)])
def test_gradient_keeps_float32_precision(rows, vocab):
    """Of a given lse, so that its own rounding does not enter.  The exponential's argument rounds
    three times (x - lse, the factor log2 e and the product), each by U of itself, its result by 2 U,
    and so do the products with the gradient."""
    from stft_mel_spectrogram_amd import token_logprobs_backward
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 1.5
    x = torch.log_softmax(x.double(), -1).float()
    lse = torch.logsumexp(x.double(), -1).float()  # about 0
    tok = torch.full((rows,), -1, device="cuda")
    tok[0] = 0
    g_top = torch.randn(rows, 1, generator=g, device="cuda")
    ids = torch.full((rows, 1), vocab - 1, device="cuda")
    ent = torch.zeros(rows, device="cuda")
    dx = token_logprobs_backward(x, tok, lse, ent, torch.zeros(rows, device="cuda"), None, ids, g_top)
    lp = x.double() - lse.double()[:, None]
    ref = -g_top.double() * lp.exp()
    tol = U * (3 * lp.abs() + 6) * ref.abs()
    ref[:, vocab - 1] += g_top.double()[:, 0]
    tol[:, vocab - 1] += 2 * U * g_top.double().abs()[:, 0]
    worst = ((dx.double() - ref).abs() / (tol + 1e-37)).max().item()
    print(f"worst error / tolerance {worst:.3g}")
    assert worst <= 1


def test_gradient_lifts_probabilities_below_float32s_range():
    """-p g and -p g_H (lp + H) with p down to 2^-185."""
    from stft_mel_spectrogram_amd import token_logprobs_backward
    for vocab in (40, 3000):
        x = torch.zeros(2, vocab, device="cuda")
        x[:, 1:] = -torch.linspace(60, 128, vocab - 1, device="cuda")
        x[:, 7] = -math.inf
        lse, ent = torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")
        tok = torch.zeros(2, dtype=torch.int64, device="cuda")
        big = torch.full((2,), 2.0 ** 100, device="cuda")
        dx = token_logprobs_backward(x, tok, lse, ent, big, None)
        lp = x.double()
        ref = -2.0 ** 100 * lp.exp()
        tol = U * (3 * lp.abs() + 6) * ref.abs()
        keep = torch.isfinite(lp) & (lp < 0)
        assert ((dx.double() - ref).abs() <= tol + 1e-44)[keep].all()
        assert (dx[:, 7] == 0).all()
        dx = token_logprobs_backward(x, tok, lse, ent, None, big)
        ref = -2.0 ** 100 * lp.exp() * lp
        tol = U * (3 * lp.abs() + 10) * ref.abs()
        assert ((dx.double() - ref).abs() <= tol + 1e-44)[keep].all()
        assert (dx[:, 7] == 0).all()


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


def test_more_rows_than_one_launch_takes():
    """2^26 rows of 64 lanes are 2^32 threads, more than a grid may have."""
    from stft_mel_spectrogram_amd import token_logprobs
    rows = (1 << 26) + 5
    x = torch.zeros(rows, 2, dtype=torch.float16, device="cuda")
    x[:, 1] = 1.0
    x[rows - 3:] = torch.tensor([3.0, 0.0], device="cuda")
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    r = token_logprobs(x, tok, 1)
    assert bool((r.top_ids[:rows - 3] == 1).all()) and bool((r.top_ids[rows - 3:] == 0).all())
    want = -math.log1p(math.e)
    assert bool(((r.logprobs[:rows - 3] - want).abs() <= 1e-6).all())
    assert bool(((r.logprobs[rows - 3:] + math.log1p(math.exp(-3.0))).abs() <= 1e-6).all())


def test_more_rows_than_one_gradient_launch_takes():
    """2^28 rows of 16 lanes."""
    from stft_mel_spectrogram_amd import token_logprobs_backward
    rows = (1 << 28) + 5
    x = torch.zeros(rows, 2, dtype=torch.float16, device="cuda")
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tok[rows - 3:] = 1
    lse = torch.full((rows,), math.log(2.0), device="cuda")
    g = torch.ones(rows, device="cuda")
    dx = token_logprobs_backward(x, tok, lse, lse, g)
    assert bool((dx[:rows - 3, 0] == 0.5).all()) and bool((dx[:rows - 3, 1] == -0.5).all())
    assert dx[rows - 3:].tolist() == [[-0.5, 0.5]] * 3
