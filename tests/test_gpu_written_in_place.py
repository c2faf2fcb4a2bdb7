"""What an operator writes into given memory counts as changed: a backward that saved
the old values says so instead of computing with the new ones."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_a_backward_that_needs_the_old_values():
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence, rms_norm
    a = torch.randn(4, 40, device="cuda", requires_grad=True)
    y = a.exp()  # keeps its result
    with torch.no_grad():
        adjust_logits(y, allowed=torch.zeros(2, dtype=torch.int32, device="cuda"), out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = a.exp()
    with torch.no_grad():
        rms_norm(torch.ones_like(a), None, y, out_sum=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = a.exp()
    x = torch.randn(4, 3, 40, device="cuda")
    with torch.no_grad():
        gated_recurrence(x, x, None, y, out_state=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_every_given_result():
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence, rms_norm, rms_norm_quantized
    x, r = torch.randn(4, 40, device="cuda"), torch.randn(4, 40, device="cuda")
    x3, state = torch.randn(2, 3, 40, device="cuda"), torch.randn(2, 40, device="cuda")
    calls = [lambda o: adjust_logits(x, out=o), lambda o: rms_norm(x, out=o), lambda o: rms_norm(x, None, r, out_sum=o),
             lambda o: rms_norm_quantized(x, None, r, out_sum=o)]
    for call in calls:
        o = torch.empty_like(x)
        before = o._version
        call(o)
        assert o._version > before
    o, s = torch.empty_like(x3), state.clone()
    before = o._version, s._version
    gated_recurrence(x3, x3, None, s, out=o, out_state=s)
    assert o._version > before[0] and s._version > before[1]


def test_inference_tensors():
    """They have no version to count and are written all the same."""
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence
    with torch.inference_mode():
        x = torch.randn(4, 40, device="cuda")
        want = adjust_logits(x, allowed=torch.ones(2, dtype=torch.int32, device="cuda"))
        assert torch.equal(adjust_logits(x, allowed=torch.ones(2, dtype=torch.int32, device="cuda"), out=x), want)
        s = torch.zeros(2, 40, device="cuda")
        x3 = torch.randn(2, 3, 40, device="cuda")
        assert gated_recurrence(x3, x3, None, s, out_state=s)[1] is s


def test_a_leafs_memory_is_refused():
    """As torch refuses out= tensors that require grad."""
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence, rms_norm, rms_norm_quantized
    x, x3 = torch.randn(4, 40, device="cuda"), torch.randn(2, 3, 40, device="cuda")
    o = torch.empty_like(x).requires_grad_(True)
    o3, s = torch.empty_like(x3).requires_grad_(True), torch.empty(2, 40, device="cuda").requires_grad_(True)
    calls = [lambda: adjust_logits(x, out=o), lambda: rms_norm(x, out=o), lambda: rms_norm(x, None, x, out_sum=o),
             lambda: rms_norm_quantized(x, None, x, out_sum=o), lambda: gated_recurrence(x3, x3, out=o3),
             lambda: gated_recurrence(x3, x3, out_state=s)]
    for call in calls:
        with pytest.raises(ValueError, match="grad"):
            call()
        with torch.no_grad():
            call()
