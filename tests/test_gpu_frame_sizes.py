"""Tensors of more than 2^31 elements: their ends against the same call on the
ends alone (bit for bit where the work is split alike), and calls of several
streams at once."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def randn(*shape):
    return torch.randn(*shape, device="cuda", dtype=BF)


def near(a, b):
    """Two roundings of values that differ by far less than a step: one step apart at most."""
    a, b = a.double(), b.double()
    return ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14).all()


def test_recurrence():
    from stft_mel_spectrogram_amd import gated_recurrence_backward, gated_recurrence_forward
    b, t, c = 2, 40000, 28000
    x, f, g, dy = (randn(b, t, c) for _ in range(4))
    assert x.numel() > 1 << 31
    f += 2
    n = torch.tensor([t, t - 700], dtype=torch.int32, device="cuda")
    y, last, saved = gated_recurrence_forward(x, f, g, lengths=n)
    dx, df, dg, _ = gated_recurrence_backward(dy, x, f, g, None, saved, lengths=n)
    for part in (slice(0, 40), slice(c - 37, c)):
        sl = [v[..., part].contiguous() for v in (x, f, g, dy)]
        y2, last2, saved2 = gated_recurrence_forward(*sl[:3], lengths=n)
        grads = gated_recurrence_backward(sl[3], *sl[:3], None, saved2, lengths=n)
        assert near(y[..., part], y2) and near(dx[..., part], grads[0])
        assert near(df[..., part], grads[1]) and near(dg[..., part], grads[2])
        assert (last[:, part] - last2).abs().max() <= 2.0 ** -18


def test_rms_norm():
    from stft_mel_spectrogram_amd import rms_norm_backward, rms_norm_forward, rms_norm_quantized
    x, r = randn(300000, 8000), randn(300000, 8000)
    assert x.numel() > 1 << 31
    w = randn(8000)
    y, total, rstd = rms_norm_forward(x, w, r)
    dx, _ = rms_norm_backward(r, total, w, rstd, x)
    q, scale = rms_norm_quantized(total, w)
    y2, total2, rstd2 = rms_norm_forward(x[-5:], w, r[-5:])
    assert torch.equal(y[-5:], y2) and torch.equal(total[-5:], total2)
    assert torch.equal(dx[-5:], rms_norm_backward(r[-5:], total2, w, rstd2, x[-5:])[0])
    q2, scale2 = rms_norm_quantized(total2, w)
    assert torch.equal(q[-5:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale[-5:], scale2)


def test_logits():
    from stft_mel_spectrogram_amd import adjust_logits, topk_distillation_backward, topk_distillation_forward
    rows, vocab, end = 17000, 131072, 2000
    x = randn(rows, vocab)
    assert x.numel() > 1 << 31
    ids = torch.randint(0, vocab, (rows, 5), device="cuda")
    lps = torch.log_softmax(torch.randn(rows, 5, device="cuda"), -1) - 0.3
    g = torch.randn(rows, device="cuda")
    loss, stats = topk_distillation_forward(x, ids, lps, rest=True)
    dx = topk_distillation_backward(g, x, ids, lps, stats, rest=True)
    loss2, stats2 = topk_distillation_forward(x[-end:], ids[-end:], lps[-end:], rest=True)
    assert torch.equal(loss[-end:], loss2)
    assert torch.equal(dx[-end:], topk_distillation_backward(g[-end:], x[-end:], ids[-end:], lps[-end:], stats2,
                                                             rest=True))
    del dx
    out = adjust_logits(x, ids, repetition=1.5, bias_ids=ids, bias=lps)
    assert torch.equal(out[-end:], adjust_logits(x[-end:], ids[-end:], repetition=1.5, bias_ids=ids[-end:],
                                                 bias=lps[-end:]))
    assert adjust_logits(x, out=x[:]).data_ptr() == x.data_ptr()


def test_streams_at_once():
    from stft_mel_spectrogram_amd import adjust_logits, gated_recurrence, rms_norm, topk_distillation
    x, f = randn(2, 3000, 60), randn(2, 3000, 60)
    z = randn(4, 20011)
    ids = torch.randint(0, 20011, (4, 9), device="cuda")
    lps = torch.log_softmax(torch.randn(4, 9, device="cuda"), -1) - 0.3
    run = lambda: (*gated_recurrence(x, f), rms_norm(x), topk_distillation(z, ids, lps, rest=True),  # noqa: E731
                   adjust_logits(z, ids, frequency=0.5))
    want = run()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
