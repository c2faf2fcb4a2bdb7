"""What the torch-facing callers of the operators refuse, before any launch."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_layer_norm():
    from stft_mel_spectrogram_amd import layer_norm, layer_norm_backward, layer_norm_forward
    x, w, b = t(4, 8), t(8), t(8)
    for args, err in (((x.int(),), TypeError), ((x.t(), t(4)), ValueError), ((t(4, 0),), ValueError),
                      ((x, t(7)), ValueError), ((x, w.half()), TypeError), ((x, w, b.float()), TypeError),
                      ((x, None, b), ValueError), ((x, w.cpu()), ValueError), ((x, w, t(9)), ValueError),
                      ((t(2, 3, 4)[:, ::2].expand(2, 2, 4)[:, :, ::2],), ValueError),
                      ((t(4, 6, 8)[:, :5],), ValueError)):
        with pytest.raises(err):
            layer_norm(*args)
    with pytest.raises(ValueError):
        layer_norm(x, w, b, out=t(4, 9))
    with pytest.raises(ValueError):
        layer_norm(x, w.requires_grad_(True), b, out=t(4, 8))
    w = w.detach()
    _, mean, rstd = layer_norm_forward(x, w, b)
    for bad in ((t(4, 9), x, w, mean, rstd), (x.float(), x, w, mean, rstd), (x, x, w, mean[:3], rstd),
                (x, x, w, mean, rstd.cpu()), (x.t().contiguous().t(), x, w, mean, rstd)):
        with pytest.raises(ValueError):
            layer_norm_backward(*bad)


def test_token_logprobs():
    from stft_mel_spectrogram_amd import token_logprobs, token_logprobs_backward
    x, tok = t(4, 50), t(4, dtype=torch.int64)
    for args, err in (((x.double(), tok), TypeError), ((x, tok.int().short()), TypeError), ((x, tok[:3]), ValueError),
                      ((x, tok, 51), ValueError), ((x, tok, -1), ValueError), ((t(4, 80), tok, 65), ValueError),
                      ((x, tok.cpu()), ValueError), ((x[:, ::2], tok), ValueError)):
        with pytest.raises(err):
            token_logprobs(*args)
    f = t(4, dtype=torch.float32)
    with pytest.raises(TypeError):
        token_logprobs_backward(x, tok, f.double(), f, f)
    with pytest.raises(ValueError):
        token_logprobs_backward(x, tok, f, f, f[:2])
    with pytest.raises(ValueError):
        token_logprobs_backward(x, tok, f, f, grad_top_logprobs=t(4, 2, dtype=torch.float32))


def test_relative_attention():
    from stft_mel_spectrogram_amd import (relative_attention, relative_attention_backward,
                                          relative_attention_forward)
    q, k, v = t(2, 4, 6, 16), t(2, 2, 9, 16), t(2, 2, 9, 16)
    table, m = t(8, 4), t(7, dtype=torch.int32)

    def refuse(err, *args, **kw):
        with pytest.raises(err):
            relative_attention(*args, **kw)

    refuse(ValueError, q[0], k, v, table, m)
    refuse(TypeError, q, k.half(), v, table, m)
    refuse(ValueError, q, k, v[:, :, :5], table, m)
    refuse(ValueError, q, t(2, 3, 9, 16), t(2, 3, 9, 16), table, m)
    refuse(ValueError, t(2, 4, 6, 130), t(2, 2, 9, 130), t(2, 2, 9, 130), table, m)
    refuse(ValueError, q.transpose(2, 3), k, v, table, m)
    refuse(ValueError, q, k, v, t(8, 3), m)
    refuse(TypeError, q, k, v, table.half(), m)
    refuse(TypeError, q, k, v, table, m.long())
    refuse(ValueError, q, k, v, table, m[:6])
    refuse(ValueError, q, k, v, table, m, key_lengths=t(3, dtype=torch.int32))
    refuse(ValueError, q, k, v, table, m, key_lengths=t(2, dtype=torch.int64))
    refuse(ValueError, q, k, v, table, m, query_offset=t(2, dtype=torch.int64))
    refuse(ValueError, q, k, v, table, m, out=t(2, 4, 6, 15))
    refuse(ValueError, q.clone().requires_grad_(True), k, v, table, m, out=t(2, 4, 6, 16))
    refuse(RuntimeError, q, k, v, table, m, scale=-1.0)
    refuse(ValueError, q, k.cpu(), v, table, m)
    o, stats = relative_attention_forward(q, k, v, table, m)
    with pytest.raises(ValueError):
        relative_attention_backward(o[:1], q, k, v, table, m, o, stats)
    with pytest.raises(ValueError):
        relative_attention_backward(o.float(), q, k, v, table, m, o, stats)
