"""A tensor that is missing is refused by name, like one of another device."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def refuses(fn, args, optional, **kw):
    fn(*args, **kw)
    for i in range(len(args)):
        with_none = [None if j == i else a for j, a in enumerate(args)]
        if i in optional:
            fn(*with_none, **kw)
            continue
        for bad in (None, 3.0):
            with pytest.raises(ValueError):
                fn(*(bad if j == i else a for j, a in enumerate(args)), **kw)


def test_missing_tensors():
    from stft_mel_spectrogram_amd import (layer_norm, layer_norm_backward, layer_norm_forward, relative_attention,
                                          relative_attention_backward, relative_attention_forward, token_logprobs,
                                          token_logprobs_backward, token_logprobs_forward)
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    refuses(layer_norm, (x, w), (1,))
    for args in ((x, None, w), (x, 3.0, w), (x, w, 3.0)):
        with pytest.raises(ValueError):
            layer_norm(*args)
    _, mean, rstd = layer_norm_forward(x, w, w)
    refuses(layer_norm_backward, (x, x, w, mean, rstd), (2,))
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    refuses(token_logprobs, (x, tok), (), top_k=2)
    r, lse = token_logprobs_forward(x, tok, 2)
    refuses(token_logprobs_backward, (x, tok, lse, r.entropy, lse, lse, r.top_ids, r.top_logprobs), (4, 5, 7))
    q, k = torch.ones(1, 2, 3, 8, device="cuda"), torch.ones(1, 2, 5, 8, device="cuda")
    table, m = torch.ones(4, 2, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    refuses(relative_attention, (q, k, k, table, m), ())
    o, stats = relative_attention_forward(q, k, k, table, m)
    refuses(relative_attention_backward, (q, q, k, k, table, m, o, stats), ())
