"""Forward-mode derivatives are refused, not dropped, by the operators' callers."""
import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad  # noqa: E402


def calls(device):
    """(tensors, call) of each operator; every floating tensor may carry a tangent."""
    from stft_mel_spectrogram_amd import (layer_norm, layer_norm_backward, relative_attention,
                                          relative_attention_backward, token_logprobs, token_logprobs_backward)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(device)  # noqa: E731
    m = torch.zeros(3, dtype=torch.int32, device=device)
    tok = torch.zeros(4, dtype=torch.int64, device=device)
    one = torch.ones(4, device=device)
    return [
        ([r(4, 8), r(8), r(8)], layer_norm),
        ([r(4, 8), r(4, 8), r(8), one, one], layer_norm_backward),
        ([r(4, 9)], lambda x: token_logprobs(x, tok, 2)),
        ([r(4, 9), one, one, one], lambda x, lse, ent, g: token_logprobs_backward(x, tok, lse, ent, g)),
        ([r(1, 2, 4, 8), r(1, 2, 5, 8), r(1, 2, 5, 8), r(3, 2)],
         lambda q, k, v, t: relative_attention(q, k, v, t, m)),
        ([r(1, 2, 4, 8), r(1, 2, 4, 8), r(1, 2, 5, 8), r(1, 2, 5, 8), r(3, 2), r(1, 2, 4, 8), r(1, 2, 4)],
         lambda g, q, k, v, t, o, lse: relative_attention_backward(g, q, k, v, t, m, o, lse)),
    ]


def test_tangents_are_refused_before_any_launch():
    """On the CPU: the first tensor's, which is looked at before its device."""
    for which, (xs, call) in enumerate(calls("cpu")):
        with forward_ad.dual_level():
            at = 1 if which in (1, 5) else 0  # x, q: the first tensor that is checked
            xs = [forward_ad.make_dual(x, torch.ones_like(x)) if i == at else x for i, x in enumerate(xs)]
            with pytest.raises(NotImplementedError, match="tangent"):
                call(*xs)
        with pytest.raises(ValueError, match="GPU"):
            call(*calls("cpu")[which][0])


@pytest.mark.gpu
def test_every_tensors_tangent_is_refused():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for xs, call in calls("cuda"):
        call(*xs)  # without tangents
        with forward_ad.dual_level():
            call(*xs)  # inside a level, still without
            for i in range(len(xs)):
                ys = [forward_ad.make_dual(x, torch.ones_like(x)) if j == i else x for j, x in enumerate(xs)]
                with pytest.raises(NotImplementedError):
                    call(*ys)
                ys[i] = forward_ad.make_dual(xs[i].clone().requires_grad_(True), torch.ones_like(xs[i]))
                with pytest.raises(NotImplementedError):
                    call(*ys)
