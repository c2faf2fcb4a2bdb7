"""Logits and tokens of a slice, read as they lie: the same results, bit for bit,
as of contiguous copies."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def same(logits, tokens, top):
    from stft_mel_spectrogram_amd import (token_logprobs, token_logprobs_backward, token_logprobs_forward)
    lead = logits.shape[:-1]
    g = torch.Generator(device="cuda")
    g.manual_seed(logits.numel())
    grads = [torch.randn(lead, generator=g, device="cuda") for _ in range(2)]
    g_top = torch.randn((*lead, top), generator=g, device="cuda") if top else None
    results = []
    for x, t in ((logits, tokens), (logits.contiguous(), tokens.contiguous())):
        r, lse = token_logprobs_forward(x, t, top)
        dx = token_logprobs_backward(x, t, lse, r.entropy, *grads, r.top_ids, g_top)
        whole = x.detach().requires_grad_(True)
        a = token_logprobs(whole, t, top)
        total = (a.logprobs * grads[0]).sum() + (a.entropy * grads[1]).sum()
        if top:
            total = total + (a.top_logprobs * g_top).sum()
        auto, = torch.autograd.grad(total, whole)
        assert torch.equal(auto, dx)
        results.append([*r, lse, dx])
    for a, b in zip(*results):
        assert a is None and b is None or torch.equal(a, b)
        assert a is None or a.is_contiguous()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,t,vocab,top", [(3, 9, 37, 0), (3, 9, 37, 5), (5, 70, 129, 0), (2, 33, 1500, 3), (4, 6, 9001, 4),
                                           (2, 3, 50001, 20), (2, 400, 9001, 0), (1, 5, 300, 0), (6, 2, 300, 2)])
def test_shifted_targets(b, t, vocab, top, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    logits = (torch.randn(b, t, vocab, generator=g, device="cuda") * 2).to(dtype)
    logits[0, 0, 1::3] = -math.inf
    tokens = torch.randint(-1, vocab, (b, t), generator=g, device="cuda")
    same(logits[:, :-1], tokens[:, 1:], top)
    same(logits[:, 1:], tokens[:, 1:].int(), top)
    same(logits.transpose(0, 1), tokens.t(), top)
    # a group of groups that lie at two strides
    same(logits[:, ::2].unsqueeze(2), tokens[:, ::2].unsqueeze(2), top)


def test_wide_slices_and_shared_rows():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.randn(4, 7, 5, 100, generator=g, device="cuda")
    tokens = torch.randint(0, 90, (4, 7, 5), generator=g, device="cuda")
    same(logits[:, 1:, :, 3:93], tokens[:, 1:], 4)                     # 7 x 5 at one stride, entries at another
    same(logits[:1, :, 2:, :90].expand(4, -1, -1, -1)[:, 0], tokens[:, 0, 2:], 0)  # entries at stride 0


def test_what_does_not_lie_at_two_strides_is_refused():
    from stft_mel_spectrogram_amd import token_logprobs
    logits = torch.zeros(4, 7, 5, 100, device="cuda")
    tokens = torch.zeros(4, 7, 5, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="two strides"):
        token_logprobs(logits[:, 1:, 1:], tokens[:, 1:, 1:])
    with pytest.raises(ValueError, match="contiguous"):
        token_logprobs(logits[:, 1:, :, ::2], tokens[:, 1:])


def test_a_slice_in_a_graph():
    from stft_mel_spectrogram_amd import token_logprobs
    logits = torch.randn(3, 8, 500, device="cuda", dtype=torch.bfloat16)
    tokens = torch.randint(0, 500, (3, 8), device="cuda")
    call = lambda: token_logprobs(logits[:, :-1], tokens[:, 1:], 3)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(3):
        logits.normal_()
        tokens.random_(0, 500)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call()):
            assert torch.equal(a, b)
