"""The operators chained under autograd, forward and backward captured into one
graph: every replay equals the eager result on the same inputs, with eager work
and synchronization between the replays."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def chain(x, w, b, table, m, tokens, heads):
    """norm -> attention (queries, keys and values: the normed rows) -> scores."""
    from stft_mel_spectrogram_amd import layer_norm, relative_attention, token_logprobs
    bs, t, c = x.shape
    h = layer_norm(x, w, b)
    split = h.view(bs, t, heads, c // heads).transpose(1, 2)
    o = relative_attention(split, split, split, table, m, causal=True)
    return token_logprobs(o.transpose(1, 2).reshape(bs, t, c), tokens, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t", [5, 130])
def test_chain_under_capture(t, dtype):
    from stft_mel_spectrogram_amd import relative_buckets
    g = torch.Generator(device="cuda")
    g.manual_seed(t)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, b, table = r(2, t, 96), r(96), r(96), r(16, 3)
    m = relative_buckets(16, 30, device="cuda")
    tokens = torch.randint(0, 96, (2, t), generator=g, device="cuda")
    ups = [torch.randn(2, t, generator=g, device="cuda") for _ in range(2)]
    ups.append(torch.randn(2, t, 3, generator=g, device="cuda"))

    def step(leaves):
        out = chain(*leaves, m, tokens, 3)
        grads = torch.autograd.grad((out.logprobs, out.entropy, out.top_logprobs), leaves, ups)
        return [o.detach() for o in out], [d.detach() for d in grads]

    fresh = lambda v: [s.clone().requires_grad_(True) for s in (v, w, b, table)]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fresh(x))  # libraries and attributes set up before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    static = fresh(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got_out, got_grads = step(static)
    for _ in range(4):
        nx = r(2, t, 96)
        with torch.no_grad():
            static[0].copy_(nx)
        graph.replay()
        torch.cuda.synchronize()
        want_out, want_grads = step(fresh(nx))
        torch.cuda.synchronize()
        for a, e in zip(got_out + got_grads, want_out + want_grads):
            assert torch.isfinite(e.float()).all() and torch.equal(a, e)


def test_step_of_the_model_repeats_bit_for_bit():
    """The same training steps twice: no sum depends on the order in which
    workgroups run."""
    from stft_mel_spectrogram_amd import relative_buckets
    m = relative_buckets(16, 30, device="cuda")
    results = []
    for _ in range(2):
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        leaves = [torch.randn(*s, generator=g, device="cuda").requires_grad_(True)
                  for s in ((3, 700, 96), (96,), (96,), (16, 3))]
        tokens = torch.randint(0, 96, (3, 700), generator=g, device="cuda")
        out = chain(*leaves, m, tokens, 3)
        results.append(torch.autograd.grad(out.logprobs, leaves, torch.ones_like(out.logprobs)))
    for a, e in zip(*results):
        assert torch.equal(a, e)
