"""Adjusted logits against the definition in 64 bits.

Tolerances: at most six roundings of the terms' sizes in float32 and one more per
bias of the same token (2^-24 each, of their sum), then half a step of the type.
Logits that nothing touches come back bit for bit.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(rows, vocab, history, biases, masked, dtype, seed, ints=torch.int64):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = dict(x=(torch.randn(rows, vocab, generator=g, device="cuda") * 2.5).to(dtype),
             history=(rand(rows, history).pow(3) * (vocab + 2)).to(ints) - 1,
             history_lengths=torch.randint(0, history + 1, (rows,), generator=g, device="cuda", dtype=torch.int32),
             prompt_lengths=torch.randint(0, history + 1, (rows,), generator=g, device="cuda",
                                          dtype=torch.int32) // 2,
             repetition=rand(rows) + 0.7, frequency=rand(rows) - 0.3, presence=rand(rows) - 0.3,
             bias_ids=None, bias=None, allowed=None)
    if biases:
        s["bias_ids"] = torch.randint(-2, vocab + 2, (rows, biases), generator=g, device="cuda")
        s["bias"] = torch.randn(rows, biases, generator=g, device="cuda") * 4
    if masked:
        s["allowed"] = torch.randint(-(1 << 31), 1 << 31, (rows, (vocab + 31) // 32), generator=g,
                                     device="cuda").int()
    return s


def reference(s):
    """(result, tolerance, touched) on the CPU, row by row."""
    c = {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    rows, vocab = c["x"].shape
    out, size, touched = c["x"].double().clone(), c["x"].double().abs(), torch.zeros(rows, vocab, dtype=torch.bool)
    at = lambda k, r: c[k][r].item() if isinstance(c[k], torch.Tensor) else c[k]  # noqa: E731
    for r in range(rows):
        h = c["history"][r] if c["history"] is not None else torch.empty(0, dtype=torch.int64)
        n = len(h) if c["history_lengths"] is None else max(0, min(len(h), at("history_lengths", r)))
        p = 0 if c["prompt_lengths"] is None else at("prompt_lengths", r)
        rep, freq, pres = (torch.tensor(at(k, r), dtype=torch.float32).double().item()
                           for k in ("repetition", "frequency", "presence"))
        for i, tok in enumerate(h[:n].tolist()):
            if not 0 <= tok < vocab:
                continue
            if not touched[r, tok]:
                touched[r, tok] = True
                v = out[r, tok].item()
                out[r, tok] = v / rep if v > 0 else v * rep
                size[r, tok] = max(abs(v), out[r, tok].abs().item())
        gen = h[max(0, p):n].long()
        gen = gen[(gen >= 0) & (gen < vocab)]
        count = torch.bincount(gen, minlength=vocab).double()
        out[r] -= freq * count + pres * (count > 0)
        size[r] += abs(freq) * count + abs(pres) * (count > 0)
        if c["bias_ids"] is not None:
            for tok, b in zip(c["bias_ids"][r].tolist(), c["bias"][r].tolist()):
                if 0 <= tok < vocab:
                    out[r, tok] += b
                    size[r, tok] += 2 * abs(b)
                    touched[r, tok] = True
        if c["allowed"] is not None:
            words = (c["allowed"] if c["allowed"].dim() == 1 else c["allowed"][r]).long() & 0xFFFFFFFF
            i = torch.arange(vocab)
            off = (words[i // 32] >> (i % 32)) & 1 == 0
            out[r, off] = -math.inf
            touched[r, off] = True
    many = 6 + (c["bias_ids"].shape[1] if c["bias_ids"] is not None else 0)
    return out, 2.0 ** -24 * many * size, touched


def run_case(s, **kw):
    from stft_mel_spectrogram_amd import adjust_logits
    got = adjust_logits(**{("logits" if k == "x" else k): v for k, v in s.items()}, **kw)
    want, tol, touched = reference(s)
    fi = torch.finfo(got.dtype)
    g = got.cpu()
    assert torch.equal(g[~touched].view(-1), s["x"].cpu()[~touched].view(-1))
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(g), fin) and torch.equal(g.double()[~fin], want[~fin])
    tol = tol + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps
    worst = ((g.double() - want).abs() / tol)[fin].max().item() if fin.any() else 0.0
    print(f"worst error / tolerance {worst:.3g}")
    assert worst <= 1.0
    return got


# one group, one workgroup, several segments and their borders
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 3, 29, 32, 33, 1023, 1024, 1025, 2048, 2049, 4097, 9001, 50001])
def test_vocabularies(vocab, dtype):
    run_case(inputs(3, vocab, 60, 10, True, DT[dtype], vocab))


@pytest.mark.parametrize("rows,vocab", [(1, 131072), (70, 17000), (300, 9001), (600, 5000)])
def test_row_counts(rows, vocab):
    """Every segment size."""
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(rows, vocab, 100, 20, True, torch.float16, rows)
    whole = adjust_logits(**{("logits" if k == "x" else k): v for k, v in s.items()})
    few = slice(0, rows, max(1, rows // 4))
    want, tol, touched = reference({k: v[few] if isinstance(v, torch.Tensor) else v for k, v in s.items()})
    g = whole[few].cpu()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(g), fin)
    assert ((g.double() - want).abs() <= tol + 2.0 ** -11 * want.abs() + 2.0 ** -24)[fin].all()


@pytest.mark.parametrize("ints", [torch.int64, torch.int32])
@pytest.mark.parametrize("history", [1, 255, 256, 1025, 5000])
def test_histories(history, ints):
    run_case(inputs(4, 3001, history, 0, False, torch.float32, history, ints))


@pytest.mark.parametrize("biases", [1, 63, 64, 65, 300, 1024])
def test_biases(biases):
    """The same token many times: their sum in order."""
    s = inputs(3, 700, 5, biases, False, torch.float32, biases)
    s["bias_ids"][0] = 13
    s["bias_ids"][1] = torch.arange(biases, device="cuda") % 3
    a = run_case(s)
    assert torch.equal(a, run_case(s))


def test_each_by_itself():
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(4, 2100, 50, 9, True, torch.bfloat16, 1)
    off = dict(history=None, history_lengths=None, prompt_lengths=None, repetition=1.0, frequency=0.0, presence=0.0,
               bias_ids=None, bias=None, allowed=None)
    assert torch.equal(adjust_logits(s["x"]), s["x"])
    for keep in (("history",), ("history", "history_lengths"), ("history", "repetition"), ("history", "prompt_lengths"),
                 ("history", "frequency"), ("history", "presence"), ("bias_ids", "bias"), ("allowed",),
                 ("repetition", "frequency", "presence")):
        run_case(dict(s, **{k: v for k, v in off.items() if k not in keep}))
    run_case(dict(s, repetition=1.3, frequency=0.25, presence=-0.5))
    run_case(dict(s, allowed=s["allowed"][2].contiguous()))


def test_history_ends():
    """No history, lengths out of range, tokens outside the vocabulary."""
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(5, 300, 40, 0, False, torch.float32, 2)
    s["history_lengths"] = torch.tensor([0, -4, 100, 40, 7], dtype=torch.int32, device="cuda")
    s["prompt_lengths"] = torch.tensor([3, 5, -1, 90, 7], dtype=torch.int32, device="cuda")
    s["history"][3, :5] = torch.tensor([-1, 300, 1 << 40, -(1 << 40), 299], device="cuda")
    got = run_case(s)
    assert torch.equal(got[:2], s["x"][:2])
    empty = torch.empty(5, 0, dtype=torch.int64, device="cuda")
    assert torch.equal(adjust_logits(s["x"], empty, repetition=2.0), s["x"])
    assert adjust_logits(s["x"][:0], s["history"][:0]).shape == (0, 300)


def test_values():
    """-inf, NaN and infinities: a mask hides all of them."""
    from stft_mel_spectrogram_amd import adjust_logits
    x = torch.zeros(1, 40, device="cuda")
    x[0, :4] = torch.tensor([-math.inf, math.inf, math.nan, torch.finfo(torch.float32).min], device="cuda")
    h = torch.arange(6, device="cuda")[None]
    y = adjust_logits(x, h, repetition=2.0, frequency=1.0)
    assert y[0, 0] == -math.inf and y[0, 1] == math.inf and y[0, 2].isnan() and y[0, 3] == -math.inf
    assert (y[0, 4:6] == -1).all() and (y[0, 6:] == 0).all()
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert (adjust_logits(x, h, repetition=2.0, allowed=none) == -math.inf).all()
    # 16 bits: a result past the type's range
    z = adjust_logits(torch.full((1, 8), -6e4, device="cuda", dtype=torch.float16), h, repetition=2.0)
    assert (z[0, :6] == -math.inf).all() and (z[0, 6:] == -6e4).all()


def test_in_place_strides_and_guards():
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(6, 5001, 80, 30, True, torch.bfloat16, 3)
    kw = {k: v for k, v in s.items() if k != "x"}
    want = adjust_logits(s["x"], **kw)
    x = s["x"].clone()
    assert adjust_logits(x, **kw, out=x) is x and torch.equal(x, want)
    wide = torch.zeros(6, 3, 5001, device="cuda", dtype=torch.bfloat16)
    wide[:, 2] = s["x"]
    hist = torch.zeros(6, 99, dtype=torch.int64, device="cuda")
    hist[:, 9:89] = s["history"]
    words = torch.zeros(6, s["allowed"].shape[1] + 5, dtype=torch.int32, device="cuda")
    words[:, 2:-3] = s["allowed"]
    room = torch.full((6 * 5001 + 64,), 3.0, device="cuda", dtype=torch.bfloat16)
    out = room[32:-32].view(6, 5001)
    adjust_logits(wide[:, 2], **dict(kw, history=hist[:, 9:89], allowed=words[:, 2:-3]), out=out)
    assert torch.equal(out, want) and (room[:32] == 3).all() and (room[-32:] == 3).all()
    lead = adjust_logits(s["x"].view(2, 3, -1), **{k: v.view(2, 3, *v.shape[1:]) for k, v in kw.items()})
    assert torch.equal(lead.view(6, -1), want)


def test_scored_afterwards():
    """A grammar's mask in front of the top alternatives: none of the forbidden
    ones, and their log probabilities add up."""
    from stft_mel_spectrogram_amd import adjust_logits, token_logprobs
    x = torch.randn(4, 96, device="cuda")
    words = torch.tensor([0b1011, 0, 1 << 5], dtype=torch.int32, device="cuda")
    r = token_logprobs(adjust_logits(x, allowed=words), torch.zeros(4, dtype=torch.int64, device="cuda"), 4)
    assert sorted(r.top_ids[0].tolist()) == [0, 1, 3, 69]
    assert (r.top_logprobs.exp().sum(-1) - 1).abs().max() <= 2.0 ** -18


def test_captured():
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(3, 3001, 70, 8, True, torch.float16, 4)
    kw = {k: v for k, v in s.items() if k != "x"}
    adjust_logits(s["x"], **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = adjust_logits(s["x"], **kw)
    for i in range(4):
        n = inputs(3, 3001, 70, 8, True, torch.float16, 30 + i)
        for k, v in n.items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = adjust_logits(s["x"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_full_of_tokens(dtype):
    """More touched tokens in a segment than are worked on as a list; results of
    exactly 0 among them."""
    s = inputs(2, 5000, 9000, 300, True, DT[dtype], 17)
    s["history"] = torch.arange(9000, device="cuda").expand(2, 9000) % 4500
    s["history_lengths"] = torch.tensor([9000, 3000], dtype=torch.int32, device="cuda")
    run_case(s)
    z = dict(s, x=torch.zeros_like(s["x"]), frequency=0.0, presence=0.0, bias_ids=None, bias=None, allowed=None)
    assert (run_case(z) == 0).all()
    assert (run_case(dict(z, history=s["history"][:, :40])) == 0).all()
