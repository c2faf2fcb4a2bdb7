"""Distillation from a teacher's top log probabilities and the logits' gradient
against the 64-bit formulas.

Tolerances.  As for the token log probabilities: with D the largest distance of a
counted entry from the row's maximum (in units of T), e = 2^-23 (D + 64 + entries of a
lane) bounds the relative error of a row's sum, and so the error of a log probability
beside the roundings of its own terms, 2^-22 (|lp| + |z| + 1).  A teacher's q is off by
2^-22 (|log q| + 4) of itself.
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


def inputs(rows, vocab, top, dtype, seed, std=2.5, noise=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * std).to(dtype)
    y = torch.log_softmax(x.float() + noise * torch.randn(rows, vocab, generator=g, device="cuda"), -1)
    best = y.topk(top, -1)
    return x, best.indices, best.values, torch.randn(rows, generator=g, device="cuda")


def reference(x, ids, lps, tau, rest, grad):
    """Loss, gradient and their tolerances; ids may be negative, rows must have
    a finite entry."""
    z = x.double() / tau
    v = x.shape[-1]
    lp = torch.log_softmax(z, -1)
    p = lp.exp()
    t = lps.double()
    there = ids >= 0
    at = ids.clamp(min=0)
    if rest:
        lq = torch.where(there, t, torch.full_like(t, -math.inf))
    else:
        tt = torch.where(there, t / tau, torch.full_like(t, -math.inf))
        lq = tt - torch.logsumexp(tt, -1, keepdim=True)
        lq = torch.where(there, lq, torch.full_like(t, -math.inf)).nan_to_num(nan=-math.inf)
    q = lq.exp()
    none = (~there).all(-1) | (q.sum(-1) == 0) & (not rest)
    lpk = lp.gather(-1, at)
    zero = torch.zeros_like(q)
    term = torch.where(q > 0, q * (lq - lpk), zero)
    loss = term.sum(-1)
    size = torch.where(q > 0, q * (lq.abs() + lpk.abs() + z.gather(-1, at).abs() + 4), zero).sum(-1)
    target = torch.zeros_like(z).scatter_add_(-1, at, torch.where(there, q, zero))
    named = torch.zeros_like(z).scatter_add_(-1, at, there.double()) > 0
    tsize = torch.zeros_like(z).scatter_add_(-1, at, torch.where(q > 0, q * (lq.abs() + 4), zero))
    if rest:
        r = (1 - q.sum(-1)).clamp(min=0)
        others = z.masked_fill(named, -math.inf)
        lse_rest = torch.logsumexp(others, -1)
        lpr = torch.logsumexp(lp.masked_fill(named, -math.inf), -1)
        has = lse_rest > -math.inf
        r = torch.where(has, r, torch.zeros_like(r))
        loss = loss + torch.where(r > 0, r * (r.log() - lpr), torch.zeros_like(r))
        # r carries a rounding of its own, and its logarithm
        size = size + torch.where(r > 0, r * (r.log().abs() + lpr.abs() + lse_rest.abs() + 4), torch.zeros_like(r))
        share = torch.where(has[:, None], (others - lse_rest[:, None]).exp(), torch.zeros_like(z)).nan_to_num()
        target = target + r[:, None] * share
        tsize = tsize + (r[:, None] * 4 + p.masked_fill(named, 0).sum(-1, keepdim=True)) * share
    total = target.sum(-1, keepdim=True)
    dx = tau * grad.double()[:, None] * (p * total - target)
    loss, dx = loss * tau ** 2, dx
    m = z.amax(-1, keepdim=True)
    dist = torch.where(lp > -200, m - z, torch.zeros_like(z)).amax(-1)
    e = 2.0 ** -23 * (dist + 64 + v / 256)
    lse = torch.logsumexp(z, -1)
    tol_loss = tau ** 2 * (e * (q.sum(-1) + (r if rest else 0)) + 2.0 ** -21 * size)
    lpa = torch.where(p > 0, lp.abs(), torch.zeros_like(lp))
    rel = 4 * e[:, None] + 2.0 ** -21 * (lpa + lse.abs()[:, None] + z.abs().clamp(max=200) + 4)
    tol_dx = tau * grad.double().abs()[:, None] * (rel * (p * total + target) + 2.0 ** -21 * tsize + 2.0 ** -125)
    loss = torch.where(none, torch.zeros_like(loss), loss)
    dx = torch.where(none[:, None], torch.zeros_like(dx), dx)
    return loss, tol_loss, dx, tol_dx


def close(name, got, want, tol):
    fi = torch.finfo(got.dtype)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), name
    assert torch.equal(got.double()[~fin], want[~fin]), name
    tol = tol + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps
    worst = ((got.double() - want).abs() / tol)[fin].max().item() if fin.any() else 0.0
    print(f"[{name}] worst error / tolerance {worst:.3g}")
    assert worst <= 1.0, (name, worst)


def run_case(x, ids, lps, g, tau=1.0, rest=False):
    from stft_mel_spectrogram_amd import (topk_distillation, topk_distillation_backward, topk_distillation_forward)
    how = dict(temperature=tau, rest=rest)
    loss, stats = topk_distillation_forward(x, ids, lps, **how)
    dx = topk_distillation_backward(g, x, ids, lps, stats, **how)
    want, tl, wdx, tdx = reference(x, ids, lps, tau, rest, g)
    close("loss", loss, want, tl)
    close("dx", dx, wdx, tdx)
    assert torch.equal(topk_distillation(x, ids, lps, **how), loss)
    return loss, dx


# one entry; the register layouts and their borders; several chunks and segments
VOCABS = [1, 2, 29, 129, 130, 511, 1023, 1024, 1025, 2048, 2049, 8193, 20011, 50001]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_vocabularies(vocab, dtype, rest):
    for top in (1, min(20, vocab)):
        if rest and top == vocab:
            continue  # nothing is left: see below
        run_case(*inputs(5, vocab, top, DT[dtype], vocab), rest=rest)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("top", [2, 15, 16, 17, 48, 63, 64])
@pytest.mark.parametrize("vocab", [70, 400, 1500, 40003])
def test_entry_counts(vocab, top, rest):
    run_case(*inputs(6, vocab, top, torch.bfloat16, top), rest=rest)


@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0, 7.5])
@pytest.mark.parametrize("vocab", [129, 9001])
def test_temperatures(vocab, tau):
    run_case(*inputs(7, vocab, 8, torch.float32, 3), tau=tau)


@pytest.mark.parametrize("rows", [0, 1, 33, 1500])
def test_row_counts(rows):
    from stft_mel_spectrogram_amd import topk_distillation
    for vocab in (100, 9001):
        x, ids, lps, g = inputs(rows, vocab, 5, torch.bfloat16, rows)
        if rows == 0:
            assert topk_distillation(x, ids, lps).shape == (0,)
        else:
            run_case(x, ids, lps, g, rest=True)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("vocab", [40, 200, 700, 30011])
def test_few_and_repeated_entries(vocab, rest):
    """Rows with fewer entries, none, the same token twice and more."""
    x, ids, lps, g = inputs(6, vocab, 12, torch.float32, 5)
    ids[0, 4:] = -1
    ids[1] = -7
    ids[2, ::2] = -1
    ids[3, 5] = ids[3, 1]
    lps[3, 5] -= 1
    ids[4, :] = ids[4, 0]
    lps[4] = math.log(0.05)
    loss, dx = run_case(x, ids, lps, g, rest=rest)
    assert loss[1] == 0 and (dx[1] == 0).all()


@pytest.mark.parametrize("vocab", [50, 3000])
def test_teacher_without_mass(vocab):
    x, ids, lps, g = inputs(4, vocab, 6, torch.float32, 6)
    lps[0, 3:] = -math.inf
    lps[1] = -math.inf
    run_case(x, ids, lps, g)
    run_case(x, ids, lps, g, rest=True)


@pytest.mark.parametrize("vocab", [64, 5003])
def test_masked_logits(vocab):
    """-inf and the type's lowest value in the student's rows."""
    from stft_mel_spectrogram_amd import topk_distillation_backward, topk_distillation_forward
    for low in (-math.inf, torch.finfo(torch.bfloat16).min):
        x, ids, lps, g = inputs(5, vocab, 6, torch.bfloat16, 7)
        keep = torch.zeros_like(x, dtype=torch.bool).scatter_(1, ids, True)
        keep[:, : vocab // 2] = True
        x[~keep] = low
        for rest in (False, True):
            run_case(x, ids, lps, g, rest=rest)
        # nothing beside the named tokens
        y = x.clone()
        y[~torch.zeros_like(keep).scatter_(1, ids, True)] = -math.inf
        run_case(y, ids, lps, g, rest=True)
        run_case(y, ids, lps, g)
    # a named token without probability
    x, ids, lps, g = inputs(3, vocab, 6, torch.float32, 8)
    x[0, ids[0, 2]] = -math.inf
    for rest in (False, True):
        loss, stats = topk_distillation_forward(x, ids, lps, rest=rest)
        assert loss[0] == math.inf and torch.isfinite(loss[1:]).all()
        assert torch.isfinite(topk_distillation_backward(g, x, ids, lps, stats, rest=rest)).all()
    # rows of -inf only, of the lowest value only
    x[1] = -math.inf
    x[2] = torch.finfo(torch.float32).min
    for rest in (False, True):
        loss, stats = topk_distillation_forward(x, ids, lps, rest=rest)
        dx = topk_distillation_backward(g, x, ids, lps, stats, rest=rest)
        assert loss[1] == math.inf and (dx[1] == 0).all()
        want, tl, wdx, tdx = reference(torch.zeros_like(x[2:]), ids[2:], lps[2:], 1.0, rest, g[2:])
        close("equal logits", loss[2:], want, tl)
        close("equal logits", dx[2:], wdx, tdx)


@pytest.mark.parametrize("vocab", [16, 64])
def test_every_token_named(vocab):
    """The rest is empty and the roundings of its mass do no harm."""
    x, ids, lps, g = inputs(9, vocab, vocab, torch.float32, 9)
    a, da = run_case(x, ids, lps, g, rest=True)
    b, db = run_case(x, ids, lps, g)
    assert (a - b).abs().max() <= 2.0 ** -16 and (da - db).abs().max() <= 2.0 ** -16


def test_not_finite_and_lost():
    from stft_mel_spectrogram_amd import topk_distillation_backward, topk_distillation_forward
    for vocab in (90, 7001):
        x, ids, lps, g = inputs(6, vocab, 4, torch.float32, 10)
        want = topk_distillation_forward(x, ids, lps)[0]
        x[0, 5] = math.nan
        x[1, 7] = math.inf
        lps[2, 1] = math.nan
        ids[3, 2] = vocab
        ids[4, 2] = 1 << 40
        for rest in (False, True):
            loss, stats = topk_distillation_forward(x, ids, lps, rest=rest)
            dx = topk_distillation_backward(g, x, ids, lps, stats, rest=rest)
            assert loss[:5].isnan().all() and torch.isfinite(loss[5])
            assert dx[0].isnan().any() and torch.isfinite(dx[3:]).all()
            if not rest:
                assert loss[5] == want[5]


def test_slices():
    """logits[:, :-1] and one strided group are read as they lie."""
    from stft_mel_spectrogram_amd import topk_distillation, topk_distillation_backward, topk_distillation_forward
    for vocab in (60, 3001):
        x, ids, lps, g = inputs(12, vocab, 7, torch.float16, 11)
        x, ids, lps, g = x.view(3, 4, -1), ids.view(3, 4, -1), lps.view(3, 4, -1), g.view(3, 4)
        part = (x[:, :-1], ids[:, 1:], lps[:, 1:], g[:, 1:].contiguous())
        dense = [v.contiguous() for v in part]
        a, sa = topk_distillation_forward(*part[:3], rest=True)
        b, sb = topk_distillation_forward(*dense[:3], rest=True)
        assert torch.equal(a, b) and torch.equal(sa, sb)
        assert torch.equal(topk_distillation_backward(part[3], *part[:3], sa, rest=True),
                           topk_distillation_backward(dense[3], *dense[:3], sb, rest=True))
        assert torch.equal(topk_distillation(x[:, 1], ids[:, 1], lps[:, 1]),
                           topk_distillation(x, ids, lps)[:, 1])


@pytest.mark.parametrize("rest,tau", [(False, 2.0), (True, 1.0)])
def test_autograd_and_differences(rest, tau):
    from stft_mel_spectrogram_amd import topk_distillation
    x, ids, lps, g = inputs(5, 300, 9, torch.float32, 12)
    leaf = x.clone().requires_grad_(True)
    (topk_distillation(leaf, ids, lps, temperature=tau, rest=rest) * g).sum().backward()
    way = torch.randn_like(x).double()

    def value(v):
        return (reference(v, ids, lps, tau, rest, g)[0] * g.double()).sum().item()

    diff = (value(x.double() + 1e-5 * way) - value(x.double() - 1e-5 * way)) / 2e-5
    tol = reference(x, ids, lps, tau, rest, g)[3]
    got = (leaf.grad.double() * way).sum().item()
    assert abs(got - diff) <= (tol * way.abs()).sum().item() + 1e-6 * (1 + abs(diff))


def test_a_teacher_scored_by_the_package():
    """top alternatives of a teacher's logits go in as they come out, and a
    student equal to the teacher has no loss."""
    from stft_mel_spectrogram_amd import token_logprobs, topk_distillation
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    for vocab in (200, 20011):
        t = torch.randn(8, vocab, generator=g, device="cuda") * 3
        r = token_logprobs(t, torch.full((8,), -1, device="cuda"), 10)
        for rest in (False, True):
            loss = topk_distillation(t, r.top_ids, r.top_logprobs, rest=rest)
            if rest:
                # both sides' errors: e of the module's head, twice
                assert loss.abs().max() <= 2 * 2.0 ** -23 * (40 + 64 + vocab / 256)
            else:
                named = topk_distillation(torch.full_like(t, -math.inf).scatter(1, r.top_ids, t.gather(1, r.top_ids)),
                                          r.top_ids, r.top_logprobs)
                assert named.abs().max() <= 2.0 ** -16
                assert (loss >= -2.0 ** -16).all()


def test_captured_and_repeated():
    from stft_mel_spectrogram_amd import topk_distillation_backward, topk_distillation_forward
    for rows, vocab in ((40, 129), (4, 30011)):
        x, ids, lps, g = inputs(rows, vocab, 8, torch.bfloat16, 14)

        def step():
            loss, stats = topk_distillation_forward(x, ids, lps, rest=True)
            return loss, topk_distillation_backward(g, x, ids, lps, stats, rest=True)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for i in range(4):
            nx, nids, nlps, ng = inputs(rows, vocab, 8, torch.bfloat16, 20 + i)
            for a, b in ((x, nx), (ids, nids), (lps, nlps), (g, ng)):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
