"""Distillation at the ends of its temperatures, of logits far from 0: only distances
within a row count, whatever T and whatever all logits share.

Tolerances, with D the largest distance from the row's maximum in units of T: a term's
exponent is a difference of exact logits, rounded once, times log2 e / T in two parts:
its error is 2^-23 (D + 2) of the term; the running sums add 64 + vocab / 256 roundings.
A log probability's own terms (1 / T is rounded too) are off by 2^-22 (|lp| + D + 2), a
teacher's q by 2^-22 (|log q| + 12) of itself.  None of it grows with |x| / T.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# rows in registers, a workgroup per row, segments that a second launch joins
@pytest.mark.parametrize("offset", [0.0, 100.0, -3000.0])
@pytest.mark.parametrize("tau", [2.0 ** -10, 1 / 700, 0.037, 1.0, 7.5, 900.0, 1024.0])
@pytest.mark.parametrize("rows,vocab", [(9, 129), (1500, 9001), (3, 50001)])
def test_logits_far_from_zero(rows, vocab, tau, offset):
    from stft_mel_spectrogram_amd import topk_distillation_backward, topk_distillation_forward
    tau = float(torch.tensor(tau, dtype=torch.float32))  # as the kernels take it
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * (2.5 * tau) + offset
    z = x.double() / tau
    lp = torch.log_softmax(z, -1)
    t = torch.log_softmax(z + torch.randn(z.shape, generator=g, device="cuda"), -1)
    best = t.topk(8, -1)
    ids, lps = best.indices, (best.values * tau).float()
    grad = torch.randn(rows, generator=g, device="cuda")
    loss, stats = topk_distillation_forward(x, ids, lps, temperature=tau)
    dx = topk_distillation_backward(grad, x, ids, lps, stats, temperature=tau)
    lq = torch.log_softmax(lps.double() / tau, -1)
    q, lpk = lq.exp(), lp.gather(-1, ids)
    want = tau ** 2 * (q * (lq - lpk)).sum(-1)
    D = (z.amax(-1) - z.amin(-1))[:, None]
    e = 2.0 ** -23 * (D + 64 + vocab / 256)
    room = e[:, 0] + (q * 2.0 ** -22 * (lpk.abs() + lq.abs() + D + 14)).sum(-1)
    err = (loss.double() - want).abs() / (tau ** 2 * room)
    print(f"loss: worst error / tolerance {err.max().item():.3g}")
    assert err.max() <= 1
    p = lp.exp()
    target = torch.zeros_like(p).scatter_add_(-1, ids, q)
    named = torch.zeros_like(p).scatter_(-1, ids, q * 2.0 ** -21 * (lq.abs() + 12))
    gt = (tau * grad.double())[:, None]
    tol = gt.abs() * (p * (4 * e + 2.0 ** -21 * (lp.abs() + D + 4)) + named + 2.0 ** -23 * target + 2.0 ** -125)
    err = (dx.double() - gt * (p - target)).abs() / tol
    print(f"dx: worst error / tolerance {err.max().item():.3g}")
    assert err.max() <= 1
