"""What the torch-facing callers of the recurrence, the RMS norm, the distillation
and the adjusted logits refuse, before any launch: by type, shape, layout, device,
missing tensors and forward-mode tangents."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


F = torch.float32


def refuse(err, fn, *args, **kw):
    with pytest.raises(err):
        fn(*args, **kw)


def test_gated_recurrence():
    from stft_mel_spectrogram_amd import (gated_recurrence, gated_recurrence_backward, gated_recurrence_forward)
    x, h = t(2, 5, 8), t(2, 8, dtype=F)
    for args, err in (((x[0], x[0]), ValueError), ((x, x.float()), TypeError), ((x.double(), x), TypeError),
                      ((x, x[:, :4]), ValueError), ((x, x, t(2, 5, 9)), ValueError), ((x, x, x, h[:1]), ValueError),
                      ((x, x, x, h.half()), TypeError), ((x, x, x, h.cpu()), ValueError),
                      ((x, t(2, 8, 5).transpose(1, 2)), ValueError), ((x, None), ValueError), ((x, 3.0), ValueError),
                      ((x, x, 3.0), ValueError), ((x, x, x, 3.0), ValueError), ((t(2, 5, 0), t(2, 5, 0)), ValueError),
                      ((x, x, x, t(8, 2, dtype=F).t()), ValueError)):
        refuse(err, gated_recurrence, *args)
    refuse(ValueError, gated_recurrence, x, x, lengths=t(2, dtype=torch.int64))
    refuse(ValueError, gated_recurrence, x, x, lengths=t(3, dtype=torch.int32))
    refuse(ValueError, gated_recurrence, x, x, out=t(2, 5, 9))
    refuse(ValueError, gated_recurrence, x, x, out=x.float())
    refuse(TypeError, gated_recurrence, x, x, out_state=h.double())
    refuse(ValueError, gated_recurrence, x, x, out_state=h.cpu())
    refuse(ValueError, gated_recurrence, x.clone().requires_grad_(True), x, out_state=h)
    y, last, saved = gated_recurrence_forward(x, x, x, h)
    ok = (y, x, x, x, h, saved)
    gated_recurrence_backward(*ok)
    for i in (0, 1, 2, 5):
        refuse(ValueError, gated_recurrence_backward, *(None if j == i else v for j, v in enumerate(ok)))
    refuse(ValueError, gated_recurrence_backward, y.float(), *ok[1:])
    refuse(ValueError, gated_recurrence_backward, *ok[:5], saved[:1])
    refuse(TypeError, gated_recurrence_backward, *ok[:5], saved.double())
    refuse(ValueError, gated_recurrence_backward, *ok, grad_state=h[:, :4])


def test_rms_norm():
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_backward, rms_norm_forward, rms_norm_quantized
    x, w = t(4, 8), t(8)
    for fn in (rms_norm, rms_norm_quantized):
        for args, err in (((x.int(),), TypeError), ((x.t(), t(4)), ValueError), ((t(4, 0),), ValueError),
                          ((x, t(7)), ValueError), ((x, w.half()), TypeError), ((x, w.cpu()), ValueError),
                          ((x, w, x.float()), TypeError), ((x, w, t(4, 9)), ValueError), ((x, w, x.cpu()), ValueError),
                          ((x, w, t(8, 4).t()), ValueError), ((x, 3.0), ValueError), ((x, w, 3.0), ValueError)):
            refuse(err, fn, *args)
        refuse(ValueError, fn, x, w, out_sum=x)
        refuse(ValueError, fn, x, w, x, out_sum=t(4, 9))
        refuse(RuntimeError, fn, x, w, None, -1.0)
    refuse(ValueError, rms_norm, x, w, out=t(4, 9))
    refuse(ValueError, rms_norm, x, w.clone().requires_grad_(True), out=t(4, 8))
    refuse(ValueError, rms_norm_quantized, x, w.clone().requires_grad_(True))
    refuse(TypeError, rms_norm_quantized, x, w, dtype=torch.float16)
    y, s, r = rms_norm_forward(x, w, x)
    for bad in ((t(4, 9), s, w, r), (x.float(), s, w, r), (x, s, w, r[:3]), (x, s, w, r.cpu()), (None, s, w, r),
                (x, s, w, None), (x, s, w, r, t(4, 9)), (x, s, w, r, 3.0)):
        refuse(ValueError, rms_norm_backward, *bad)
    refuse(TypeError, rms_norm_backward, x, s, w, r.double())


def test_topk_distillation():
    from stft_mel_spectrogram_amd import (topk_distillation, topk_distillation_backward, topk_distillation_forward)
    x, ids, lps = t(4, 50), t(4, 5, dtype=torch.int64), t(4, 5, dtype=F)
    for args, err in (((x.double(), ids, lps), TypeError), ((x, ids.int(), lps), TypeError),
                      ((x, ids, lps.half()), TypeError), ((x, ids[:3], lps), ValueError),
                      ((x, ids, lps[:, :4]), ValueError), ((x, ids[:, :0], lps[:, :0]), ValueError),
                      ((x, t(4, 65, dtype=torch.int64), t(4, 65, dtype=F)), ValueError), ((x, ids.cpu(), lps), ValueError),
                      ((x[:, ::2], ids, lps), ValueError), ((x, None, lps), ValueError), ((x, ids, 3.0), ValueError),
                      ((x, ids, lps.clone().requires_grad_(True)), ValueError), ((x, ids[:, 0], lps), ValueError)):
        refuse(err, topk_distillation, *args)
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=2.0, rest=True)):
        refuse(RuntimeError, topk_distillation, x, ids, lps, **kw)
    loss, stats = topk_distillation_forward(x, ids, lps)
    for bad, err in (((loss[:3], x, ids, lps, stats), ValueError), ((loss.half(), x, ids, lps, stats), TypeError),
                     ((loss, x, ids, lps, stats[:, :1]), ValueError), ((None, x, ids, lps, stats), ValueError),
                     ((loss, x, ids, lps, None), ValueError)):
        refuse(err, topk_distillation_backward, *bad)


def test_adjust_logits():
    from stft_mel_spectrogram_amd import adjust_logits
    x, h, n = t(4, 50), t(4, 7, dtype=torch.int64), t(4, dtype=torch.int32)
    ids, b = t(4, 3, dtype=torch.int64), t(4, 3, dtype=F)
    for args, kw, err in (((x.double(),), {}, TypeError), ((x[:, ::2],), {}, ValueError), ((x, h.short()), {}, TypeError),
                          ((x, h[:3]), {}, ValueError), ((x, h[0]), {}, ValueError), ((x, h, n.long()), {}, ValueError),
                          ((x, h, n[:3]), {}, ValueError), ((x, None, n), {}, ValueError), ((x, h.cpu()), {}, ValueError),
                          ((x, h), dict(prompt_lengths=n.long()), ValueError), ((x, h), dict(repetition=0.0), RuntimeError),
                          ((x, h), dict(repetition=b[:, 0].double()), TypeError),
                          ((x, h), dict(frequency=b[:3, 0].contiguous()), ValueError),
                          ((x, h), dict(presence=float("nan")), RuntimeError), ((x,), dict(bias=b), ValueError),
                          ((x,), dict(bias_ids=ids), ValueError), ((x,), dict(bias_ids=ids.int(), bias=b), TypeError),
                          ((x,), dict(bias_ids=ids, bias=b.half()), TypeError),
                          ((x,), dict(bias_ids=ids[:, :2], bias=b), ValueError),
                          ((x,), dict(allowed=t(4, 2)), TypeError), ((x,), dict(allowed=t(3, dtype=torch.int32)), ValueError),
                          ((x,), dict(allowed=t(3, 2, dtype=torch.int32)), ValueError),
                          ((x,), dict(out=t(4, 51)), ValueError), ((x,), dict(out=x.float()), ValueError),
                          ((x.clone().requires_grad_(True),), {}, ValueError),
                          ((x,), dict(bias_ids=t(4, 1025, dtype=torch.int64), bias=t(4, 1025, dtype=F)), RuntimeError)):
        refuse(err, adjust_logits, *args, **kw)
    with torch.no_grad():
        adjust_logits(x.clone().requires_grad_(True), h, n)


def test_every_tensors_tangent_is_refused():
    from torch.autograd import forward_ad
    from stft_mel_spectrogram_amd import (adjust_logits, gated_recurrence, gated_recurrence_backward, rms_norm,
                                          rms_norm_backward, topk_distillation, topk_distillation_backward)
    x, h, one, s = t(2, 5, 8, dtype=F), t(2, 8, dtype=F), t(2, 5, dtype=F), t(2, 1, 8, dtype=F)
    ids, h8 = t(2, 5, 3, dtype=torch.int64), t(8, dtype=F)
    lps = t(2, 5, 3, dtype=F)
    calls = [([x, x, x, h], gated_recurrence), ([x, x, x, x, h, s], gated_recurrence_backward),
             ([x, h8, x], rms_norm), ([x, x, h8, one, x], rms_norm_backward),
             ([x, lps], lambda a, b: topk_distillation(a, ids, b)),
             ([one, x, lps, t(2, 5, 4, dtype=F)], lambda g, a, b, st: topk_distillation_backward(g, a, ids, b, st)),
             ([x, one], lambda a, r: adjust_logits(a, ids, repetition=r))]
    for xs, call in calls:
        call(*xs)
        with forward_ad.dual_level():
            call(*xs)  # inside a level, without tangents
            for i in range(len(xs)):
                ys = [forward_ad.make_dual(v.clone(), torch.ones_like(v)) if j == i else v for j, v in enumerate(xs)]
                with pytest.raises(NotImplementedError):
                    call(*ys)
