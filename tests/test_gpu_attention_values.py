"""Attention at values where a type's range or its smallest steps matter, against
the float64 implementation and the tolerances of test_gpu_relative_attention.

float16 probabilities and score gradients are scaled by powers of two for their
products, so that half a step (h) of each is relative for probabilities down to
2^-25 of the row's largest and for score gradients down to 2^-24 of the largest
that the row (dq) or the key (dk) can have.
"""

import pytest

torch = pytest.importorskip("torch")
import test_gpu_relative_attention as plain  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("value,grad", [(1100.0, 1e-3), (6e4, 1e-3), (300.0, 2.0), (1100.0, 2e-5), (0.5, 3.0)])
@pytest.mark.parametrize("h,hk,tq,tk,d", [
    (1, 1, 1, 2, 128),      # one tile: delta from p and dp
    (2, 2, 40, 45, 64),
    (4, 1, 300, 300, 40),   # shares of the queries for dk, dv
    (2, 1, 60, 1030, 128),  # ranges of the keys for dq
    (2, 2, 70, 75, 33),     # odd rows
])
def test_float16_gradients_of_large_values(h, hk, tq, tk, d, value, grad):
    """Values of one sign per key and gradients of one sign: sum |do| |v| is reached, d times
    the largest |do| times the largest |v|, which one scale for the largest |do| alone would
    lift past float16's range.  Every result is finite in float16."""
    q, k, v, table, m, do = plain.make(2, h, hk, tq, tk, d, "f16", seed=d, std=1.7)
    sign = torch.where(v[..., :1] > 0, 1.0, -1.0)
    v = (sign * value * (1 + v.float().abs() / 64)).clamp(-6.5e4, 6.5e4).half()
    do = (grad * (0.5 + do.float().abs() / 4) / max(1.0, value * grad * d / 2000)).half()
    plain.run_case(q, k, v, table, m, do)


def test_float16_overflow_of_two_keys():
    """Two keys of probability 1/2 each, values 1100 and -1100, gradients of 1e-3 in 128 columns:
    ds is +-70."""
    from stft_mel_spectrogram_amd import relative_attention_backward, relative_attention_forward
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    q, k, v = z(1, 1, 1, 128) + 1, z(1, 1, 2, 128) + 1, z(1, 1, 2, 128)
    v[:, :, 0], v[:, :, 1] = 1100, -1100
    do = z(1, 1, 1, 128) + 1e-3
    table, m = z(1, 1), torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = relative_attention_forward(q, k, v, table, m)
    dq, dk, dv, dt = relative_attention_backward(do, q, k, v, table, m, o, lse)
    ds = 0.5 * 1100 * 128 * do[0, 0, 0, 0].item()
    scale = 128 ** -0.5
    h = 2.0 ** -11
    # three roundings: p, ds and the result; float32's roundings beside them
    assert (dk[0, 0, 0].double() - ds * scale).abs().max() <= 3.1 * h * ds * scale
    assert (dk[0, 0, 1].double() + ds * scale).abs().max() <= 3.1 * h * ds * scale
    assert (dq.double().abs() <= 2.1 * h * 2 * ds * scale).all()  # ds of both cancel
    assert (dv.double() - 0.5e-3).abs().max() <= 3.1 * h * 0.5e-3
    assert torch.isfinite(dt).all()


def sink_case(tq, tk, d, nats, at, seed):
    """A key of value 0 whose score is `nats` above all others', which lie close together."""
    q, k, v, table, m, do = plain.make(1, 2, 2, tq, tk, d, "f16", seed=seed, layout="bhtd")
    table = torch.zeros_like(table)
    q = q / 8
    k = k / 4
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, :, at] = 0
    k[:, :, at, 0] = nats * d ** 0.5 / 4
    v[:, :, at] = 0
    return q, k, v, table, m, do


@pytest.mark.parametrize("nats", [12, 14, 16, 17])
@pytest.mark.parametrize("tq,tk,d", [(60, 310, 64), (150, 1500, 128), (1, 1501, 64), (7, 1501, 128),
                                     (1, 5000, 40), (17, 2500, 33)])
def test_float16_probabilities_beside_a_sink(tq, tk, d, nats):
    """The general kernel and the cache kernel, each in one range and in several."""
    for at in (0, tk - 1):
        q, k, v, table, m, do = sink_case(tq, tk, d, nats, at, nats + tk)
        plain.run_case(q, k, v, table, m, do, backward=False)


@pytest.mark.parametrize("nats", [10, 13, 15])
@pytest.mark.parametrize("tq,tk,d", [(60, 310, 64), (150, 700, 128), (200, 90, 40)])
def test_float16_gradients_beside_a_sink(tq, tk, d, nats):
    for at in (0, tk - 1):
        q, k, v, table, m, do = sink_case(tq, tk, d, nats, at, nats + tk)
        plain.run_case(q, k, v, table, m, do)
