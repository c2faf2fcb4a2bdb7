"""Attention at values where a type's range or its smallest steps matter, against
the float64 implementation and the tolerances of test_gpu_relative_attention.

float16 probabilities and score gradients are scaled by powers of two for their
products, so that half a step (h) of each is relative for probabilities down to
2^-25 of the row's largest and for score gradients down to 2^-24 of the largest
that the row (dq) or the key (dk) can have.
"""
import math

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


@pytest.mark.parametrize("h,hk,d", [(2, 2, 64), (4, 1, 40), (1, 1, 128)])
@pytest.mark.parametrize("one,others", [(2e3, 2e-3), (2e-2, 2e3)])
def test_float16_gradients_of_very_different_rows(h, hk, d, one, others):
    """A query whose gradient is 10^6 times the others' (or a 10^5th) and that sees one key only:
    the other keys' gradients come from the other queries alone."""
    q, k, v, table, m, do = plain.make(1, h, hk, 900, 900, d, "f16", seed=d, layout="bhtd")
    table = torch.zeros_like(table)
    at, key = 645, 30
    q[..., 0], q[:, :, at] = 0, 0
    k[..., 0] = 0
    q[:, :, at, 0], k[:, :, key, 0] = 20.0, 2.5 * d ** 0.5  # 50 nats
    sizes = torch.full((900, 1), others, device="cuda")
    sizes[at] = one
    plain.run_case(q, k, v, table, m, (do.float() * sizes).half())


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


LIMIT = 65536.0


@pytest.mark.parametrize("low", ["min", "max", -1e9, -65504.0, -1e4])
@pytest.mark.parametrize("dtype,table_dtype", [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                               ("bf16", "f32")])
@pytest.mark.parametrize("tq,tk,d", [(70, 75, 64), (150, 1100, 40), (1, 400, 64), (7, 5000, 128), (1, 1, 8)])
def test_rows_whose_keys_all_have_a_bias_of_the_lowest_value(tq, tk, d, dtype, table_dtype, low):
    """Finite table values count as at most 2^16 either way, so a row of such keys alone is an
    ordinary row.  Its scores are held in float32 at 2^16: in units of the product, 2^16 / scale,
    every one of the D / 16 accumulations (six times as many in float32, up to four roundings each)
    and the scaling round by half a step, 2^-8 in the scores, the log sum exp likewise."""
    from stft_mel_spectrogram_amd import relative_attention_backward, relative_attention_forward
    q, k, v, table, m, do = plain.make(1, 2, 2, tq, tk, d, dtype, seed=tk, far=20, buckets=12)
    dt = plain.DT[table_dtype]
    big = {"min": torch.finfo(dt).min, "max": torch.finfo(dt).max}.get(low, low)
    if abs(big) > torch.finfo(dt).max:
        pytest.skip("not a value of the type")
    table = torch.full((12, 2), big, device="cuda").to(dt)
    want = table.double().clamp(-LIMIT, LIMIT)
    off = torch.zeros(1, device="cuda")
    v = torch.ones_like(v)  # o is 1 whatever the probabilities are
    o, stats = relative_attention_forward(q, k, v, table, m)
    half = torch.finfo(q.dtype).eps / 2
    # half a step of p and of o; float32 sums
    assert ((o.double() - 1).abs() <= 2 * half + 2.0 ** -18).all()
    lse = plain.reference(q, k, v, want, m, do, d ** -0.5, False, torch.full((1,), tk, device="cuda"), off)[2]
    steps = (d + 15) // 16 * (24 if dtype == "f32" else 4) + 8
    assert ((stats.double() - lse).abs() <= steps * 2.0 ** -8).all()
    got = relative_attention_backward(do, q, k, v, table, m, o, stats)
    assert all(torch.isfinite(g).all() for g in got)
    # dv: probabilities within exp of the scores' and the log sum exp's error
    dv = plain.reference(q, k, v, want, m, do, d ** -0.5, False, torch.full((1,), tk, device="cuda"), off)[4]["dv"]
    p_tol = math.expm1(2 * steps * 2.0 ** -8) + 4 * half
    size = plain.reference(q, k, v, want, m, do.abs(), d ** -0.5, False, torch.full((1,), tk, device="cuda"),
                           off)[4]["dv"]
    tiny = torch.finfo(q.dtype).smallest_normal
    assert ((got[2].double() - dv).abs() <= p_tol * size + tiny).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tq", [1, 60])
def test_a_bias_of_the_lowest_value_still_hides_a_key_from_others(tq, dtype):
    q, k, v, table, m, do = plain.make(1, 2, 2, tq, 600, 64, dtype, seed=5)
    table[2] = torch.finfo(table.dtype).min
    m[m.numel() // 2] = 0
    from stft_mel_spectrogram_amd import relative_attention
    hidden = table.clone()
    hidden[2] = -math.inf
    assert torch.equal(relative_attention(q, k, v, table, m), relative_attention(q, k, v, hidden, m))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tq", [1, 7])
@pytest.mark.parametrize("tk", [300, 1500, 5000])
def test_nan_past_the_lengths_of_a_cache(tk, tq, dtype):
    """The kernel for few queries, in one range and in several."""
    q, k, v, table, m, do = plain.make(2, 4, 2, tq, tk, 64, dtype, seed=tk, layout="bhtd")
    ends = (tk - 37, tk // 3 + 1)
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for how in (dict(lengths=lengths), dict(lengths=lengths, causal=True, offset=lengths - tq)):
        clean = plain.run_case(q, k, v, table, m, do, backward=False, **how)
        k2, v2 = k.clone(), v.clone()
        for e, n in enumerate(ends):
            k2[e, :, n:], v2[e, :, n:] = math.nan, math.inf
        assert torch.equal(plain.run_case(q, k2, v2, table, m, do, backward=False, **how), clean)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,hk,t,d,far", [
    (2, 2, 70, 40, 20), (4, 1, 300, 64, 60), (2, 2, 90, 33, 20), (2, 1, 140, 128, 300), (3, 3, 75, 96, 5),
    # few query blocks: ranges of the keys
    (2, 1, 1030, 64, 60), (1, 1, 515, 40, 20), (3, 3, 777, 33, 300), (2, 2, 900, 128, 20)])
def test_gradients_without_the_tables(h, hk, t, d, far, dtype):
    """A table that is not trained: dq from kernels of their own."""
    from stft_mel_spectrogram_amd import relative_attention
    q, k, v, table, m, do = plain.make(2, h, hk, t, t, d, dtype, seed=t, far=far)
    for causal, second in ((False, t // 3), (True, t), (True, 0)):
        lengths = torch.tensor([t, second], dtype=torch.int32, device="cuda")
        leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
        relative_attention(*leaves, table, m, causal=causal, key_lengths=lengths).backward(do)
        grads, tols = plain.reference(q, k, v, table, m, do, d ** -0.5, causal, lengths,
                                      torch.zeros(2, device="cuda"))[4:]
        for leaf, name in zip(leaves, ("dq", "dk", "dv")):
            plain.close(name, leaf.grad, grads[name], tols[name])
