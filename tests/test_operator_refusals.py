"""Refusals of the speech-model operators, on the CPU: the C ABI checks every
argument before any HIP call, so made-up device addresses are never used."""
import ctypes
import math

import pytest

from stft_mel_spectrogram_amd import _native as N

torch = pytest.importorskip("torch")
P = 1 << 20  # an address that must not be touched


def norm(rows=4, width=8, x=P, stride=8, w=P, b=P, y=P, eps=1e-5, dtype=N.FM_F32, pdtype=N.FM_F32):
    return N.lib.fm_layer_norm_forward(x, stride, w, b, y, None, None, rows, width, eps, dtype, pdtype, None)


def norm_back(rows=4, width=8, dy=P, x=P, w=P, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P, dtype=N.FM_F32,
              pdtype=N.FM_F32, stride=8):
    return N.lib.fm_layer_norm_backward(dy, stride, x, stride, w, mean, rstd, dx, dw, db, ws, rows, width, dtype,
                                        pdtype, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=-3), dict(dtype=N.FM_I16), dict(dtype=9),
    dict(dtype=N.FM_BF16, pdtype=N.FM_F16), dict(w=None), dict(x=None), dict(y=None), dict(eps=-1.0),
    dict(eps=math.nan), dict(eps=math.inf), dict(stride=-8), dict(x=P + 2), dict(y=P + 1)])
def test_layer_norm_forward_refuses(kw):
    assert norm(**kw) == N.FM_E_INVAL
    assert b"layer norm" in N.lib.fm_last_error()


def test_layer_norm_limits():
    assert norm(width=(1 << 20) + 1) == N.FM_E_UNSUPPORTED
    assert norm(rows=0, x=None, y=None) == N.FM_OK  # nothing to do, nothing launched
    assert N.lib.fm_layer_norm_backward_workspace(4, 0, N.FM_F32) == N.FM_E_INVAL
    assert N.lib.fm_layer_norm_backward_workspace(16, 1024, N.FM_BF16) == 0  # one workgroup
    for rows, width in ((500, 1), (50, 1000), (100000, 1024), (100000, 30000)):
        parts = N.lib.fm_layer_norm_backward_workspace(rows, width, N.FM_BF16) / (8 * width)
        assert parts == int(parts) and 1 <= parts <= 1024


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(dtype=N.FM_I16), dict(dtype=N.FM_F16, pdtype=N.FM_BF16), dict(dy=None),
    dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None, rows=5000), dict(ws=P + 4, rows=5000), dict(dw=None),
    dict(w=None), dict(stride=-1), dict(dx=P + 2)])
def test_layer_norm_backward_refuses(kw):
    assert norm_back(**kw) == N.FM_E_INVAL


def score(rows=4, vocab=100, x=P, stride=100, tok=P, bits=64, ids=P, tops=P, ws=P, top=5, dtype=N.FM_F32):
    return N.lib.fm_token_logprobs(x, stride, tok, bits, P, P, P, ids, tops, ws, rows, vocab, top, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 31) - 1), dict(top=-1), dict(top=65),
    dict(vocab=4, top=5), dict(dtype=N.FM_I16), dict(bits=16), dict(x=None), dict(tok=None), dict(ids=None),
    dict(tops=None), dict(stride=-1), dict(x=P + 1), dict(tok=P + 4), dict(vocab=50000, ws=None),
    dict(vocab=50000, ws=P + 8)])
def test_token_logprobs_refuses(kw):
    assert score(**kw) == N.FM_E_INVAL
    assert b"token log probabilities" in N.lib.fm_last_error()


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(tok=None), dict(lse=None), dict(dx=None), dict(ent=None), dict(ids=None), dict(top=0),
    dict(bits=8), dict(dtype=7), dict(vocab=0), dict(rows=-2), dict(stride=-1), dict(dx=P + 3)])
def test_token_logprobs_backward_refuses(kw):
    a = dict(rows=4, vocab=100, x=P, stride=100, tok=P, bits=64, lse=P, ent=P, ids=P, dx=P, top=5, dtype=N.FM_F32)
    a.update(kw)
    assert N.lib.fm_token_logprobs_backward(a["x"], a["stride"], a["tok"], a["bits"], a["lse"], a["ent"], P, P,
                                            a["ids"], P, a["dx"], a["rows"], a["vocab"], a["top"], a["dtype"],
                                            None) == N.FM_E_INVAL


def attention(backward=False, ws=P, **kw):
    a = N.AttentionArgs()
    v = dict(dtype=N.FM_BF16, table_dtype=N.FM_BF16, causal=0, far=8, num_buckets=4, batch=2, heads=4, kv_heads=2,
             q_len=100, k_len=100, head_dim=64, query_offset_value=0, scale=0.125)
    v.update({n: P for n in ("q", "k", "v", "table", "bucket_map", "o", "lse", "grad_o", "grad_q", "grad_k",
                             "grad_v", "grad_table")})
    v.update({f"{t}_stride_{x}": 64 for t in ("q", "k", "v", "o", "grad_o", "grad_q", "grad_k", "grad_v")
              for x in ("entry", "head", "time")})
    v.update(kw)
    for name, value in v.items():
        setattr(a, name, value)
    fn = N.lib.fm_attention_backward if backward else N.lib.fm_attention_forward
    return fn(ctypes.byref(a), ws, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [
    dict(dtype=N.FM_I16), dict(table_dtype=N.FM_F16), dict(batch=-1), dict(heads=0), dict(kv_heads=0),
    dict(kv_heads=3), dict(q_len=-1), dict(k_len=-5), dict(k_len=1 << 30), dict(head_dim=0), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-60), dict(far=-1),
    dict(num_buckets=0), dict(query_offset_value=1 << 31), dict(q=None), dict(k=None), dict(v=None), dict(o=None),
    dict(table=None), dict(bucket_map=None), dict(q=P + 1), dict(key_lengths=P + 2), dict(k_stride_time=-64),
    dict(heads=60000, kv_heads=60000, batch=60000)])
def test_attention_refuses(kw, backward):
    assert attention(backward, **kw) == N.FM_E_INVAL
    assert b"attention" in N.lib.fm_last_error()


@pytest.mark.parametrize("kw", [dict(lse=None), dict(grad_o=None), dict(grad_q=None), dict(grad_k=None),
                                dict(grad_v=None), dict(ws=None), dict(ws=P + 8), dict(grad_k_stride_head=-1)])
def test_attention_backward_refuses(kw):
    assert attention(True, **kw) == N.FM_E_INVAL


def test_attention_limits():
    for kw in (dict(head_dim=129), dict(far=1025), dict(num_buckets=1025)):
        assert attention(**kw) == N.FM_E_UNSUPPORTED
    assert attention(q_len=0, q=None, o=None, ws=None) == N.FM_OK
    assert attention(batch=0, ws=None) == N.FM_OK
    # long keys and few rows need the workspace of the key ranges
    assert attention(q_len=1, k_len=100000, ws=None) == N.FM_E_INVAL
    assert N.lib.fm_attention_forward(None, None, None) == N.FM_E_INVAL
    assert N.lib.fm_attention_workspace(None, 1) == N.FM_E_INVAL


def test_python_callers_refuse_tensors_off_the_gpu():
    from stft_mel_spectrogram_amd import layer_norm, relative_attention, token_logprobs
    x = torch.zeros(2, 4, 8, 16)
    with pytest.raises(ValueError, match="GPU"):
        layer_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        token_logprobs(x, torch.zeros(2, 4, 8, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        relative_attention(x, x, x, x, x)
    with pytest.raises(ValueError, match="tensor"):
        layer_norm([1.0])


@pytest.mark.parametrize("buckets,distance,both", [(32, 128, True), (32, 128, False), (32, 800, True), (8, 17, False),
                                                   (4, 2, True), (2, 2, False), (64, 1024, True), (5, 40, True)])
def test_relative_buckets_on_the_cpu(buckets, distance, both):
    """Against 60-digit logarithms; borders where the logarithm's ratio is a whole number go up."""
    import decimal
    from stft_mel_spectrogram_amd import relative_buckets
    got = relative_buckets(buckets, distance, both, device="cpu").tolist()
    assert len(got) == 2 * distance + 1
    side = buckets // 2 if both else buckets
    near = side // 2
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        tie = decimal.Decimal(10) ** -40

        def one(n):
            if n < near:
                return n
            r = (side - near) * (decimal.Decimal(n) / near).ln() / (decimal.Decimal(distance) / near).ln()
            return min(side - 1, near + int(r + tie))

        for d in range(-distance, distance + 1):
            want = one(abs(d)) + (side if d > 0 else 0) if both else one(max(-d, 0))
            assert got[d + distance] == want, d
    assert set(got) <= set(range(buckets))


@pytest.mark.parametrize("args", [(1, 128, False), (3, 128, True), (1025, 4000, True), (32, 8, True), (32, 1025, True)])
def test_relative_buckets_refuse(args):
    from stft_mel_spectrogram_amd import relative_buckets
    with pytest.raises(ValueError):
        relative_buckets(*args, device="cpu")
