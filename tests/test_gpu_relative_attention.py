"""Attention with a learned relative position bias against a plain float64
implementation on the same inputs.

Tolerances, elementwise.  U = 2^-24, h = half a step of the element type
(eps / 2).  A score is off by at most S = U ((D + 8) scale sum|q k| + 8 (|s| +
|max|)); probabilities by 4 S + 64 U relative; they are rounded once (h) for
their product, and so are the score gradients ds; every result is rounded
once (h |result|).  So, with sums over absolute values:
  o       h |o| + (h + P) sum p |v|,                       P = 4 S + 64 U
  ds      E = p [P (|dp| + |delta|) + 2 D U (sum|do v| + sum|do o|)
                 + (h + P) sum_d |do| (sum p |v| + |o|)]    (delta from the rounded o)
  dq      h |dq| + scale sum (E + h |ds|) |k|,  dk the same over queries
  dv      h |dv| + (h + P) sum p |do|
  dtable  h |dtable| + sum E + U (64 + pairs / 64) sum |ds|
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reference(q, k, v, table, buckets, do, scale, causal, lengths, offset):
    """Results, gradients and their tolerances (without the rounding of the
    result itself)."""
    b, h, tq, d = q.shape
    hk, tk = k.shape[1:3]
    dt, dev, g = q.dtype, q.device, h // hk
    half = torch.finfo(dt).eps / 2
    qd = q.double()
    kd, vd = (t.double().repeat_interleave(g, 1) for t in (k, v))
    far = (buckets.numel() - 1) // 2
    pos = offset.long()[:, None] + torch.arange(tq, device=dev)
    j = torch.arange(tk, device=dev)
    seen = (j < lengths.long()[:, None])[:, None].expand(b, tq, tk)
    if causal:
        seen = seen & (j <= pos[..., None])
    # keys past a length may hold anything
    past = (j >= lengths.long()[:, None])[:, None, :, None]
    kd, vd = (torch.where(past, torch.zeros_like(t), t) for t in (kd, vd))
    bucket = buckets.long()[(j - pos[..., None]).clamp(-far, far) + far]      # [b, tq, tk]
    has = (bucket >= 0) & (bucket < table.shape[0])
    bias = table.double()[torch.where(has, bucket, torch.zeros_like(bucket))].permute(0, 3, 1, 2)
    bias = torch.where(has[:, None], bias, torch.zeros_like(bias))
    s = qd @ kd.transpose(-1, -2) * scale + bias
    sabs = scale * (qd.abs() @ kd.abs().transpose(-1, -2))
    s = torch.where(seen[:, None], s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True) if tk else torch.full((b, h, tq, 1), -math.inf, device=dev, dtype=torch.float64)
    m0 = torch.where(m.isinf(), torch.zeros_like(m), m)
    e = (s - m0).exp()
    z = e.sum(-1, keepdim=True)
    p = e / torch.where(z == 0, torch.ones_like(z), z)
    lse = torch.where(z == 0, torch.full_like(z, -math.inf), z.log() + m0)[..., 0]
    o = p @ vd
    dod = do.double()
    dp = dod @ vd.transpose(-1, -2)
    delta = (dod * o).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    rel = 4 * U * ((d + 8) * sabs + 8 * (s.abs().nan_to_num(posinf=0) + m0.abs())) + 64 * U
    rel = torch.where(seen[:, None], rel, torch.zeros_like(rel))
    rel = rel + rel.amax(-1, keepdim=True) if tk else rel  # its own score's and the sum's
    fold = lambda t: t.view(b, hk, g, *t.shape[2:]).sum(2)  # noqa: E731
    pe = p * rel
    o_tol = (half * p + pe) @ vd.abs()
    err = p * (rel * (dp.abs() + delta.abs())
               + 2 * d * U * (dod.abs() @ vd.abs().transpose(-1, -2) + (dod * o).abs().sum(-1, keepdim=True))
               + ((dod.abs() * (o_tol + half * (p @ vd.abs() + o.abs())))).sum(-1, keepdim=True))
    wds = err + half * ds.abs()
    grads = dict(dq=ds @ kd * scale, dk=fold(ds.transpose(-1, -2) @ qd) * scale,
                 dv=fold(p.transpose(-1, -2) @ dod))
    tols = dict(dq=scale * (wds @ kd.abs()), dk=scale * fold(wds.transpose(-1, -2) @ qd.abs()),
                dv=fold((half * p + pe).transpose(-1, -2) @ dod.abs()))
    dtab = torch.zeros(table.shape, dtype=torch.float64, device=dev)
    dtab_tol = torch.zeros_like(dtab)
    idx = torch.where(has, bucket, torch.zeros_like(bucket)).reshape(-1)
    n_tol = U * (64 + b * tq * tk / 64)
    for i in range(h):
        keep = has.reshape(-1).double()
        dtab[:, i].index_add_(0, idx, ds[:, i].reshape(-1) * keep)
        dtab_tol[:, i].index_add_(0, idx, (err[:, i] + n_tol * ds[:, i].abs()).reshape(-1) * keep)
    grads["dtable"], tols["dtable"] = dtab, dtab_tol
    return o, o_tol, lse, rel.amax(-1) if tk else torch.zeros_like(lse), grads, tols


def close(name, got, ref, tol):
    if ref.numel() == 0:
        return
    fi = torch.finfo(got.dtype)
    tol = tol + fi.eps / 2 * ref.abs() + fi.smallest_normal * fi.eps + 1e-30
    assert torch.isfinite(got).all(), name
    worst = ((got.double() - ref).abs() / tol).max().item()
    print(f"[{name}] worst error / tolerance {worst:.3g}")
    assert worst <= 1.0, (name, worst)


def make(b, h, hk, tq, tk, d, dtype, seed=0, layout="bthd", far=20, buckets=12, table32=False, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DT[dtype]
    if layout == "bthd":
        q = (r(b, tq, h, d) * std).to(dt).transpose(1, 2)
        k, v = ((r(b, tk, hk, d) * s).to(dt).transpose(1, 2) for s in (std, 1.0))
        do = r(b, tq, h, d).to(dt).transpose(1, 2)
    else:
        q, do = (r(b, h, tq, d) * std).to(dt), r(b, h, tq, d).to(dt)
        k, v = (r(b, hk, tk, d) * std).to(dt), r(b, hk, tk, d).to(dt)
    table = r(buckets, h).to(torch.float32 if table32 else dt)
    m = torch.randint(0, buckets, (2 * far + 1,), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, table, m, do


def run_case(q, k, v, table, m, do, scale=None, causal=False, lengths=None, offset=0, backward=True):
    from stft_mel_spectrogram_amd import (relative_attention, relative_attention_backward,
                                          relative_attention_forward)
    b, h, tq, d = q.shape
    how = dict(scale=scale, causal=causal, key_lengths=lengths, query_offset=offset)
    o, stats = relative_attention_forward(q, k, v, table, m, **how)
    full = torch.full((b,), k.shape[2], device="cuda") if lengths is None else lengths.clamp(0, k.shape[2])
    off = offset if isinstance(offset, torch.Tensor) else torch.full((b,), offset, device="cuda")
    ro, o_tol, lse, lse_tol, grads, tols = reference(q, k, v, table, m, do, d ** -0.5 if scale is None else scale,
                                                     causal, full, off)
    close("o", o, ro, o_tol)
    empty = lse == -math.inf
    assert torch.equal(stats == -math.inf, empty)
    assert (o[empty] == 0).all()
    fin = ~empty
    close("lse", torch.where(fin, stats, torch.zeros_like(stats)),
          torch.where(fin, lse, torch.zeros_like(lse)), lse_tol + 64 * U * (1 + lse.abs().nan_to_num(posinf=0)))
    assert torch.equal(relative_attention(q, k, v, table, m, **how), o)
    if not backward:
        return o
    got = dict(zip(("dq", "dk", "dv", "dtable"),
                   relative_attention_backward(do, q, k, v, table, m, o, stats, **how)))
    for name in got:
        close(name, got[name], grads[name], tols[name])
    again = relative_attention_backward(do, q, k, v, table, m, o, stats, **how)
    for a, e in zip(again, got.values()):
        assert torch.equal(a, e)
    return o, got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [1, 8, 33, 40, 64, 72, 80, 96, 127, 128])
def test_head_dims(d, dtype):
    run_case(*make(2, 2, 2, 70, 75, d, dtype, seed=d))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tq,tk", [(1, 1), (1, 2), (17, 1), (31, 33), (32, 32), (64, 64), (65, 127), (128, 128),
                                   (129, 257), (300, 45), (40, 700)])
def test_lengths(tq, tk, dtype):
    run_case(*make(1, 3, 3, tq, tk, 64, dtype, seed=tq))
    run_case(*make(1, 3, 3, tq, tk, 64, dtype, seed=tq + 1), causal=True, offset=tk - tq)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,hk", [(4, 1), (4, 2), (6, 2), (20, 1), (5, 5)])
def test_shared_key_heads(h, hk, dtype):
    run_case(*make(2, h, hk, 50, 61, 64, dtype, seed=h))
    run_case(*make(2, h, hk, 50, 61, 128, dtype, seed=h, layout="bhtd"), causal=True)
    run_case(*make(2, h, hk, 1, 61, 96, dtype, seed=h), causal=True, offset=60)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tq", [1, 2, 7, 16, 17, 40])
def test_new_tokens_against_a_cache(tq, dtype):
    # ragged caches, several key ranges and their join, offsets from the cache lengths
    for d, tk, h, hk in ((64, 1501, 4, 4), (128, 3000, 8, 2), (80, 260, 2, 1)):
        q, k, v, table, m, do = make(3, h, hk, tq, tk, d, dtype, seed=tq + d, layout="bhtd")
        lengths = torch.tensor([tk, tk // 2 + 1, max(tq, 3)], dtype=torch.int32, device="cuda")
        run_case(q, k, v, table, m, do, causal=True, lengths=lengths, offset=lengths - tq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ragged_lengths_and_empty_rows(dtype):
    for causal in (False, True):
        q, k, v, table, m, do = make(5, 2, 2, 90, 100, 64, dtype, seed=3)
        lengths = torch.tensor([100, 0, 1, 64, 500], dtype=torch.int32, device="cuda")  # 500: clamped
        run_case(q, k, v, table, m, do, causal=causal, lengths=lengths)
        # the first queries lie before every key
        run_case(q, k, v, table, m, do, causal=causal, lengths=lengths, offset=-37)
    for tq in (1, 3):
        q, k, v, table, m, do = make(3, 2, 2, tq, 50, 64, dtype, seed=4)
        run_case(q, k, v, table, m, do, lengths=torch.tensor([0, 50, 1], dtype=torch.int32, device="cuda"))
        run_case(q, k, v, table, m, do, causal=True, offset=-2)


def test_no_keys_and_no_queries():
    from stft_mel_spectrogram_amd import relative_attention, relative_attention_backward, relative_attention_forward
    for tq in (1, 40):
        o, g = run_case(*make(2, 2, 2, tq, 0, 64, "bf16"))
        assert (o == 0).all() and (g["dq"] == 0).all() and (g["dtable"] == 0).all()
    q, k, v, table, m, do = make(2, 2, 2, 0, 30, 64, "bf16")
    o, stats = relative_attention_forward(q, k, v, table, m)
    assert o.shape == (2, 2, 0, 64)
    dq, dk, dv, dt = relative_attention_backward(do, q, k, v, table, m, o, stats)
    assert (dk == 0).all() and (dv == 0).all() and (dt == 0).all()
    q, k, v, table, m, do = make(0, 2, 2, 4, 30, 64, "bf16")
    assert relative_attention(q, k, v, table, m).shape == (0, 2, 4, 64)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_nan_past_the_lengths_does_no_harm(dtype):
    for tq in (1, 60):
        q, k, v, table, m, do = make(2, 4, 2, tq, 150, 64, dtype, seed=5)
        lengths = torch.tensor([70, 33], dtype=torch.int32, device="cuda")
        clean = run_case(q, k, v, table, m, do, lengths=lengths)
        for e, n in enumerate((70, 33)):
            k[e, :, n:], v[e, :, n:] = math.nan, math.inf
        o, g = run_case(q, k, v, table, m, do, lengths=lengths)
        assert torch.equal(o, clean[0])
        for name in g:
            assert torch.equal(g[name], clean[1][name]), name
        assert (g["dk"][0, :, 70:] == 0).all() and (g["dv"][1, :, 33:] == 0).all()


@pytest.mark.parametrize("far,buckets", [(0, 1), (1, 3), (5, 4), (128, 32), (1024, 1024)])
def test_bias_maps(far, buckets):
    for dtype in ("f32", "bf16"):
        run_case(*make(1, 2, 2, 200, 190, 64, dtype, seed=far, far=far, buckets=buckets))
        run_case(*make(1, 2, 2, 3, 1300, 64, dtype, seed=far, far=far, buckets=buckets), causal=True, offset=1297)


def test_distances_without_a_bucket_and_masking_bias():
    q, k, v, table, m, do = make(1, 2, 2, 80, 80, 64, "f32", seed=6)
    m[3], m[30] = -1, 12
    run_case(q, k, v, table, m, do)
    # a bucket of -inf hides its pairs; of the type's lowest value, too
    for low in (-math.inf, torch.finfo(torch.float32).min / 4):
        t2 = table.clone()
        t2[2] = low
        m2 = m.clone()
        m2[m.numel() // 2] = 0  # every query keeps itself
        run_case(q, k, v, t2, m2, do)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_float32_table(dtype):
    _, g = run_case(*make(2, 2, 2, 70, 75, 64, dtype, table32=True))
    assert g["dtable"].dtype == torch.float32


def test_packed_projection_and_other_strides():
    for dtype in ("f32", "bf16"):
        g = torch.Generator(device="cuda")
        g.manual_seed(8)
        qkv = torch.randn(2, 77, 3, 4, 64, generator=g, device="cuda").to(DT[dtype])
        q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        _, _, _, table, m, do = make(2, 4, 4, 77, 77, 64, dtype, seed=8)
        run_case(q, k, v, table, m, do)
        # odd element offsets and strides
        wide = torch.randn(2, 4, 77, 71, generator=g, device="cuda").to(DT[dtype])
        run_case(wide[..., 3:66], wide[..., 5:68], wide[..., 1:64], table, m, do[..., :63])
        # keys shared by all entries
        run_case(q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), table, m, do)


def test_scale_and_large_scores():
    run_case(*make(1, 2, 2, 100, 100, 64, "f32", seed=9, std=4.0))
    run_case(*make(1, 2, 2, 100, 100, 64, "bf16", seed=9, std=3.0), scale=0.5)
    run_case(*make(1, 2, 2, 1, 900, 64, "bf16", seed=9, std=3.0), scale=0.5)


@pytest.mark.parametrize("size", [1e-4, 3e4])
def test_float16_gradients_keep_small_and_large_scales(size):
    q, k, v, table, m, do = make(1, 2, 2, 300, 310, 64, "f16", seed=10)
    table = table.float()
    do = (do.float() * size / 4).clamp(-6e4, 6e4).half()
    from stft_mel_spectrogram_amd import relative_attention_backward, relative_attention_forward
    o, stats = relative_attention_forward(q, k, v, table, m)
    got = relative_attention_backward(do, q, k, v, table, m, o, stats)
    ref = reference(q, k, v, table, m, do, 64 ** -0.5, False, torch.tensor([310], device="cuda"),
                    torch.tensor([0], device="cuda"))[4]
    # relative to the gradient's size: the roundings of p, ds, o and the result, and float16's
    # smallest step where the result itself is subnormal
    for g, name in zip(got, ("dq", "dk", "dv", "dtable")):
        r = ref[name]
        floor = 0 if g.dtype == torch.float32 else 2.0 ** -25 * math.sqrt(r.numel())
        assert (g.double() - r).norm() <= 4 * 2.0 ** -11 * r.norm() + floor, name


def test_autograd():
    from stft_mel_spectrogram_amd import relative_attention
    q, k, v, table, m, do = make(2, 4, 2, 60, 66, 64, "bf16", seed=11)
    _, g = run_case(q, k, v, table, m, do, causal=True, offset=6)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v, table)]
    relative_attention(*leaves, m, causal=True, query_offset=6).backward(do)
    for leaf, name in zip(leaves, ("dq", "dk", "dv", "dtable")):
        assert torch.equal(leaf.grad, g[name]), name
    only = table.clone().requires_grad_(True)
    off = torch.full((2,), 6, dtype=torch.int32, device="cuda")
    relative_attention(q, k, v, only, m, causal=True, query_offset=off).backward(do)
    assert torch.equal(only.grad, g["dtable"])
    q2 = q.clone().requires_grad_(True)
    relative_attention(q2, k, v, table, m).sum().backward()  # an expanded gradient
    assert torch.isfinite(q2.grad).all()


def test_gradient_against_differences():
    q, k, v, table, m, do = make(1, 2, 1, 9, 11, 16, "f32", seed=12, far=4, buckets=5)
    from stft_mel_spectrogram_amd import relative_attention_backward, relative_attention_forward
    o, stats = relative_attention_forward(q, k, v, table, m, causal=True, query_offset=2)
    got = relative_attention_backward(do, q, k, v, table, m, o, stats, causal=True, query_offset=2)

    def value(*xs):
        o = reference(*xs, m, do, 0.25, True, torch.tensor([11], device="cuda"),
                      torch.tensor([2], device="cuda"))[0]
        return (o * do.double()).sum().item()

    base = [t.double() for t in (q, k, v, table)]
    # reference() rounds nothing of float64 inputs; finfo(float64) enters its tolerances only
    step = 1e-5
    for which, g in enumerate(got):
        flat = g.reshape(-1)
        for at in (0, flat.numel() // 2, flat.numel() - 1):
            vals = []
            for sign in (1, -1):
                xs = [t.clone() for t in base]
                x = xs[which].contiguous()
                x.view(-1)[at] += sign * step
                xs[which] = x
                vals.append(value(*xs))
            num = (vals[0] - vals[1]) / (2 * step)
            # h^2 of the differences, 1e-16 * 100 / h of their rounding, 2^-24 * some hundred of the kernel
            assert abs(num - flat[at].item()) <= 1e-6 + 512 * U * 4, (which, at)


def test_out_and_layout_of_results():
    from stft_mel_spectrogram_amd import relative_attention
    q, k, v, table, m, do = make(2, 3, 3, 20, 21, 64, "bf16", seed=13)
    o = relative_attention(q, k, v, table, m)
    assert o.transpose(1, 2).is_contiguous()  # as q
    out = torch.zeros(2, 3, 20, 64, dtype=torch.bfloat16, device="cuda")
    assert relative_attention(q, k, v, table, m, out=out) is out and torch.equal(out, o)


def test_another_stream_and_graph_replays():
    from stft_mel_spectrogram_amd import (relative_attention, relative_attention_backward,
                                          relative_attention_forward)
    for dtype in ("bf16", "f16"):
        q, k, v, table, m, do = make(2, 4, 2, 150, 160, 64, dtype, seed=14)
        t1, kc, vc = q[:, :, :1], k.contiguous(), v.contiguous()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, stats = relative_attention_forward(q, k, v, table, m)
            relative_attention_backward(do, q, k, v, table, m, o, stats)
            relative_attention(t1, kc, vc, table, m, causal=True, query_offset=159)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        sq, sdo = q.clone(), do.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go, gs = relative_attention_forward(sq, k, v, table, m)
            gg = relative_attention_backward(sdo, sq, k, v, table, m, go, gs)
            gt = relative_attention(sq[:, :, :1], kc, vc, table, m, causal=True, query_offset=159)
        for seed in range(3):
            nq, _, _, _, _, ndo = make(2, 4, 2, 150, 160, 64, dtype, seed=40 + seed)
            sq.copy_(nq)
            sdo.copy_(ndo)
            graph.replay()
            torch.cuda.synchronize()
            eo, es = relative_attention_forward(nq, k, v, table, m)
            eg = relative_attention_backward(ndo, nq, k, v, table, m, eo, es)
            et = relative_attention(nq[:, :, :1], kc, vc, table, m, causal=True, query_offset=159)
            torch.cuda.synchronize()
            for a, e in zip((go, gt, *gg), (eo, et, *eg)):
                assert torch.equal(a, e)


def test_relative_buckets():
    from stft_mel_spectrogram_amd import relative_buckets
    b = relative_buckets(32, 128)
    assert b.dtype == torch.int32 and b.is_cuda and b.numel() == 257


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,hk,tq,tk,d", [
    (4, 1, 7, 2500, 40),   # 28 rows of a key head, key ranges
    (2, 2, 32, 300, 64),   # the most queries, no ranges
    (6, 2, 11, 257, 128),  # the fewest keys, three fragments with a short last one
    (3, 3, 17, 2048, 33),  # odd rows
    (8, 1, 1, 2100, 96),
])
def test_few_queries_against_a_cache(h, hk, tq, tk, d, dtype):
    q, k, v, table, m, do = make(2, h, hk, tq, tk, d, dtype, seed=tk + d, layout="bhtd", far=40)
    lengths = torch.tensor([tk, tk // 3], device="cuda", dtype=torch.int32)
    offset = torch.tensor([tk - tq, tk // 3 - tq], device="cuda", dtype=torch.int32)
    run_case(q, k, v, table, m, do, causal=True, lengths=lengths, offset=offset, backward=False)
    run_case(q, k, v, table, m, do, lengths=lengths, offset=offset, backward=False)
    # an entry without keys, one whose queries lie before every key
    lengths[1], offset[0] = 0, -tq
    run_case(q, k, v, table, m, do, causal=True, lengths=lengths, offset=offset, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,hk,t,d", [(4, 1, 300, 40), (6, 2, 517, 64), (8, 1, 140, 128), (2, 2, 530, 33)])
def test_shares_of_queries(h, hk, t, d, dtype):
    """Few key blocks: dk and dv from several workgroups each."""
    q, k, v, table, m, do = make(2, h, hk, t, t, d, dtype, seed=t)
    lengths = torch.tensor([t, t // 2 + 3], device="cuda", dtype=torch.int32)
    for causal in (False, True):
        run_case(q, k, v, table, m, do, causal=causal, lengths=lengths)
    lengths[0] = 0
    run_case(q, k, v, table, m, do, lengths=lengths)


@pytest.mark.parametrize("tk", [1024, 1500, 5000])
def test_ranges_of_many_queries(tk):
    q, k, v, table, m, do = make(2, 2, 2, 150, tk, 72, "bf16", seed=tk)
    lengths = torch.tensor([tk, 3], device="cuda", dtype=torch.int32)
    run_case(q, k, v, table, m, do, lengths=lengths, backward=False)
    lengths[1] = 0
    run_case(q, k, v, table, m, do, causal=True, lengths=lengths, offset=tk - 150, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,hk,t,d,far", [(2, 1, 1030, 64, 60), (1, 1, 515, 40, 20), (3, 3, 777, 33, 300), (2, 2, 900, 128, 20)])
def test_ranges_of_keys_in_the_backward(h, hk, t, d, far, dtype):
    """Few query blocks: dq and the bias table's gradient from several key ranges."""
    q, k, v, table, m, do = make(2, h, hk, t, t, d, dtype, seed=t, far=far)
    lengths = torch.tensor([t, t // 3], device="cuda", dtype=torch.int32)
    for causal in (False, True):
        run_case(q, k, v, table, m, do, causal=causal, lengths=lengths)
    lengths[0] = 0
    run_case(q, k, v, table, m, do, lengths=lengths)
