"""The gated recurrence and its gradients against a 64-bit loop over the frames.

Tolerances.  With y = f log2 e rounded once and log2 e off by 0.22 of 2^-24, an
exponential is off by 2^-24 (1.25 |f| + 2), and sigmoid(f), 1 - sigmoid(f) and
silu by eta = 2^-24 (6 + 1.25 |f|) of themselves.  A state is a sum of products
of these; the errors obey the recurrence itself on absolute values: E = a E' + eta (a
H' + |u|) + 2^-24 J (a H' + |u|), H = a H' + |u|.  J = 4 counts the roundings of a frame's
own steps; the joins of ranges (frames of a lane, 6 lane exchanges, 8 waves, tiles and
time ranges) add 2^-24 (32 + tiles) H once.  The same holds for m, backwards in time.
Results in 16 bits add half a step.  An exponential past 2^128 makes its sigmoid 0, and
results below 2^-126 become 0, so sigmoids below 2^-126 may be lost: each frame's are
off by 2^-126 absolutely, times the factors that go with them.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(b, t, c, dtype, seed, gate=True, state=True, shift=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = r(b, t, 3 * c)
    p[..., c:2 * c] = p[..., c:2 * c] * 2 + shift
    p = p.to(dtype)
    return dict(x=p[..., :c], forget=p[..., c:2 * c], gate=p[..., 2 * c:] if gate else None,
                state=r(b, c) if state else None, dy=r(b, t, c).to(dtype), dlast=r(b, c) if state else None)


def reference(s, lengths=None):
    """Results, gradients and their tolerances without the rounding to the type."""
    x, f, dy = s["x"].double(), s["forget"].double(), s["dy"].double()
    b, t, c = x.shape
    zero = torch.zeros(b, c, dtype=torch.float64, device=x.device)
    g = s["gate"].double() if s["gate"] is not None else None
    n = torch.full((b,), t, device=x.device) if lengths is None else lengths.clamp(0, t)
    on = torch.arange(t, device=x.device) < n[:, None]
    x, f, dy = (torch.where(on[..., None], v, torch.zeros_like(v)) for v in (x, f, dy))
    a, rest = torch.sigmoid(f), torch.sigmoid(-f)
    eta = U * (6 + 1.25 * f.abs())
    sl, dsl, eta_g = torch.ones_like(x), torch.zeros_like(x), torch.zeros_like(x)
    sg = torch.zeros_like(x)
    if g is not None:
        g = torch.where(on[..., None], g, torch.zeros_like(g))
        sg = torch.sigmoid(g)
        sl, dsl, eta_g = g * sg, sg * (1 + g * (1 - sg)), U * (6 + 1.25 * g.abs())
    joins = U * (32 + t / 64)
    h = s["state"].double() if s["state"] is not None else zero
    E, H = zero, h.abs()
    hs, Es, Hs, before = [], [], [], []
    for i in range(t):
        m = on[:, i, None]
        before.append(h)
        mag = a[:, i] * H + (rest[:, i] * x[:, i]).abs()
        E = torch.where(m, a[:, i] * E + (eta[:, i] + 4 * U) * mag, E)
        h = torch.where(m, a[:, i] * h + rest[:, i] * x[:, i], h)
        H = torch.where(m, mag, H)
        hs.append(h), Es.append(E + joins * H), Hs.append(H)
    st = lambda v: torch.stack(v, 1) if v else x  # noqa: E731
    h_all, E_all, H_all, before = st(hs), st(Es), st(Hs), st(before)
    keep = on[..., None]
    y = h_all * sl * keep
    out = dict(y=(y, (E_all * sl.abs() + (eta_g + U) * y.abs()) * keep), last=(h, E + joins * H))
    d = s["dlast"].double() if s["dlast"] is not None else zero
    F, D = zero, d.abs()
    ds, Fs, Ds = [None] * t, [None] * t, [None] * t
    for i in reversed(range(t)):
        m = on[:, i, None]
        e = dy[:, i] * sl[:, i]
        mag = e.abs() + D
        F_in = F + (eta_g[:, i] + 2 * U) * e.abs()
        dd = e + d
        ds[i], Fs[i], Ds[i] = dd, F_in + joins * mag + U * mag, mag
        d = torch.where(m, a[:, i] * dd, d)
        F = torch.where(m, a[:, i] * F_in + (eta[:, i] + 4 * U) * a[:, i] * mag, F)
        D = torch.where(m, a[:, i] * mag, D)
    dd, Fd, _ = st(ds), st(Fs), None
    dx = rest * dd * keep
    tx = (rest * Fd + (eta + 2 * U) * dx.abs()) * keep
    # (1 - a) d (h - x): h - x = a (h' - x)
    df = dx * (h_all - x)
    tf = tx * (h_all - x).abs() + dx.abs() * (E_all + 2 * U * (h_all.abs() + x.abs())) + 2 * U * df.abs()
    out |= dict(dx=(dx, tx), dforget=(df, tf))
    if g is not None:
        dg = dy * h_all * dsl * keep
        out["dgate"] = (dg, (dy.abs() * (E_all * dsl.abs() + H_all * 4 * (eta_g + U) * (sg + sl.abs()))) * keep)
    if s["state"] is not None:
        out["dstate"] = (d, F + joins * D + U * D)
    big = 1 + max(v.abs().max().item() for v in (x, dy, hs[0] if hs else zero, d, h, *(() if g is None else (g,))))
    floor = 2.0 ** -126 * 4 * t * big ** 3
    return {k: (v, tol + floor) for k, (v, tol) in out.items()}


def close(name, got, ref):
    want, tol = ref
    fi = torch.finfo(got.dtype)
    tol = tol + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps
    assert torch.isfinite(got).all(), name
    worst = ((got.double() - want).abs() / tol).max().item() if want.numel() else 0.0
    print(f"[{name}] worst error / tolerance {worst:.3g}")
    assert worst <= 1.0, (name, worst)


def run_case(s, lengths=None):
    from stft_mel_spectrogram_amd import (gated_recurrence, gated_recurrence_backward, gated_recurrence_forward)
    args = (s["x"], s["forget"], s["gate"], s["state"])
    y, last, saved = gated_recurrence_forward(*args, lengths=lengths)
    grads = gated_recurrence_backward(s["dy"], *args, saved, lengths=lengths, grad_state=s["dlast"])
    ref = reference(s, lengths)
    got = dict(y=y, last=last, dx=grads[0], dforget=grads[1])
    if s["gate"] is not None:
        got["dgate"] = grads[2]
    if s["state"] is not None:
        got["dstate"] = grads[3]
    for name, v in got.items():
        close(name, v, ref[name])
    y2, last2 = gated_recurrence(*args, lengths=lengths)
    close("y alone", y2, ref["y"])
    close("last alone", last2, ref["last"])
    return got


# one frame, the walk of few frames, tiles of every size and their borders
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t", [1, 2, 8, 9, 63, 64, 65, 128, 129, 255, 300, 520, 777])
def test_lengths(t, dtype):
    run_case(inputs(2, t, 40, DT[dtype], t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c", [1, 2, 3, 4, 5, 7, 16, 17, 31, 33, 63, 64, 65, 130])
def test_channels(c, dtype):
    for t in (5, 70, 300):
        run_case(inputs(2, t, c, DT[dtype], c + t))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate,state", [(False, False), (False, True), (True, False)])
def test_without_gate_or_state(gate, state, dtype):
    for t in (3, 200):
        run_case(inputs(3, t, 24, DT[dtype], t, gate, state))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_take_wider_ones(dtype):
    for b, c in ((260, 64), (130, 70)):
        for t in (40, 130):
            run_case(inputs(b, t, c, DT[dtype], b))


# few channels and many frames: time ranges that are joined
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("b,t,c", [(1, 5000, 8), (2, 4099, 37), (1, 9001, 1)])
def test_time_ranges(b, t, c, dtype):
    s = inputs(b, t, c, DT[dtype], t, shift=4.0)
    run_case(s)
    run_case(s, torch.tensor([t - 1700] * b, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t", [6, 90, 400, 3000])
def test_lengths_of_entries(t, dtype):
    """Ragged entries, empty ones, lengths out of range; NaN past them does no harm."""
    b = 6
    s = inputs(b, t, 20, DT[dtype], t)
    n = torch.tensor([t, 0, 1, t // 2, t + 5, -3], dtype=torch.int32, device="cuda")
    past = torch.arange(t, device="cuda") >= n.clamp(0, t)[:, None]
    want = run_case(s, n)
    for k in ("x", "forget", "gate", "dy"):
        s[k] = s[k].clone()
        s[k][past] = float("nan")
    got = run_case(s, n)
    for k in got:
        assert torch.equal(got[k], want[k]), k
        if got[k].dim() == 3:
            assert (got[k][past] == 0).all()
    assert torch.equal(got["last"][1], s["state"][1]) and torch.equal(got["dstate"][1], s["dlast"][1])


@pytest.mark.parametrize("t", [4, 100])
def test_infinite_forget(t):
    """+inf keeps the state, -inf replaces it: packed sequences."""
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, t, 12, torch.float32, t, gate=False)
    f = s["forget"].clone()
    f[:, 1] = float("inf")
    f[:, t - 2] = float("-inf")
    y, last = gated_recurrence(s["x"], f, None, s["state"])
    assert torch.equal(y[:, 1], y[:, 0]) or t - 2 == 1
    assert torch.equal(y[:, t - 2], s["x"][:, t - 2])
    again, _ = gated_recurrence(s["x"][:, t - 2:], f[:, t - 2:])
    assert (again[:, 1] - last).abs().max() <= 16 * U * (1 + last.abs().max())


def test_large_arguments():
    """Gates and forgets far out: no overflow, no NaN."""
    s = inputs(2, 80, 16, torch.float32, 3)
    for k in ("forget", "gate"):
        s[k] = s[k] * 40
    run_case(s)


def test_pieces_equal_the_whole():
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, 700, 33, torch.float32, 5)
    whole = reference(s)
    h = s["state"].clone()
    ys = []
    for a, b in ((0, 1), (1, 5), (5, 300), (300, 301), (301, 700)):
        y, h2 = gated_recurrence(*(s[k][:, a:b] for k in ("x", "forget", "gate")), h, out_state=h)
        assert h2 is h
        ys.append(y)
    close("y", torch.cat(ys, 1), whole["y"])
    close("last", h, whole["last"])


@pytest.mark.parametrize("t,c", [(1, 70), (3000, 9)])
def test_state_in_place(t, c):
    """out_state may be the state itself, also where time ranges are joined."""
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(3, t, c, torch.bfloat16, t)
    y, last = gated_recurrence(s["x"], s["forget"], s["gate"], s["state"])
    h = s["state"].clone()
    out = torch.full_like(y, 7.0)
    y2, h2 = gated_recurrence(s["x"], s["forget"], s["gate"], h, out=out, out_state=h)
    assert y2 is out and h2 is h and torch.equal(y2, y) and torch.equal(h, last)


def test_empty():
    from stft_mel_spectrogram_amd import (gated_recurrence, gated_recurrence_backward, gated_recurrence_forward)
    h = torch.randn(2, 5, device="cuda")
    e = torch.empty(2, 0, 5, device="cuda")
    y, last = gated_recurrence(e, e, e, h)
    assert y.shape == (2, 0, 5) and torch.equal(last, h)
    y, last = gated_recurrence(e, e)
    assert (last == 0).all()
    y, last, saved = gated_recurrence_forward(e, e, e, h)
    assert torch.equal(last, h) and saved.shape == (2, 0, 5)
    dx, df, dg, ds = gated_recurrence_backward(e, e, e, e, h, saved, grad_state=last)
    assert dx.shape == e.shape and torch.equal(ds, last)
    n = torch.empty(0, 9, 5, device="cuda")
    y, last = gated_recurrence(n, n)
    assert y.shape == (0, 9, 5) and last.shape == (0, 5)


def test_strides():
    """Time outermost, a broadcast forget, an odd offset; guards around the results."""
    from stft_mel_spectrogram_amd import gated_recurrence_backward, gated_recurrence_forward
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    b, t, c = 3, 150, 21
    base = torch.randn(t, b, 3 * c + 1, generator=g, device="cuda").bfloat16()
    x = base[..., 1:c + 1].transpose(0, 1)
    f = torch.randn(c, generator=g, device="cuda").bfloat16().expand(b, t, c)
    gate = base[..., 2 * c:3 * c].transpose(0, 1)
    dy = torch.randn(t, b, c, generator=g, device="cuda").bfloat16().transpose(0, 1)
    got = gated_recurrence_forward(x, f, gate)
    want = gated_recurrence_forward(*(v.contiguous() for v in (x, f, gate)))
    for a, e in zip(got, want):
        assert torch.equal(a, e)
    got = gated_recurrence_backward(dy, x, f, gate, None, got[2])
    want = gated_recurrence_backward(dy.contiguous(), x.contiguous(), f.contiguous(), gate.contiguous(), None, want[2])
    for a, e in zip(got[:3], want[:3]):
        assert torch.equal(a, e)
    from stft_mel_spectrogram_amd import gated_recurrence
    room = torch.full((b * t * c + 64,), 9.0, device="cuda", dtype=torch.bfloat16)
    out = room[32:-32].view(b, t, c)
    gated_recurrence(x, f, gate, out=out)
    assert (room[:32] == 9).all() and (room[-32:] == 9).all()


@pytest.mark.parametrize("state,gate", [(True, True), (False, False)])
def test_autograd_and_differences(state, gate):
    """Through autograd, against central differences of the 64-bit forward."""
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, 90, 10, torch.float32, 12, gate, state)
    names = [k for k in ("x", "forget", "gate", "state") if s[k] is not None]
    leaves = {k: s[k].detach().clone().requires_grad_(True) for k in names}
    y, last = gated_recurrence(*(leaves.get(k) for k in ("x", "forget", "gate", "state")))
    w = torch.randn(2, 10, device="cuda")
    ((y * s["dy"]).sum() + (last * w).sum()).backward()

    def value(at):
        r = reference(dict(s, **at, dlast=None))
        return (r["y"][0] * s["dy"].double()).sum() + (r["last"][0] * w.double()).sum()

    ref = reference(dict(s, dlast=w))
    for k, r in zip(("x", "forget", "gate", "state"), ("dx", "dforget", "dgate", "dstate")):
        if k not in leaves:
            continue
        way = torch.randn_like(s[k]).double()
        step = 1e-5
        up, down = ({k: s[k].double() + sign * step * way} for sign in (1, -1))
        diff = (value(up) - value(down)).item() / (2 * step)
        want, tol = ref.get(r, (None, None)) if r in ref else (None, None)
        got = (leaves[k].grad.double() * way).sum().item()
        room = ((tol + U * want.abs()) * way.abs()).sum().item() if want is not None else 0.0
        # the differences' own: third derivatives of order 1 per element times step^2, cancellation of 2^-52
        assert abs(got - diff) <= room + 1e-6 * (1 + abs(diff)), (k, got, diff)


def test_unused_results_and_needs():
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, 70, 8, torch.float32, 13)
    x = s["x"].clone().requires_grad_(True)
    y, last = gated_recurrence(x, s["forget"], s["gate"], s["state"])
    g1, = torch.autograd.grad(last.sum(), x, retain_graph=True)
    want = reference(dict(s, dy=torch.zeros_like(s["dy"]), dlast=torch.ones_like(s["state"])))
    close("dx of the last state", g1, want["dx"])
    g2, = torch.autograd.grad(y.sum(), x)
    want = reference(dict(s, dy=torch.ones_like(s["dy"]), dlast=None, state=s["state"]))
    close("dx of y", g2, want["dx"])
    with torch.no_grad():
        gated_recurrence(x, s["forget"], out=torch.empty_like(s["dy"]))
    with pytest.raises(ValueError):
        gated_recurrence(x, s["forget"], out=torch.empty_like(s["dy"]))


def test_streams_and_repeats():
    from stft_mel_spectrogram_amd import gated_recurrence_backward, gated_recurrence_forward
    s = inputs(2, 4000, 20, torch.bfloat16, 14)
    args = (s["x"], s["forget"], s["gate"], s["state"])
    want = gated_recurrence_forward(*args)
    wantg = gated_recurrence_backward(s["dy"], *args, want[2], grad_state=s["dlast"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for st in streams:
        with torch.cuda.stream(st):
            r = gated_recurrence_forward(*args)
            results.append((*r, *gated_recurrence_backward(s["dy"], *args, r[2], grad_state=s["dlast"])))
    torch.cuda.synchronize()
    for r in results:
        for a, e in zip(r, (*want, *wantg)):
            assert torch.equal(a, e)


@pytest.mark.parametrize("t", [1, 60, 3000])
def test_captured(t):
    """Replays against new inputs and a state that goes on in place."""
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, t, 12, torch.float16, t)
    x, f, g = (s[k].clone() for k in ("x", "forget", "gate"))
    h, hr = s["state"].clone(), s["state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gated_recurrence(x, f, g, h.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = gated_recurrence(x, f, g, h, out_state=h)
    for i in range(4):
        n = inputs(2, t, 12, torch.float16, 100 + i)
        for a, k in ((x, "x"), (f, "forget"), (g, "gate")):
            a.copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        want, hr = gated_recurrence(n["x"], n["forget"], n["gate"], hr)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, hr)
