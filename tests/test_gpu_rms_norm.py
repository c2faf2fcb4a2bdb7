"""RMS norm with the residual's addition, its gradients and its 8-bit output
against the 64-bit formulas.

Tolerances.  A row's sum of squares passes through at most 32 + width / 1024
additions one after another (elements of a lane, lanes, waves, sweeps), so rstd is
off by half of 2^-24 times that and 4 roundings more: U (20 + width / 1024).  Products
and sums of it add single roundings.  Results in 16 bits add half a step, e4m3 2^-4
of the value (2^-10 of the scale below 2^-6), int8 half of the scale.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(rows, width, dtype, seed, wtype=None, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=(r(rows, width) * std).to(dtype), residual=(r(rows, width) * 3 * std).to(dtype),
                w=(r(width) * 0.2 + 1).to(wtype or dtype), dy=r(rows, width).to(dtype),
                dsum=r(rows, width).to(dtype))


def close(name, got, want, tol):
    fi = torch.finfo(got.dtype)
    tol = tol + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps
    assert torch.isfinite(got).all(), name
    worst = ((got.double() - want).abs() / tol).max().item() if want.numel() else 0.0
    print(f"[{name}] worst error / tolerance {worst:.3g}")
    assert worst <= 1.0, (name, worst)


def run_case(s, residual=True, eps=EPS, weight=True):
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_backward, rms_norm_forward
    res, w = (s["residual"] if residual else None), (s["w"] if weight else None)
    total = (s["x"].float() + res.float()).to(s["x"].dtype) if residual else s["x"]
    y, normed, rstd = rms_norm_forward(s["x"], w, res, eps)
    assert torch.equal(normed, total)
    n = total.shape[-1]
    z = total.double()
    wd = w.double() if weight else torch.ones(n, dtype=torch.float64, device="cuda")
    r = (z.square().mean(-1, keepdim=True) + eps) ** -0.5
    rel = U * (20 + n / 1024)
    close("rstd", rstd, r[..., 0], rel * r[..., 0])
    u = z * r
    close("y", y, u * wd, (rel + 3 * U) * (u * wd).abs())
    again = rms_norm(s["x"], w, res, eps)
    for a, e in zip(again if residual else (again,), (y, normed)):
        assert torch.equal(a, e)
    ds = s["dsum"] if residual else None
    dx, dw = rms_norm_backward(s["dy"], normed, w, rstd, ds)
    dy = s["dy"].double()
    g = dy * wd
    m, mabs = (g * u).mean(-1, keepdim=True), (g * u).abs().mean(-1, keepdim=True)
    want = r * (g - u * m) + (ds.double() if residual else 0)
    size = r * (g.abs() + u.abs() * mabs)
    close("dx", dx, want, (3 * rel + 8 * U) * size + U * want.abs())
    if weight:
        rows = z.shape[0]
        chain = rows / 16 + 64  # rows of a workgroup's lane, partial rows
        close("dw", dw, (dy * u).sum(0), (rel + U * chain) * (dy * u).abs().sum(0))
    else:
        assert dw is None
    dx2, none = rms_norm_backward(s["dy"], normed, w, rstd, ds, params=False)
    assert none is None and torch.equal(dx, dx2)
    return y


# one element, every lane layout and its borders, rows that are swept
WIDTHS = [1, 2, 7, 64, 65, 128, 129, 513, 1024, 1025, 2048, 2051, 4096, 4097, 8193, 16385, 20011]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    for rows in (3, 70):
        run_case(inputs(rows, width, DT[dtype], width), residual=rows == 70)


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 65, 1000, 9001])
@pytest.mark.parametrize("width", [80, 1030])
def test_row_counts(rows, width):
    run_case(inputs(rows, width, torch.bfloat16, rows))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_float32_weight(dtype):
    run_case(inputs(40, 300, DT[dtype], 1, torch.float32))
    run_case(inputs(40, 9000, DT[dtype], 1, torch.float32))
    run_case(inputs(40, 300, DT[dtype], 2), weight=False)


def test_no_rows():
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_backward, rms_norm_quantized
    x, w = torch.empty(0, 8, device="cuda"), torch.ones(8, device="cuda")
    y, s = rms_norm(x, w, x)
    assert y.shape == s.shape == (0, 8)
    dx, dw = rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 8) and (dw == 0).all()
    q, scale = rms_norm_quantized(x, w)
    assert q.shape == (0, 8) and scale.shape == (0,)


def test_rows_of_zeros_and_extremes():
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_quantized
    x = torch.zeros(4, 96, device="cuda")
    x[1] = 1e18
    x[2, 3] = float("nan")
    x[3] = 1e-12
    y = rms_norm(x)
    assert (y[0] == 0).all() and (y[1] - 1).abs().max() <= 64 * U and y[2].isnan().all()
    assert (y[3].double() - 1e-12 / (1e-24 + EPS) ** 0.5).abs().max() <= 1e-9 * 64 * U
    for dt in (torch.float8_e4m3fn, torch.int8):
        q, scale = rms_norm_quantized(x, dtype=dt)
        assert scale[0] == 1 and (q[0].float() == 0).all() and scale[2].isnan()
        assert (q[1].float() == (448 if dt == torch.float8_e4m3fn else 127)).all()
    # a scale below the smallest normal number
    tiny = torch.full((1, 64), 1e-42, device="cuda")
    q, scale = rms_norm_quantized(tiny, eps=1.0)
    assert scale[0] == 2.0 ** -126 and torch.isfinite(q.float()).all()


@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("width", [1, 3, 80, 129, 1000, 2051, 8193, 16390])
def test_8_bits(width, dtype, out):
    from stft_mel_spectrogram_amd import rms_norm_quantized
    s = inputs(33, width, DT[dtype], width)
    q, scale, total = rms_norm_quantized(s["x"], s["w"], s["residual"], EPS, out)
    assert torch.equal(total, (s["x"].float() + s["residual"].float()).to(s["x"].dtype))
    z = total.double()
    y = z * (z.square().mean(-1, keepdim=True) + EPS) ** -0.5 * s["w"].double()
    most = 448 if out == torch.float8_e4m3fn else 127
    rel = U * (26 + width / 1024)
    want = y.abs().amax(-1) / most
    assert ((scale.double() - want).abs() <= (rel + 2 * U) * want).all()
    v = y / scale.double()[:, None]
    slack = (rel + 4 * U) * v.abs()
    half = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) if most == 448 else 0.5
    assert ((q.double() - v).abs() <= half + slack).all()
    # rounded to nearest, not only near: the mean error of a rounding is about a quarter of a step
    if width > 500 and most == 127:
        assert (q.double() - v).abs().mean() < 0.27
    q2, scale2 = rms_norm_quantized(total, s["w"], None, EPS, out)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale2, scale)


def test_strides_and_places():
    """Slices of wider rows, the residual updated in place, results in given memory."""
    from stft_mel_spectrogram_amd import rms_norm
    for width in (100, 17000):
        s = inputs(9, width, torch.bfloat16, 4)
        wide = torch.zeros(9, width + 7, device="cuda", dtype=torch.bfloat16)
        wide[:, 3:3 + width] = s["x"]
        y, total = rms_norm(s["x"], s["w"], s["residual"])
        y2, total2 = rms_norm(wide[:, 3:3 + width], s["w"], s["residual"])
        assert torch.equal(y, y2) and torch.equal(total, total2)
        res = s["residual"].clone()
        room = torch.full((9 * width + 32,), 5.0, device="cuda", dtype=torch.bfloat16)
        out = room[16:-16].view(9, width)
        y3, total3 = rms_norm(s["x"], s["w"], res, out=out, out_sum=res)
        assert y3 is out and total3 is res and torch.equal(out, y) and torch.equal(res, total)
        assert (room[:16] == 5).all() and (room[-16:] == 5).all()


def test_leading_axes():
    from stft_mel_spectrogram_amd import rms_norm
    x = torch.randn(2, 3, 5, 40, device="cuda")
    assert torch.equal(rms_norm(x), rms_norm(x.view(30, 40)).view(2, 3, 5, 40))
    assert torch.equal(rms_norm(x[:, :, 2]), rms_norm(x[:, :, 2].contiguous()))


def test_autograd_and_differences():
    from stft_mel_spectrogram_amd import rms_norm
    s = inputs(6, 90, torch.float32, 7)
    leaves = [s[k].clone().requires_grad_(True) for k in ("x", "w", "residual")]
    y, total = rms_norm(*leaves)
    ((y * s["dy"]).sum() + (total * s["dsum"]).sum()).backward()
    assert torch.equal(leaves[0].grad, leaves[2].grad)

    def value(x, w, r):
        z = x + r
        return ((z * (z.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w * s["dy"].double()).sum()
                + (z * s["dsum"].double()).sum())

    d = [v.detach().double() for v in leaves]
    for i in range(3):
        way = torch.randn_like(d[i])
        up, down = ([v + sign * 1e-5 * way if j == i else v for j, v in enumerate(d)] for sign in (1, -1))
        diff = (value(*up) - value(*down)).item() / 2e-5
        got = (leaves[i].grad.double() * way).sum().item()
        # 90 columns: gradients to 64 U of terms of order 4 (the sum rounded to 32 bits included), 540 of them
        assert abs(got - diff) <= 540 * 64 * U * 4 + 1e-6 * abs(diff), i


def test_which_gradients():
    from stft_mel_spectrogram_amd import rms_norm
    s = inputs(5, 40, torch.float32, 9)
    x = s["x"].clone().requires_grad_(True)
    y, total = rms_norm(x, s["w"], s["residual"])
    g, = torch.autograd.grad((total * s["dy"]).sum(), x, retain_graph=True)  # only the sum
    assert torch.equal(g, s["dy"])
    g, = torch.autograd.grad(y.sum(), x)  # only y
    assert torch.isfinite(g).all() and g.abs().max() > 0
    r = s["residual"].clone().requires_grad_(True)
    y, total = rms_norm(s["x"], s["w"], r)
    assert torch.autograd.grad((y * s["dy"]).sum(), r)[0].abs().max() > 0


def test_captured():
    from stft_mel_spectrogram_amd import rms_norm
    x, r, w = (torch.randn(*s, device="cuda").bfloat16() for s in ((64, 200), (64, 200), (200,)))
    rms_norm(x, w, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total = rms_norm(x, w, r, out_sum=r)
    want_r = r.clone()
    for _ in range(4):
        x.copy_(torch.randn(64, 200, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want, want_r = rms_norm(x, w, want_r)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(r, want_r)


def test_gradients_repeat_bit_for_bit():
    from stft_mel_spectrogram_amd import rms_norm_backward, rms_norm_forward
    s = inputs(5000, 700, torch.bfloat16, 11)
    y, n, r = rms_norm_forward(s["x"], s["w"], s["residual"])
    a, b = (rms_norm_backward(s["dy"], n, s["w"], r, s["dsum"]) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
