"""The forget gate's gradient to its own precision, whatever the gate: df = (1 - a) d a
(h' - x), h' the state before the frame.

Tolerances, besides those of dx (the module of the recurrence's tests): a is off by eta of
itself, h' by its own E' (and the joins' roundings), their difference and the two
products by a rounding each: tf = |a (h' - x)| tx + |dx| (a E' + (eta + 3 U) a |h' - x|) + U
|df|.  All of it is in proportion to a: nothing of the size of x alone.
"""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_gated_recurrence import DT, U, close, inputs, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def forget_reference(s, lengths=None):
    """df and its tolerance."""
    x, f = s["x"].double(), s["forget"].double()
    b, t, c = x.shape
    dx, tx = reference(s, lengths)["dx"]
    a, rest = torch.sigmoid(f), torch.sigmoid(-f)
    eta = U * (6 + 1.25 * f.abs())
    joins = U * (32 + t / 64)
    h = s["state"].double() if s["state"] is not None else torch.zeros(b, c, dtype=torch.float64, device=x.device)
    E, H = torch.zeros_like(h), h.abs()
    n = torch.full((b,), t, device=x.device) if lengths is None else lengths.clamp(0, t)
    df, tf = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(t):
        on = (i < n)[:, None]
        step = a[:, i] * (h - x[:, i])
        df[:, i] = dx[:, i] * step
        tf[:, i] = (step.abs() * tx[:, i] + dx[:, i].abs() * (a[:, i] * (E + joins * H) + (eta[:, i] + 3 * U) * step.abs())
                    + U * df[:, i].abs()) * on
        df[:, i] *= on
        mag = a[:, i] * H + (rest[:, i] * x[:, i]).abs()
        E = torch.where(on, a[:, i] * E + (eta[:, i] + 4 * U) * mag, E)
        h = torch.where(on, a[:, i] * h + rest[:, i] * x[:, i], h)
        H = torch.where(on, mag, H)
    return df, tf + 2.0 ** -126


def run(s, lengths=None):
    from stft_mel_spectrogram_amd import gated_recurrence_backward, gated_recurrence_forward
    args = (s["x"], s["forget"], s["gate"], s["state"])
    saved = gated_recurrence_forward(*args, lengths=lengths)[2]
    df = gated_recurrence_backward(s["dy"], *args, saved, lengths=lengths, grad_state=s["dlast"])[1]
    close("dforget", df, forget_reference(s, lengths))
    return df


# nearly shut, nearly open and between
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [-24.0, -18.0, -14.0, -11.0, -8.0, -4.0, 0.0, 6.0, 14.0])
def test_gates(shift, dtype):
    s = inputs(3, 150, 37, DT[dtype], 21, shift=shift)
    if shift < -20:  # float16 ends at 2^-24: a scale that keeps the products above it
        s["dy"], s["dlast"] = s["dy"] * 256, s["dlast"] * 256
    df = run(s)
    assert (df != 0).float().mean() > (0.9 if dtype != "f16" else 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(dtype):
    """One frame, few channels, time ranges, lengths, without gate and state."""
    for b, t, c in ((2, 1, 8), (2, 70, 3), (1, 3000, 12)):
        s = inputs(b, t, c, DT[dtype], t, shift=-9.0)
        run(s)
        run(s, torch.tensor([(t + 1) // 2] * b, dtype=torch.int32, device="cuda"))
    run(inputs(2, 90, 20, DT[dtype], 3, gate=False, state=False, shift=-12.0))


def test_infinite_gates():
    """Gradients of gates at either end are 0, not NaN."""
    from stft_mel_spectrogram_amd import gated_recurrence_backward, gated_recurrence_forward
    s = inputs(2, 80, 8, torch.float32, 4)
    f = s["forget"].clone()
    f[:, 5], f[:, 40] = float("inf"), float("-inf")
    saved = gated_recurrence_forward(s["x"], f, s["gate"], s["state"])[2]
    grads = gated_recurrence_backward(s["dy"], s["x"], f, s["gate"], s["state"], saved, grad_state=s["dlast"])
    assert all(torch.isfinite(g).all() for g in grads)
    assert (grads[1][:, 5] == 0).all() and (grads[1][:, 40] == 0).all()


def test_through_autograd():
    from stft_mel_spectrogram_amd import gated_recurrence
    s = inputs(2, 40, 6, torch.float32, 5, shift=-13.0)
    f = s["forget"].clone().requires_grad_(True)
    y, last = gated_recurrence(s["x"], f, s["gate"], s["state"])
    ((y * s["dy"]).sum() + (last * s["dlast"]).sum()).backward()
    close("dforget", f.grad, forget_reference(s))
