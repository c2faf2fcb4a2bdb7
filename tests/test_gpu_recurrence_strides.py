"""Frames far apart: one or two of them out of a buffer that lies time by time."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("time", [1, 2])
@pytest.mark.parametrize("channels", [3, 40])
def test_few_frames_far_apart(time, channels, dtype):
    from stft_mel_spectrogram_amd import (gated_recurrence, gated_recurrence_backward, gated_recurrence_forward)
    g = torch.Generator(device="cuda")
    g.manual_seed(time)
    b, far = 2, 1 << 22  # 8 MiB and more

    def frames():
        room = torch.randn(time * far, generator=g, device="cuda").to(dtype)
        return room.as_strided((b, time, channels), (channels, far, 1))

    x, f, gate, dy = (frames() for _ in range(4))
    state = torch.randn(b, channels, generator=g, device="cuda")
    dense = [v.contiguous() for v in (x, f, gate, dy)]
    for a, e in zip(gated_recurrence(x, f, gate, state), gated_recurrence(*dense[:3], state)):
        assert torch.equal(a, e)
    if time > 1:
        with pytest.raises(RuntimeError, match="apart"):
            gated_recurrence_forward(x, f, gate, state)
        return
    got, want = gated_recurrence_forward(x, f, gate, state), gated_recurrence_forward(*dense[:3], state)
    for a, e in zip(got, want):
        assert torch.equal(a, e)
    for a, e in zip(gated_recurrence_backward(dy, x, f, gate, state, got[2], grad_state=state),
                    gated_recurrence_backward(dense[3], *dense[:3], state, want[2], grad_state=state)):
        assert torch.equal(a, e)
