"""Every kernel of the recurrence against the 64-bit loop over the frames: 64- and
128-byte rows, several whole tiles one after another (the state carried from tile to
tile, the next tile's loads), time ranges of several tiles; whole entries and ragged ones
with NaN past their ends.  Tolerances as in the recurrence's tests."""
import pytest

torch = pytest.importorskip("torch")
from recurrence_paths import PATHS  # noqa: E402
from test_gpu_forget_gradient import forget_reference  # noqa: E402
from test_gpu_gated_recurrence import DT, close, inputs, run_case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype,shape", [(d, p[1]) for p in PATHS for d in p[0]])
def test_path(dtype, shape):
    b, t, c = shape
    s = inputs(b, t, c, DT[dtype], t + c)
    got = run_case(s)
    close("dforget", got["dforget"], forget_reference(s))
    n = (t - (torch.arange(b, device="cuda") * t) // (b - 1)).int()  # from all frames to none
    past = torch.arange(t, device="cuda") >= n[:, None]
    for k in ("x", "forget", "gate", "dy"):
        s[k] = s[k].masked_fill(past[..., None], float("nan"))
    ragged = run_case(s, n)
    for k, v in ragged.items():
        if v.dim() == 3:
            assert (v[past] == 0).all(), k
    whole = n == t
    assert all(torch.equal(ragged[k][whole], got[k][whole]) for k in got)


@pytest.mark.parametrize("dtype,shape", [("bf16", (8, 700, 1021)), ("f32", (6, 600, 1000)), ("f16", (60, 3000, 64))])
def test_without_gate_and_state(dtype, shape):
    run_case(inputs(*shape, DT[dtype], 5, gate=False, state=False))
