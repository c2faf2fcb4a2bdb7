"""Distillation in every row layout and type, with and without the rest: whole rows of
many chunks (a workgroup each), segments of several chunks, 64 lanes of one to four
groups; more entries than a row has lanes.  Tolerances as in the distillation's tests."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_distillation import DT, inputs, run_case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(1300, 9001, 20), (700, 2600, 64), (300, 40009, 7), (3, 131072, 40),
                                            (9, 250, 64), (9, 190, 3), (9, 380, 33), (9, 900, 64)])
def test_layout(rows, vocab, top, dtype, rest):
    run_case(*inputs(rows, vocab, top, DT[dtype], rows + vocab), rest=rest)
    if not rest:
        run_case(*inputs(rows, vocab, top, DT[dtype], rows), tau=3.0)
