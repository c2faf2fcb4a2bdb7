"""Adjusted logits at every segment length of every type (16-byte groups of a lane: 1, 2
and in float32 4, by how many rows there are), against the 64-bit definition on rows
from all over the batch; histories longer than one pass of a workgroup."""
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")
from test_gpu_adjust_logits import DT, inputs, reference  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# type, rows, vocabulary, groups of a lane
SHAPES = [("f32", 600, 5000, 4), ("f32", 150, 17000, 2), ("f32", 40, 9001, 1),
          ("f16", 600, 5000, 2), ("f16", 40, 9001, 1), ("bf16", 300, 16400, 2), ("bf16", 40, 9001, 1)]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_groups_of_a_lane(tmp_path):
    main = tmp_path / "main.cpp"
    calls = "".join(f'  std::printf("%d\\n", fm::adjust_vecs({n}, {v}, {4 if t == "f32" else 8}));\n'
                    for t, n, v, _ in SHAPES)
    main.write_text('#include <cstdio>\n#include "fm_logit.h"\nint main() {\n' + calls + "}\n")
    exe = str(tmp_path / "groups")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "stft_mel_spectrogram_amd", "csrc"), str(main), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [s[3] for s in SHAPES]


@pytest.mark.gpu
@pytest.mark.parametrize("history", [40, 4500])
@pytest.mark.parametrize("dtype,rows,vocab", [s[:3] for s in SHAPES])
def test_segments(dtype, rows, vocab, history):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from stft_mel_spectrogram_amd import adjust_logits
    s = inputs(rows, vocab, history, 70, True, DT[dtype], rows + history)
    got = adjust_logits(**{("logits" if k == "x" else k): v for k, v in s.items()})
    few = torch.tensor([0, 1, rows // 3, rows // 2, rows - 9, rows - 1], device="cuda")
    want, tol, touched = reference({k: v[few] if isinstance(v, torch.Tensor) else v for k, v in s.items()})
    g, x = got[few].cpu(), s["x"][few].cpu()
    assert torch.equal(g[~touched], x[~touched])
    fi = torch.finfo(g.dtype)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(g), fin) and torch.equal(g.double()[~fin], want[~fin])
    tol = tol + fi.eps / 2 * want.abs() + fi.smallest_normal * fi.eps
    worst = ((g.double() - want).abs() / tol)[fin].max().item()
    print(f"worst error / tolerance {worst:.3g}")
    assert worst <= 1.0
