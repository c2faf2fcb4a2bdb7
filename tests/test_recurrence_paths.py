"""The rule that chooses the recurrence's kernels, for the shapes that stand for each of
them (built with g++ from the library's own header)."""
import os
import shutil
import subprocess

import pytest

from recurrence_paths import PATHS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "stft_mel_spectrogram_amd", "csrc")
MAIN = """
#include <cstdio>
#include <cstdlib>
#include "fm_seq.h"
int main(int n, char** v) {
  for (int i = 1; i + 3 < n; i += 4) {
    const int size = std::atoi(v[i]), b = std::atoi(v[i + 1]), t = std::atoi(v[i + 2]), c = std::atoi(v[i + 3]);
    for (int backward = 0; backward < 2; ++backward) {
      const fm::ScanSplit p = fm::scan_split(b, t, c, size, backward != 0);
      const int tile = fm::scan_tile(p.row, p.frames, size), most = p.chunk < t ? p.chunk : t;
      std::printf("%d %d %d %d\\n", p.row, p.frames, p.splits, (most + tile - 1) / tile);
    }
  }
}
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("paths")
    (d / "main.cpp").write_text(MAIN)
    r = subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(d / "main.cpp"), "-o",
                        str(d / "paths")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(size, shape):
        out = subprocess.run([str(d / "paths"), str(size), *map(str, shape)], capture_output=True, text=True, check=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]

    return run


@pytest.mark.parametrize("dtypes,shape,forward,backward", PATHS)
def test_split(dtypes, shape, forward, backward, splits):
    assert splits(4 if dtypes == ("f32",) else 2, shape) == [forward, backward]


def test_every_kernel_is_there():
    """Rows and frames that the launches choose among for four channels and more; one
    walk and time ranges, each with two whole tiles and more."""
    want = {(4, 0): {(64, 2), (128, 4)}, (2, 0): {(64, 4), (128, 4)}, (4, 1): {(64, 2), (128, 2)}, (2, 1): {(128, 2)}}
    for (size, way), kernels in want.items():
        mine = [p[2 + way] for p in PATHS if (p[0] == ("f32",)) == (size == 4)]
        assert {(row, frames) for row, frames, _, tiles in mine if tiles > 2} == kernels
        assert any(n == 1 and tiles > 2 for _, _, n, tiles in mine)
        assert any(n > 1 and tiles > 2 for _, _, n, tiles in mine)
