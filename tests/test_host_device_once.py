"""A kernel's attributes are set once on every device that launches it, on the
CPU (a process with several GPUs; the first call's device alone is not enough)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "stft_mel_spectrogram_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_once_on_every_device(tmp_path):
    exe = str(tmp_path / "device_once")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "host_sanitize", "device_once_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=60)
    assert r.returncode == 0, (r.stdout, r.stderr[-3000:])


def test_no_attribute_is_set_once_per_process():
    """No function-local constant holds the status of setting one."""
    import glob
    import re
    for f in glob.glob(os.path.join(CSRC, "fm_*")):
        src = open(f, encoding="utf-8").read()
        assert not re.search(r"static\s+const\s+\w+\s+\w+\s*=[^;]*(lds_opt_in|hipFuncSetAttribute)", src), f
