"""The host side of the recurrence, the RMS norm, the distillation and the
adjusted logits (argument checks, split rules, workspace layouts) built with g++
under AddressSanitizer and UndefinedBehaviorSanitizer, the launches stubbed by
functions that write the whole of every workspace region a kernel uses."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "stft_mel_spectrogram_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host_sanitize")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_frame_operators_host_side_under_asan_and_ubsan(tmp_path):
    exe = str(tmp_path / "fm_frames_sanitized")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           *(os.path.join(CSRC, f) for f in ("fm_plan.cpp", "fm_api.cpp", "fm_seq.cpp", "fm_logit.cpp")),
           *(os.path.join(HERE, f) for f in ("device_stubs.cpp", "frame_stubs.cpp", "frame_driver.cpp")),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    print(r.stdout[-2000:])
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
