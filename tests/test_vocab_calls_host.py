"""Host-side tests of calls at the vocabulary matrix that the header allows (no
GPU, no kernel launched), in a build of the host code with AddressSanitizer and
UndefinedBehaviorSanitizer (tests/host/vocab_calls_driver.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_distributed_optimizer_amd", "csrc")


def hipcc():
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        pytest.skip("hipcc not available")
    return path


def test_allowed_calls_under_host_sanitizers(tmp_path):
    import torch
    if torch.cuda.is_available():
        pytest.skip("runs on a host without a GPU (the plans must stay host-only)")
    exe = str(tmp_path / "vocab_calls_driver")
    cmd = [hipcc(), "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(ROOT, "tests", "host", "vocab_calls_driver.cpp"),
           *[os.path.join(CSRC, f) for f in ("plan.cpp", "abi.cpp", "vocab_abi.cpp")], "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "ok: calls that the header allows" in r.stdout
