"""Host-side tests of the vocabulary calls (no GPU, no kernel launched): the
library exports what include/zdo_vocab.h declares; the places of parameters, the
workspace layouts and every refusal, in a build of the host code with
AddressSanitizer and UndefinedBehaviorSanitizer (tests/host/vocab_driver.cpp);
the binding's own checks."""

import os
import re
import shutil
import subprocess

import pytest

import zero_distributed_optimizer_amd as Z
from zero_distributed_optimizer_amd import vocab as ZV

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_distributed_optimizer_amd", "csrc")


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "zdo_vocab.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"^\s*[A-Za-z_][\w\s\*]*?\b([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))
    assert len(names) == 6 and sorted(ZV.VOCAB_EXPORTS) == names
    L = Z.require_library()
    for n in names:
        assert hasattr(L, n), n
        assert callable(getattr(Z, n.removeprefix("zdo_")))


def test_checks_and_layouts_under_host_sanitizers(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    import torch
    if torch.cuda.is_available():
        pytest.skip("runs on a host without a GPU (the plans must stay host-only)")
    exe = str(tmp_path / "vocab_driver")
    cmd = [hipcc, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(ROOT, "tests", "host", "vocab_driver.cpp"),
           *[os.path.join(CSRC, f) for f in ("plan.cpp", "abi.cpp", "vocab_abi.cpp")], "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "ok: starts, layouts, refusals" in r.stdout


def test_workspaces_do_not_grow_with_the_logits():
    """n * vocab logits of 4 bytes would be 2.1 GB and 69 GB here."""
    assert Z.linear_cross_entropy_workspace_bytes(4096, 128256, 4096) < 700 << 20
    assert Z.linear_cross_entropy_workspace_bytes(131072, 131072, 1024) < 2 << 30
    assert Z.embedding_grad_workspace_bytes(0, 8) > 0
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 0), (2 ** 22 + 1, 8, 8)):
        with pytest.raises(ValueError, match="out of range"):
            Z.linear_cross_entropy_workspace_bytes(*bad)
    for bad in ((-1, 8), (8, 0), (2 ** 30 + 1, 8)):
        with pytest.raises(ValueError, match="out of range"):
            Z.embedding_grad_workspace_bytes(*bad)


def test_binding_refuses_before_the_library():
    import torch
    plan = Z.build_range_map([1000, 24], 600, 4, 1)
    host = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        Z.embedding_lookup(plan, 0, 10, host, torch.zeros(4, dtype=torch.int64), host)
    with pytest.raises(TypeError, match="torch tensor"):
        Z.embedding_grad(plan, 0, 10, None, None, None, None)
    with pytest.raises(TypeError, match="torch tensor"):
        Z.linear_cross_entropy(plan, 0, 10, host, [[0.0]], None, None, None, None)
    with pytest.raises(ValueError, match="device"):
        Z.linear_cross_entropy_grad(plan, 0, 10, host, host, None, None, None, None, None, None)


def test_calls_on_a_host_only_plan_are_errors():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    L = Z.require_library()
    plan = Z.build_range_map([10, 20], 16, 2, 0)
    h = plan.handle
    assert L.embedding_lookup(h, 0, 1, 4, 16, 32, 1, 1.0, 48, 0, 4, None) == Z.EHIP
    assert L.embedding_grad(h, 0, 1, 4, 16, 1, 32, 0, 4, 1.0, 0, 48, 64, None) == Z.EHIP
    assert L.linear_cross_entropy(h, 0, 1, 4, 16, 32, 4, 48, 1, 64, 80, 96, None) == Z.EHIP
    assert L.linear_cross_entropy_grad(h, 0, 1, 4, 16, 32, 4, 48, 1, 64, 80, 96, 0, 4, 0, 112, 128, None) == Z.EHIP
    assert b"device" in L.zdo_last_error()
