"""What the products' hand-written instructions need of the code around them,
read from the source and from the assembly of a build (no GPU)."""

import glob
import os
import re
import subprocess

from test_vocab_calls_host import CSRC, ROOT, hipcc

from zero_distributed_optimizer_amd import build as ZB


def test_overwritten_registers_are_named():
    """Inline assembly that writes m0 says so."""
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.h*")):
        for block in re.findall(r"asm volatile\((.*?)\);", open(path).read(), flags=re.S):
            code, last = block.split('"', 2)[1], block.rsplit(":", 1)[1]   # instructions, what is overwritten
            if re.search(r"\bm0\b", code):
                seen += 1
                assert '"m0"' in last, (path, block)
    assert seen == 1


def test_m0_belongs_to_the_copies(tmp_path):
    """In the products' code m0 occurs in the copies' instructions only: nothing of
    the compiler's lives there, before or after."""
    out = str(tmp_path / "vocab_gemm.s")
    flags = [f for f in ZB.FLAGS if f not in ("-fPIC", "-shared") and not f.startswith("-Wl")]
    cmd = [hipcc(), *flags, "--cuda-device-only", "-S", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(CSRC, "vocab_gemm.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    assert "inline-asm" not in r.stderr
    written, ours = 0, False
    for line in open(out):
        if "#ASMSTART" in line:
            ours = True
        elif "#ASMEND" in line:
            ours = False
        elif re.search(r"\bm0\b", line.split(";")[0]):
            assert ours and re.fullmatch(r"\s*s_mov_b32 m0, s\d+\s*", line.split(";")[0]), line
            written += 1
    assert written > 100
