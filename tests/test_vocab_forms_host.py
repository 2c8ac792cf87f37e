"""The forms of the cross entropy's gradients that tests/test_gpu_vocab_exact.py
runs, held to the library's rules (tests/host/vocab_forms.cpp), so that a rule that
changes does not leave a form without a test. No GPU."""

import os
import subprocess

from test_gpu_vocab_exact import WHOLE_CASES
from test_vocab_calls_host import CSRC, ROOT, hipcc


def test_the_cases_take_the_forms_they_name(tmp_path):
    exe = str(tmp_path / "vocab_forms")
    r = subprocess.run([hipcc(), "-x", "hip", "--offload-arch=gfx950", "-O1", "-std=c++17", f"-I{CSRC}",
                        f"-I{os.path.join(ROOT, 'include')}", os.path.join(ROOT, "tests", "host", "vocab_forms.cpp"),
                        "-o", exe], capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    args = [str(x) for n, vocab, dim, before, _ in WHOLE_CASES
            for x in (n, vocab, dim, int(dim % 64 == 0 and before % 8 == 0))]
    r = subprocess.run([exe, *args], capture_output=True, text=True)
    assert r.returncode == 0
    assert r.stdout.splitlines() == [form for *_, form in WHOLE_CASES]


def test_every_form_has_a_case():
    """Both tiles of both sums, with and without splits, in one piece and in
    several, from a copy and in place."""
    forms = [form.split("; ") for *_, form in WHOLE_CASES]
    for part in ("sum", "rows"):
        for tile in (128, 256):
            for split in (False, True):
                assert any(f"{part} {tile}/1" in products.split(", ") if not split else
                           any(x.startswith(f"{part} {tile}/") and not x.endswith("/1") for x in products.split(", "))
                           for _, products in forms), (part, tile, split)
    for how in ("copied", "in place"):
        assert any(how in pieces and int(pieces.split()[0]) >= 3 for pieces, _ in forms)
        assert any("256/" in products and how in pieces and int(pieces.split()[0]) >= 3 for pieces, products in forms)
