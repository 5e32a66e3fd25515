"""What importing the package and its host-only functions needs and leaves
alone, each in a process of its own."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("blockwise_bit_codebook_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_one_hip_runtime_whatever_is_imported_first():
    # torch holds a HIP runtime of its own: with another one beside it in the
    # process the GPU cannot be used
    pytest.importorskip("torch")
    maps = "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"
    kb = "import blockwise_bit_codebook_amd as kb; kb.codebook_nf(4)"
    assert python(f"{kb}\nimport torch\n{maps}").split() == ["1"]
    assert python(f"import torch\n{kb}\n{maps}").split() == ["1"]
