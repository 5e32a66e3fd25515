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


def test_import_star_without_torch():
    out = python("import sys; sys.modules['torch'] = None\nfrom blockwise_bit_codebook_amd import *\n"
                 "print(len(codebook_nf(4)), 'rope' in globals())")
    assert out.split() == ["16", "False"]


def test_import_star_before_the_libraries_are_built(tmp_path):
    package = tmp_path / "blockwise_bit_codebook_amd"
    package.mkdir()
    for name in os.listdir(os.path.join(ROOT, "blockwise_bit_codebook_amd")):
        if name.endswith(".py"):
            (package / name).write_text(open(os.path.join(ROOT, "blockwise_bit_codebook_amd", name)).read())
    out = python(f"import sys; sys.path.insert(0, {str(tmp_path)!r})\nfrom blockwise_bit_codebook_amd import *\n"
                 "print(n_words(33, 4))\n"
                 "try:\n    codebook_nf(4)\nexcept ImportError as e:\n    print('build' in str(e))")
    assert out.split() == ["8", "True"]


def test_import_star_with_both():
    pytest.importorskip("torch")
    out = python("from blockwise_bit_codebook_amd import *\nprint(rope.__module__, codebook_nf.__module__)")
    assert out.split() == ["blockwise_bit_codebook_amd.layer", "blockwise_bit_codebook_amd"]
