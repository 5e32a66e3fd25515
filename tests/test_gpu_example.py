"""The example's chain (int8 projection, head norms with rotation, paged
append) for prompts and single tokens: the script itself compares both."""

import importlib.util
import os

import pytest

from tests.gpu_util import case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [["--tokens", "300", "--hidden", "512", "--heads", "6", "--kv-heads", "2"],
                                  ["--tokens", "50", "--steps", "2", "--hidden", "500", "--heads", "3", "--kv-heads", "1",
                                   "--dim", "80"]])
def test_attention_input(args):
    case(f"attention input example {args}")
    spec = importlib.util.spec_from_file_location("attention_input", os.path.join(ROOT, "examples", "attention_input.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.main(args)
