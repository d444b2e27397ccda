"""The example that runs the block operators together: it learns, and a token
decoded alone gives what it gives inside a prompt."""

import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_ternary_blocks():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("ternary_blocks", os.path.join(ROOT, "examples", "ternary_blocks.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, diff = m.main(["--dim", "256", "--blocks", "2", "--steps", "20", "--tokens", "128"])
    assert losses[-1] < 0.8 * losses[0], losses
    # two bf16 roundings of each block's activations apart at most
    assert diff < 2.0 ** -6
