"""The example layer runs, its router's load evens out, and its MXFP4 output is as near
to the bf16 one as rounding both operands to E2M1 leaves it."""
import importlib.util
import os

import pytest

from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu


def test_example_layer():
    ensure_library()
    path = os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples", "mxfp4_layer.py")
    spec = importlib.util.spec_from_file_location("mxfp4_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.main(["--steps", "12"])
    first, last = history[0], history[-1]
    assert last[0] < first[0] and last[1] < first[1]
    # E2M1 rounds a normal value by about a tenth of it (at most a quarter of the block's
    # largest); two operands and sums of independent errors stay below 0.25
    assert all(0.05 < far < 0.25 for _, _, far in history)
