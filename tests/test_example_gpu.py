"""The training-step example: the loss falls with both state widths, and the answers from the INT4
codes differ from the bf16 weights' by the quantiser's error alone. A block of 256 normal
weights has its largest near 2.8 sigma, so a step of 2.8 sigma / 7 = 0.4 sigma and a rounding error of
0.4 / sqrt(12) = 0.115 of the weights' norm."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "shard_step.py")


@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_step_example(state_bits):
    spec = importlib.util.spec_from_file_location("shard_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    first, last, off = module.main(steps=40, state_bits=state_bits)
    assert last < 0.2 * first
    assert 0.05 < off < 0.2
