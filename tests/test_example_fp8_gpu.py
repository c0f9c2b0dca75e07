"""The fp8 layer's example runs, and its token's answer from the codes is off by their roundings: each
code by at most half a step, 2^-4 of its value, so each product by at most (1 + 2^-4)^2 - 1 = 0.129, and
a sum of products whose signs are mixed by no more than that of its size."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_layer.py")


def test_fp8_layer_example():
    spec = importlib.util.spec_from_file_location("fp8_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    first, last, off = module.main(rows=200, cols=384, steps=6, batch=96)
    assert math.isfinite(first) and math.isfinite(last)
    assert 0.0 < off < 0.129
