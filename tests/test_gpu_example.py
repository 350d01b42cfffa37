"""The quantised bottleneck example runs, and its 8-bit result stays near the FP32 one: rows and
weights of ~N(0, 1) rounded to 127 steps of their maximum (about 3.5 and 2.5 standard deviations
over 256 channels) err by step / sqrt(12) each, 0.8 % and 0.6 % of a value; together 1.0 %, and BF16
of the result 0.2 %.  2 % leaves a factor of two."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_quantized_block_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantized_block.py")
    spec = importlib.util.spec_from_file_location("quantized_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert 0.0 < mod.main() < 0.02
