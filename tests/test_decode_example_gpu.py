"""The example of a decode loop gives the plain form's result."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("steps", [1, 33, 200])
def test_decode_steps(detfold_lib, steps):
    path = os.path.join(ROOT, "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # float32 out: the query, the keys and the values are the same bfloat16
    # values on both sides but where a rounding of the rotated ones falls the
    # other way, one bfloat16 step (2^-7) of values of about 1 to 4, and what is
    # left is binary32's.
    assert example.main(steps) < 2.0 ** -5
