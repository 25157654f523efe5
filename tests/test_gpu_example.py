"""examples/train_and_decode.py as it would be run."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_train_and_decode():
    spec = importlib.util.spec_from_file_location(
        "train_and_decode", os.path.join(ROOT, "examples", "train_and_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, right = example.main()
    assert last < 0.5 * first
    assert right > 0.5
