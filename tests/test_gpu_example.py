"""The training and serving example runs, learns, and serves what it learned."""

import importlib.util
import os

import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_train_and_serve_8bit():
    say("example: train and serve in 8 bits")
    path = os.path.join(ROOT, "examples", "train_and_serve_8bit.py")
    spec = importlib.util.spec_from_file_location("train_and_serve_8bit", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, error = example.main(["--dim", "64", "--steps", "80", "--length", "64"])
    assert losses[-1] < 0.5 * losses[0]
    assert error < 0.03
